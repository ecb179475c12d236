// tree_positions.cu -- where the nodes of draft trees, or the rows of chains, stand.
//
// A node's position is prefix_len + context_len[b] + its depth.  Depths come by pointer jumping:
// every node adds the count of the ancestor that it points at and then points at that one's, so
// a tree is done after ceil(log2(depth)) rounds.  Eight bytes a row: the launch, a few dependent
// reads and a barrier a round are the whole time.  One GB300, in a CUDA graph: 32 trees of 128
// nodes 1.8 us, 256 of 1 to 1024 nodes 3.5, chains of up to 32768 rows 1.7.
#include "common.cuh"
#include "kernels.h"

namespace gdn {
namespace {

constexpr int kThreads = 256;

// the rows and the context of a sequence are in range
__device__ __forceinline__ bool in_range(const PositionArgs& a, int first, int stop, int ctx) {
  return first >= 0 && stop >= first && stop <= a.T && stop - first <= a.N && ctx >= 0;
}
__device__ __forceinline__ int context_of(const PositionArgs& a, int b) {
  return a.context_len ? a.context_len[b] : 0;
}

// A thread a row, which looks its sequence up: a grid over the rows there are is right for batches
// of any raggedness, and for any number of sequences.
__global__ void __launch_bounds__(kThreads) chain_positions_kernel(const PositionArgs a) {
  const long long x = (long long)blockIdx.x * kThreads + threadIdx.x;
  const auto fits = [&](int b, long long* start) {
    const int first = a.cu[b], stop = a.cu[b + 1], ctx = context_of(a, b);
    *start = (long long)a.prefix_len + ctx;
    return in_range(a, first, stop, ctx) && *start + (stop - first) - 1 <= 0x7fffffffll;
  };
  long long start;
  if (x < a.B && a.dev_status && !fits((int)x, &start))
    atomicMax(a.dev_status + x, GDN_TREE_STATUS_BAD_LAYOUT);
  if (x >= a.T) return;
  const int t = (int)x;
  int lo = -1, hi = a.B + 1;  // the last b with cu[b] <= t (whatever cu holds, within [-1, B])
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (a.cu[mid] <= t) lo = mid;
    else hi = mid;
  }
  if (lo < 0 || lo >= a.B || !fits(lo, &start)) return;
  const int j = t - a.cu[lo];
  if (t < a.cu[lo + 1]) a.positions[t] = (int)(start + j);
}

// a barrier of the first `threads` threads, and whether x holds for any of them
__device__ __forceinline__ bool sync_any(int threads, bool x) {
  uint32_t any;
  asm volatile(
      "{.reg .pred p, q; setp.ne.u32 q, %1, 0;\n"
      "barrier.red.or.pred p, 1, %2, q; selp.u32 %0, 1, 0, p;}"
      : "=r"(any)
      : "r"((uint32_t)x), "r"(threads)
      : "memory");
  return any != 0;
}

__global__ void __launch_bounds__(kMaxNLong) tree_positions_kernel(const PositionArgs a) {
  // a node's count so far (high half) and the ancestor it points at, plus 1 (low half), of the
  // last round and of this one
  __shared__ uint32_t nodes[2][kMaxNLong];
  const int b = blockIdx.x, t = threadIdx.x;
  const int first = a.cu[b], stop = a.cu[b + 1], ctx = context_of(a, b);
  if (!in_range(a, first, stop, ctx)) {
    if (a.dev_status && t == 0) atomicMax(a.dev_status + b, GDN_TREE_STATUS_BAD_LAYOUT);
    return;
  }
  // (the warps of a smaller tree's missing nodes leave)
  const int n = stop - first, threads = (n + 31) / 32 * 32;
  if (t >= threads) return;
  int up = t < n ? a.parent[first + t] : -1;
  uint32_t depth = up >= 0;
  const bool bad = up < -1 || up >= t;
  nodes[0][t] = bad ? 0u : depth << 16 | (uint32_t)(up + 1);
  if (sync_any(threads, bad)) {
    if (a.dev_status && t == 0) atomicMax(a.dev_status + b, GDN_TREE_STATUS_BAD_TREE);
    return;
  }
  // (a round at least halves the longest way to a root, and reads what the one before wrote)
  for (int now = 0; sync_any(threads, up >= 0); now ^= 1) {
    if (up >= 0) {
      const uint32_t next = nodes[now][up];
      depth += next >> 16;
      up = (int)(next & 0xffffu) - 1;
    }
    nodes[now ^ 1][t] = depth << 16 | (uint32_t)(up + 1);
  }
  const long long at = (long long)a.prefix_len + ctx + depth;
  if (sync_any(threads, t < n && at > 0x7fffffffll)) {
    if (a.dev_status && t == 0) atomicMax(a.dev_status + b, GDN_TREE_STATUS_BAD_LAYOUT);
    return;
  }
  if (t < n) a.positions[first + t] = (int)at;
}

}  // namespace

cudaError_t launch_tree_positions(const PositionArgs& a, cudaStream_t stream) {
  if (a.parent) {
    const int threads = a.N > 32 ? (a.N + 31) / 32 * 32 : 32;
    tree_positions_kernel<<<a.B, threads, 0, stream>>>(a);
    return cudaGetLastError();
  }
  const long long threads = a.T > a.B ? a.T : a.B;
  const unsigned blocks = (unsigned)((threads + kThreads - 1) / kThreads);
  chain_positions_kernel<<<blocks, kThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace gdn
