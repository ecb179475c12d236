// tree_positions.cu -- where the nodes of draft trees, or the rows of chains, stand.
//
// A node's position is prefix_len + context_len[b] + its depth.  Depths come by pointer jumping:
// every node adds the count of the ancestor that it points at and then points at that one's, so
// a tree is done after ceil(log2(depth)) rounds.  Eight bytes a row: the launch and a few
// dependent reads are the whole time.
#include "common.cuh"
#include "kernels.h"

namespace gdn {
namespace {

constexpr int kThreads = 256;

// rows, and their positions, are in range
__device__ __forceinline__ bool in_range(const PositionArgs& a, int first, int stop, int ctx) {
  return first >= 0 && stop >= first && stop <= a.T && stop - first <= a.N && ctx >= 0;
}

__global__ void __launch_bounds__(kThreads) chain_positions_kernel(const PositionArgs a) {
  const int groups = gridDim.x / a.B, b = blockIdx.x / groups;
  const int first = a.cu[b], stop = a.cu[b + 1], ctx = a.context_len ? a.context_len[b] : 0;
  const int j0 = (blockIdx.x % groups) * kThreads;
  const long long start = (long long)a.prefix_len + ctx;
  if (!in_range(a, first, stop, ctx) || start + (stop - first) - 1 > 0x7fffffffll) {
    if (a.dev_status && j0 == 0 && threadIdx.x == 0)
      atomicMax(a.dev_status + b, GDN_TREE_STATUS_BAD_LAYOUT);
    return;
  }
  // (the grid has a CTA for each kThreads of the most rows there may be)
  const int j = j0 + threadIdx.x;
  if (j < stop - first) a.positions[first + j] = (int)(start + j);
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
  const int first = a.cu[b], stop = a.cu[b + 1], ctx = a.context_len ? a.context_len[b] : 0;
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
  const long long groups = a.N > kThreads ? ((long long)a.N + kThreads - 1) / kThreads : 1;
  if (groups * a.B > 0x7fffffffll) return cudaErrorInvalidConfiguration;
  chain_positions_kernel<<<(unsigned)(groups * a.B), kThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace gdn
