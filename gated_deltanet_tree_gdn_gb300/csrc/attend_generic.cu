// attend_generic.cu -- attention over a paged cache with a shared prefix, any shape and
// type, on CUDA cores in fp32.
//
// A CTA takes kM query rows (row = node * G + g of one sequence and key head) and runs
// over the keys they see -- the prefix's pages, the sequence's own pages, the tree's own
// rows -- kN at a time with the running maximum and sum of a softmax:
//     m' = max(m, max_j s_j),  l' = l e^{m-m'} + sum_j e^{s_j-m'},
//     O' = O e^{m-m'} + sum_j e^{s_j-m'} v_j,
// and divides by l at the end.  The mask is applied by selection, never by adding, and
// rows past a length are not read, so what they hold does not matter.  m starts at
// -inf; while it is, the rescaling factor is taken as 0 and nothing is subtracted.
#include "common.cuh"
#include "kernels.h"

namespace gdn {
namespace {

constexpr int kThreads = 128;
constexpr int kM = 16, kN = 32;
constexpr int kLanes = kThreads / kM;   // threads a row (one warp holds whole rows)
constexpr int kKeys = kN / kLanes;      // keys a thread
constexpr int kCols = kMaxD / kLanes;   // output columns a thread, at most
constexpr int kPad = 4;

template <typename T>
__global__ void __launch_bounds__(kThreads)
attend_generic_kernel(const T* __restrict__ q, const T* __restrict__ k, const T* __restrict__ v,
                      const int32_t* __restrict__ parent, const int32_t* __restrict__ cu,
                      const T* __restrict__ k_cache, const T* __restrict__ v_cache,
                      const int32_t* __restrict__ table, const int32_t* __restrict__ context_len,
                      const int32_t* __restrict__ prefix_pages, float scale, T* __restrict__ o,
                      float* __restrict__ lse, gdn_tree_attend_dims d, int tiles,
                      int32_t* dev_status) {
  extern __shared__ float smem[];
  const int ld = d.D + kPad;
  float* sQ = smem;               // [kM][ld]
  float* sK = sQ + kM * ld;       // [kN][ld]
  float* sV = sK + kN * ld;       // [kN][ld]
  float* sP = sV + kN * ld;       // [kM][kN + 1]
  uint32_t* sAnc = reinterpret_cast<uint32_t*>(sP + kM * (kN + 1));  // [kM][kMaxNLong / 32]
  int32_t* sParent = reinterpret_cast<int32_t*>(sAnc + kM * (kMaxNLong / 32));  // [N]
  __shared__ long long sRow[kN];  // the key's row in its array, -1: none

  const int tile = blockIdx.x % tiles;
  const int hk = (blockIdx.x / tiles) % d.Hkv;
  const int b = blockIdx.x / tiles / d.Hkv;
  const int tid = threadIdx.x, r = tid / kLanes, ln = tid % kLanes;
  const int G = d.Hq / d.Hkv;

  const int first = cu[b], stop = cu[b + 1], n = stop - first, ctx = context_len[b];
  const long long cap = (long long)d.table_width * d.page_size;
  if (first < 0 || n < 0 || stop > d.T || n > d.N || ctx < 0 || ctx > cap) {
    if (dev_status && tid == 0) atomicMax(dev_status + b, GDN_TREE_STATUS_BAD_LAYOUT);
    return;
  }
  if (tile * kM >= n * G) return;
  const bool tree = k != nullptr && parent != nullptr;
  if (tree) {
    bool bad = false;
    for (int i = tid; i < n; i += kThreads) {
      const int p = parent[first + i];
      bad |= p < -1 || p >= i;
      sParent[i] = p;
    }
    for (int i = tid; i < kM * (kMaxNLong / 32); i += kThreads) sAnc[i] = 0u;
    if (__syncthreads_or(bad)) {
      if (dev_status && tid == 0) atomicMax(dev_status + b, GDN_TREE_STATUS_BAD_TREE);
      return;
    }
  }
  const int gr = tile * kM + r;  // this thread's row: node gr / G, head hk * G + gr % G
  const int node = gr / G;
  const bool live = gr < n * G;
  if (tree && ln == 0 && live)
    for (int a = node; a >= 0; a = sParent[a]) sAnc[r * (kMaxNLong / 32) + (a >> 5)] |= 1u << (a & 31);
  for (int e = tid; e < kM * d.D; e += kThreads) {
    const int rr = e / d.D, c = e - rr * d.D, g2 = tile * kM + rr;
    sQ[rr * ld + c] = g2 < n * G ? scale * to_f32(q[((size_t)(first + g2 / G) * d.Hq + hk * G + g2 % G) * d.D + c]) : 0.f;
  }

  float m = -INFINITY, l = 0.f, O[kCols];
#pragma unroll
  for (int i = 0; i < kCols; ++i) O[i] = 0.f;
  const int nown = k != nullptr ? n : 0;
  const int total[3] = {d.prefix_len, ctx, nown};
  for (int part = 0; part < 3; ++part) {
    const T* kb = part == 2 ? k : k_cache;
    const T* vb = part == 2 ? v : v_cache;
    for (int j0 = 0; j0 < total[part]; j0 += kN) {
      __syncthreads();  // the previous keys have been used
      if (tid < kN) {
        const int j = j0 + tid;
        long long row = -1;
        if (j < total[part]) {
          if (part == 2) {
            row = first + j;
          } else {
            const int pg = part == 0 ? prefix_pages[j / d.page_size]
                                     : table[(size_t)b * d.table_width + j / d.page_size];
            if (pg >= 0 && pg < d.n_pages)
              row = (long long)pg * d.page_size + j % d.page_size;
            else if (dev_status)
              atomicMax(dev_status + b, GDN_TREE_STATUS_BAD_LAYOUT);
          }
        }
        sRow[tid] = row;
      }
      __syncthreads();
      for (int e = tid; e < kN * d.D; e += kThreads) {
        const int j = e / d.D, c = e - j * d.D;
        const long long row = sRow[j];
        const size_t at = ((size_t)row * d.Hkv + hk) * d.D + c;
        sK[j * ld + c] = row >= 0 ? to_f32(kb[at]) : 0.f;
        sV[j * ld + c] = row >= 0 ? to_f32(vb[at]) : 0.f;
      }
      __syncthreads();
      float s[kKeys], top = m;
      bool seen[kKeys];
#pragma unroll
      for (int i = 0; i < kKeys; ++i) {
        const int j = ln + kLanes * i;
        float acc = 0.f;
        const float* qr = sQ + r * ld;
        const float* kr = sK + j * ld;
        for (int c = 0; c < d.D; c += 4) {
          const float4 a = *reinterpret_cast<const float4*>(qr + c);
          const float4 x = *reinterpret_cast<const float4*>(kr + c);
          acc = fmaf(a.x, x.x, fmaf(a.y, x.y, fmaf(a.z, x.z, fmaf(a.w, x.w, acc))));
        }
        bool sees = live && sRow[j] >= 0;
        if (part == 2) {
          const int jj = j0 + j;
          if (!tree) sees = sees && jj <= node;
          else sees = sees && ((sAnc[r * (kMaxNLong / 32) + (jj >> 5 & (kMaxNLong / 32 - 1))] >> (jj & 31)) & 1u);
        }
        seen[i] = sees;
        s[i] = sees ? acc : -INFINITY;
        top = fmaxf(top, s[i]);
      }
#pragma unroll
      for (int off = 1; off < kLanes; off <<= 1)
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
      const float base = top == -INFINITY ? 0.f : top;
      const float keep = m == -INFINITY ? 0.f : expf(m - base);
      float sum = 0.f;
#pragma unroll
      for (int i = 0; i < kKeys; ++i) {
        const float p = expf(s[i] - base);  // (-inf: 0)
        sum += p;
        sP[r * (kN + 1) + ln + kLanes * i] = seen[i] ? p : -1.f;
      }
#pragma unroll
      for (int off = 1; off < kLanes; off <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
      l = l * keep + sum;
      m = top;
      __syncwarp();
#pragma unroll
      for (int i = 0; i < kCols; ++i) O[i] *= keep;
      for (int j = 0; j < kN; ++j) {
        const float p = sP[r * (kN + 1) + j];
        if (p < 0.f) continue;  // not seen, whatever v holds
#pragma unroll
        for (int i = 0; i < kCols; ++i) {
          const int c = ln + kLanes * i;
          if (c < d.D) O[i] = fmaf(p, sV[j * ld + c], O[i]);
        }
      }
    }
  }
  if (!live) return;
  const size_t out = (size_t)(first + node) * d.Hq + hk * G + gr % G;
  const float inv = l > 0.f ? 1.f / l : 0.f;
#pragma unroll
  for (int i = 0; i < kCols; ++i) {
    const int c = ln + kLanes * i;
    if (c < d.D) o[out * d.D + c] = from_f32<T>(O[i] * inv);
  }
  if (lse && ln == 0) lse[out] = m + logf(l);
}

template <typename T>
cudaError_t launch_typed(const AttendArgs& a, cudaStream_t stream) {
  const gdn_tree_attend_dims& d = a.d;
  const int tiles = (d.N * (d.Hq / d.Hkv) + kM - 1) / kM;
  const long long blocks = (long long)d.B * d.Hkv * tiles;
  if (blocks > 0x7fffffffll) return cudaErrorInvalidConfiguration;
  const size_t bytes = sizeof(float) * ((size_t)(kM + 2 * kN) * (d.D + kPad) + kM * (kN + 1)) +
                       sizeof(uint32_t) * kM * (kMaxNLong / 32) + sizeof(int32_t) * (size_t)d.N;
  cudaError_t err = cudaFuncSetAttribute(attend_generic_kernel<T>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize, 64 * 1024);
  if (err != cudaSuccess) return err;
  attend_generic_kernel<T><<<(unsigned)blocks, kThreads, bytes, stream>>>(
      static_cast<const T*>(a.q), static_cast<const T*>(a.k), static_cast<const T*>(a.v),
      a.parent, a.cu, static_cast<const T*>(a.k_cache), static_cast<const T*>(a.v_cache),
      a.page_table, a.context_len, a.prefix_pages, a.scale, static_cast<T*>(a.o), a.lse, d,
      tiles, a.dev_status);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_attend_generic(const AttendArgs& a, cudaStream_t stream) {
  return a.d.dtype == GDN_TREE_BF16 ? launch_typed<__nv_bfloat16>(a, stream)
                                    : launch_typed<float>(a, stream);
}

}  // namespace gdn
