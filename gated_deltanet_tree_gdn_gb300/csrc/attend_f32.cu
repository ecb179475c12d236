// attend_f32.cu -- attention over a paged cache with a shared prefix in fp32, on CUDA cores.
//
// A CTA takes 32 query rows (row = node * G + g of one sequence and key head) and runs over
// the keys they see -- the prefix's pages, the sequence's own pages, the tree's own rows --
// 64 (heads of up to 64) or 32 at a time with the running maximum and sum of a softmax:
//     m' = max(m, max_j s_j),  l' = l e^{m-m'} + sum_j e^{s_j-m'},
//     O' = O e^{m-m'} + sum_j e^{s_j-m'} v_j.
// Where there are few rows a cluster of C CTAs takes them, each every C-th tile of keys, and
// adds up the results through its shared memory:
//     M = max_c m_c,  L = sum_c l_c e^{m_c - M},  o = sum_c O_c e^{m_c - M} / L.
//
// Bound by the latency of the tiles where there are few keys, else by shared memory reads: a
// thread takes 4 rows and kKeys keys of S, then 4 rows and 4 or 8 columns of O, so 16 bytes
// read are worth 8 to 11 multiply-adds.  The next tile's keys and values come meanwhile
// (cp.async, rows past a length filled with zeros; the page numbers a tile further ahead).
//
// The mask is applied by selection, never by adding, and what an own row that is masked for
// some rows holds is not multiplied either (0 * inf).  m starts at -inf; while it is, the
// rescaling factor is taken as 0 and nothing is subtracted.
// 32 trees of 64 nodes with 32 heads of 128 over 768 keys take 0.98 ms (27 TFLOP/s); 3 trees of
// up to 40 nodes over up to 277 keys 13.1 us.
#include <cooperative_groups.h>

#include "common.cuh"
#include "kernels.h"

namespace cg = cooperative_groups;

namespace gdn {
namespace {

constexpr int kThreads = 128, kWarps = kThreads / 32;
constexpr int kM = 32;            // rows: 8 groups of 4, each 16 threads
constexpr int kMaxCluster = 8;
constexpr int kWords = kMaxNLong / 32;

template <int DP>  // D <= DP: 64 or 128
struct Shared {
  static constexpr int kKeys = DP == 64 ? 4 : 2;  // a thread's keys
  static constexpr int kN = 16 * kKeys;
  static constexpr int kLd = DP + 4;  // (rows 16 bytes apart in the banks)
  float K[2][kN][kLd], V[2][kN][kLd];
  float Q[kM][kLd];                   // at the end O
  float P[kN][kM];                    // -1: not seen
  int there[2][kN];                   // the key's row in its array, -1: none
  uint32_t anc[kM][kWords];           // the own nodes that a row sees
  float m[kM], l[kM], w[kM][kMaxCluster];
};

__device__ __forceinline__ void cp_async16_zfill(void* dst, const void* src, bool take) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(
                   (uint32_t)__cvta_generic_to_shared(dst)),
               "l"(src), "r"(take ? 16u : 0u)
               : "memory");
}

__device__ __forceinline__ void fma4(float4& d, float a, float4 b) {
  d.x = fmaf(a, b.x, d.x);
  d.y = fmaf(a, b.y, d.y);
  d.z = fmaf(a, b.z, d.z);
  d.w = fmaf(a, b.w, d.w);
}

template <int DP>
__global__ void __launch_bounds__(kThreads)
attend_f32_kernel(const float* __restrict__ q, const float* __restrict__ k,
                  const float* __restrict__ v, const int32_t* __restrict__ parent,
                  const int32_t* __restrict__ cu, const float* __restrict__ k_cache,
                  const float* __restrict__ v_cache, const int32_t* __restrict__ table,
                  const int32_t* __restrict__ context_len,
                  const int32_t* __restrict__ prefix_pages, float scale, float* __restrict__ o,
                  float* __restrict__ lse, gdn_tree_attend_dims d, int tiles,
                  int32_t* dev_status) {
  using L = Shared<DP>;
  constexpr int kN = L::kN, kKeys = L::kKeys, kJ = DP / 64;
  extern __shared__ __align__(16) unsigned char smem_raw[];
  L& S = *reinterpret_cast<L*>(smem_raw);
  int32_t* sParent = reinterpret_cast<int32_t*>(smem_raw + sizeof(L));  // [N]
  cg::cluster_group cluster = cg::this_cluster();
  const int C = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  const int unit = blockIdx.x / C;
  const int tile = tiles - 1 - unit % tiles;  // (a chain's last rows see the most keys)
  const int hk = (unit / tiles) % d.Hkv;
  const int b = unit / tiles / d.Hkv;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int r0 = 4 * (tid >> 4), kg = tid & 15;  // the thread's rows; its keys kg + 16 i
  const int G = d.Hq / d.Hkv;

  const int first = cu[b], stop = cu[b + 1], n = stop - first, ctx = context_len[b];
  const long long cap = (long long)d.table_width * d.page_size;
  // (stop < first, not n < 0: of two numbers far apart the difference may wrap)
  if (first < 0 || stop < first || stop > d.T || n > d.N || ctx < 0 || ctx > cap) {
    if (dev_status && tid == 0) atomicMax(dev_status + b, GDN_TREE_STATUS_BAD_LAYOUT);
    return;  // (every CTA of the cluster)
  }
  const int rows = min(kM, n * G - tile * kM);
  if (rows <= 0) return;
  const bool own = k != nullptr, tree = own && parent != nullptr;

  // ---- the keys, kN at a time: prefix, context, the own rows up to the last node's ---------
  const int node_end = min(n, (tile * kM + rows - 1) / G + 1);
  const int nP = (d.prefix_len + kN - 1) / kN, nC = (ctx + kN - 1) / kN;
  const int all = nP + nC + (own ? (node_end + kN - 1) / kN : 0);
  const size_t stride = (size_t)d.Hkv * d.D;
  constexpr int kMine = kN / kWarps;  // the keys that a warp copies
  // lanes 0 .. kMine - 1: the row of the warp's key `lane` of tile t, -1 where there is none
  auto rows_of = [&](int t) -> int {
    if (t >= all || lane >= kMine) return -1;
    const bool pre = t < nP, mine = t >= nP + nC;
    const int j = kN * (pre ? t : mine ? t - nP - nC : t - nP) + kMine * warp + lane;
    if (j >= (pre ? d.prefix_len : mine ? node_end : ctx)) return -1;
    if (mine) return first + j;
    const int pi = j / d.page_size;
    const int pg = pre ? prefix_pages[pi] : table[(size_t)b * d.table_width + pi];
    if (pg >= 0 && pg < d.n_pages) return pg * d.page_size + (j - pi * d.page_size);
    if (dev_status) {  // a bad page of the prefix is every sequence's error
      if (!pre) atomicMax(dev_status + b, GDN_TREE_STATUS_BAD_LAYOUT);
      else
        for (int i = 0; i < d.B; ++i) atomicMax(dev_status + i, GDN_TREE_STATUS_BAD_LAYOUT);
    }
    return -1;
  };
  constexpr int kChunks = DP / 4, kAtOnce = 32 / kChunks;
  const int ch = lane % kChunks, sub = lane / kChunks;
  auto fetch = [&](int t, int row, int stage) {
    if (t < all) {
      const bool mine = t >= nP + nC;
      const size_t col = (size_t)hk * d.D + 4 * ch;
      const float *kb = mine ? k : k_cache, *vb = mine ? v : v_cache;
      if (lane < kMine) S.there[stage][kMine * warp + lane] = row;
#pragma unroll
      for (int i = 0; i < kMine; i += kAtOnce) {
        const int x = __shfl_sync(0xffffffffu, row, i + sub), key = kMine * warp + i + sub;
        const bool take = x >= 0 && 4 * ch < d.D;
        const size_t off = take ? x * stride + col : 0;
        cp_async16_zfill(&S.K[stage][key][4 * ch], take ? kb + off : q, take);
        cp_async16_zfill(&S.V[stage][key][4 * ch], take ? vb + off : q, take);
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  int next_row = rows_of(rank);
  fetch(rank, next_row, 0);
  next_row = rows_of(rank + C);

  if (tree) {
    bool bad = false;
    for (int i = tid; i < n; i += kThreads) {
      const int p = parent[first + i];
      bad |= p < -1 || p >= i;
      sParent[i] = p;
    }
    for (int i = tid; i < kM * kWords; i += kThreads) S.anc[0][i] = 0u;
    if (__syncthreads_or(bad)) {
      if (dev_status && tid == 0) atomicMax(dev_status + b, GDN_TREE_STATUS_BAD_TREE);
      asm volatile("cp.async.wait_all;" ::: "memory");
      return;  // (every CTA of the cluster)
    }
    if (tid < rows)
      for (int a = (tile * kM + tid) / G; a >= 0; a = sParent[a]) S.anc[tid][a >> 5] |= 1u << (a & 31);
  }
  auto out_row = [&](int r) {
    const int x = tile * kM + r, node = x / G;
    return (size_t)(first + node) * d.Hq + hk * G + (x - node * G);
  };
  for (int e = tid; e < kM * kChunks; e += kThreads) {
    const int r = e / kChunks, c = 4 * (e % kChunks);
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
    if (r < rows && c < d.D) {
      x = *reinterpret_cast<const float4*>(q + out_row(r) * d.D + c);
      x = make_float4(scale * x.x, scale * x.y, scale * x.z, scale * x.w);
    }
    *reinterpret_cast<float4*>(&S.Q[r][c]) = x;
  }

  float m[4], l[4];
  float4 O[4][kJ];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    m[i] = -INFINITY;
    l[i] = 0.f;
#pragma unroll
    for (int j = 0; j < kJ; ++j) O[i][j] = make_float4(0.f, 0.f, 0.f, 0.f);
  }
  int stage = 0;
  for (int t = rank; t < all; t += C, stage ^= 1) {
    const bool mine = t >= nP + nC;
    asm volatile("cp.async.wait_all;" ::: "memory");
    __syncthreads();  // the tile is there, and the one before has been used
    fetch(t + C, next_row, stage ^ 1);
    next_row = rows_of(t + 2 * C);

    float s[4][kKeys];
    {
      float2 acc[4][kKeys] = {};  // (even and odd columns)
#pragma unroll 4
      for (int c = 0; c < d.D; c += 4) {
        float4 x[kKeys];
#pragma unroll
        for (int i = 0; i < kKeys; ++i)
          x[i] = *reinterpret_cast<const float4*>(&S.K[stage][kg + 16 * i][c]);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const float4 y = *reinterpret_cast<const float4*>(&S.Q[r0 + r][c]);
#pragma unroll
          for (int i = 0; i < kKeys; ++i) {
            fma2(acc[r][i], make_float2(x[i].x, x[i].y), make_float2(y.x, y.y));
            fma2(acc[r][i], make_float2(x[i].z, x[i].w), make_float2(y.z, y.w));
          }
        }
      }
#pragma unroll
      for (int r = 0; r < 4; ++r)
#pragma unroll
        for (int i = 0; i < kKeys; ++i) s[r][i] = acc[r][i].x + acc[r][i].y;
    }
    bool seen[4][kKeys];
#pragma unroll
    for (int i = 0; i < kKeys; ++i) {
      const int key = kg + 16 * i, j = kN * (t - nP - nC) + key;  // (j: of the own rows)
      const bool on = S.there[stage][key] >= 0;
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        bool sees = on;
        if (mine && on)
          sees = tree ? (S.anc[r0 + r][j >> 5] >> (j & 31)) & 1u
                      : j <= (tile * kM + r0 + r) / G;
        seen[r][i] = sees;
        if (!sees) s[r][i] = -INFINITY;
      }
    }
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      float top = m[r];
#pragma unroll
      for (int i = 0; i < kKeys; ++i) top = fmaxf(top, s[r][i]);
#pragma unroll
      for (int off = 1; off < 16; off <<= 1)
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
      const float base = top == -INFINITY ? 0.f : top;
      const float keep = m[r] == -INFINITY ? 0.f : expf(m[r] - base);
      m[r] = top;
      l[r] *= keep;
#pragma unroll
      for (int i = 0; i < kKeys; ++i) {
        s[r][i] = expf(s[r][i] - base);  // (-inf: 0)
        l[r] += s[r][i];  // (this thread's keys; the 16 threads add up at the end)
      }
#pragma unroll
      for (int j = 0; j < kJ; ++j)
        O[r][j] = make_float4(keep * O[r][j].x, keep * O[r][j].y, keep * O[r][j].z, keep * O[r][j].w);
    }
#pragma unroll
    for (int i = 0; i < kKeys; ++i) {
      float4 p = make_float4(s[0][i], s[1][i], s[2][i], s[3][i]);
      if (mine)  // -1: not multiplied
        p = make_float4(seen[0][i] ? p.x : -1.f, seen[1][i] ? p.y : -1.f, seen[2][i] ? p.z : -1.f,
                        seen[3][i] ? p.w : -1.f);
      *reinterpret_cast<float4*>(&S.P[kg + 16 * i][r0]) = p;
    }
    __syncwarp();  // (a row's 16 threads are in one warp)
    if (!mine) {
#pragma unroll 4
      for (int j = 0; j < kN; ++j) {
        const float4 p = *reinterpret_cast<const float4*>(&S.P[j][r0]);
#pragma unroll
        for (int c = 0; c < kJ; ++c) {
          const float4 x = *reinterpret_cast<const float4*>(&S.V[stage][j][4 * kg + 64 * c]);
          fma4(O[0][c], p.x, x);
          fma4(O[1][c], p.y, x);
          fma4(O[2][c], p.z, x);
          fma4(O[3][c], p.w, x);
        }
      }
    } else {
      for (int j = 0; j < kN; ++j) {
        const float4 p = *reinterpret_cast<const float4*>(&S.P[j][r0]);
#pragma unroll
        for (int c = 0; c < kJ; ++c) {
          const float4 x = *reinterpret_cast<const float4*>(&S.V[stage][j][4 * kg + 64 * c]);
          if (!(p.x < 0.f)) fma4(O[0][c], p.x, x);
          if (!(p.y < 0.f)) fma4(O[1][c], p.y, x);
          if (!(p.z < 0.f)) fma4(O[2][c], p.z, x);
          if (!(p.w < 0.f)) fma4(O[3][c], p.w, x);
        }
      }
    }
    __syncwarp();  // P has been read
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
#pragma unroll
  for (int r = 0; r < 4; ++r)
#pragma unroll
    for (int off = 1; off < 16; off <<= 1) l[r] += __shfl_xor_sync(0xffffffffu, l[r], off);

  if (C == 1) {
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      if (r0 + r >= rows) continue;
      const size_t at = out_row(r0 + r);
      const float inv = l[r] == 0.f ? 0.f : 1.f / l[r];  // (NaN is kept)
#pragma unroll
      for (int c = 0; c < kJ; ++c)
        if (4 * kg + 64 * c < d.D)
          *reinterpret_cast<float4*>(o + at * d.D + 4 * kg + 64 * c) = make_float4(
              inv * O[r][c].x, inv * O[r][c].y, inv * O[r][c].z, inv * O[r][c].w);
      if (lse && kg == 0) lse[at] = m[r] + logf(l[r]);
    }
    return;
  }

  // ---- the cluster's sums -------------------------------------------------------------------
  __syncthreads();  // Q has been used
#pragma unroll
  for (int r = 0; r < 4; ++r) {
#pragma unroll
    for (int c = 0; c < kJ; ++c)
      *reinterpret_cast<float4*>(&S.Q[r0 + r][4 * kg + 64 * c]) = O[r][c];
    if (kg == 0) {
      S.m[r0 + r] = m[r];
      S.l[r0 + r] = l[r];
    }
  }
  cluster.sync();
  if (tid < rows) {
    float M = -INFINITY, sum = 0.f;
    for (int c = 0; c < C; ++c) M = fmaxf(M, *cluster.map_shared_rank(&S.m[tid], c));
    for (int c = 0; c < C; ++c) {
      const float mc = *cluster.map_shared_rank(&S.m[tid], c);
      const float f = mc == -INFINITY ? 0.f : expf(mc - M);
      sum = fmaf(f, *cluster.map_shared_rank(&S.l[tid], c), sum);
      S.w[tid][c] = f;
    }
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    for (int c = 0; c < C; ++c) S.w[tid][c] *= inv;
    if (lse && rank == 0) lse[out_row(tid)] = M + logf(sum);
  }
  __syncthreads();
  for (int e = rank * kThreads + tid; e < rows * kChunks; e += C * kThreads) {
    const int r = e / kChunks, x = 4 * (e % kChunks);
    if (x >= d.D) continue;
    float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int c = 0; c < C; ++c)  // (a CTA that saw nothing has weight 0 and sums of 0)
      fma4(y, S.w[r][c], *reinterpret_cast<const float4*>(cluster.map_shared_rank(&S.Q[r][x], c)));
    *reinterpret_cast<float4*>(o + out_row(r) * d.D + x) = y;
  }
  cluster.sync();  // no CTA leaves while another reads its shared memory
}

template <int DP>
cudaError_t launch_dp(const AttendArgs& a, cudaStream_t stream) {
  using L = Shared<DP>;
  const gdn_tree_attend_dims& d = a.d;
  // (N = 0: one, that reports the sequences with rows all the same)
  const int tiles = d.N > 0 ? (int)(((long long)d.N * (d.Hq / d.Hkv) + kM - 1) / kM) : 1;
  const long long units = (long long)d.B * d.Hkv * tiles;
  const size_t bytes = sizeof(L) + (a.parent ? sizeof(int32_t) * (size_t)d.N : 0);
  cudaError_t err = cudaFuncSetAttribute(attend_f32_kernel<DP>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         (int)(sizeof(L) + sizeof(int32_t) * kMaxNLong));
  if (err != cudaSuccess) return err;
  // more CTAs a unit up to two an SM, as long as each has a tile of keys.  Measured, up to two
  // an SM, up to one with two tiles each, and no clusters: the 3 small trees 13.1, 15.5 and
  // 34.8 us, one row over 277 keys 10.4, 13.8, 33.7; 8 trees of 64 nodes (128 units, 832 keys)
  // 79.5, 103, 103.
  const long long sms = sm_count() > 0 ? sm_count() : 152;
  const long long keys = (long long)d.table_width * d.page_size + d.N + d.prefix_len;
  int C = 1;
  while (C < kMaxCluster && units * C <= sms && keys > C * L::kN) C *= 2;
  if (units * C > 0x7fffffffll) return cudaErrorInvalidConfiguration;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(units * C));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = bytes;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)C;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  typedef const float* fp;
  err = cudaLaunchKernelEx(&cfg, attend_f32_kernel<DP>, static_cast<fp>(a.q), static_cast<fp>(a.k),
                           static_cast<fp>(a.v), a.parent, a.cu, static_cast<fp>(a.k_cache),
                           static_cast<fp>(a.v_cache), a.page_table, a.context_len,
                           a.prefix_pages, a.scale, static_cast<float*>(a.o), a.lse, d, tiles,
                           a.dev_status);
  return err != cudaSuccess ? err : cudaGetLastError();
}

}  // namespace

cudaError_t launch_attend_f32(const AttendArgs& a, cudaStream_t stream) {
  return a.d.D <= 64 ? launch_dp<64>(a, stream) : launch_dp<128>(a, stream);
}

}  // namespace gdn
