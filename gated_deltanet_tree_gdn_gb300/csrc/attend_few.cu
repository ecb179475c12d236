// attend_few.cu -- attention over a paged cache for sequences of at most 16 query rows
// (row = node * G + g of one key head): a token of each sequence, small trees.  bf16.
//
// Bound by the cache's bytes (each key and value is used by 16 rows at most), or by
// latency where there are few of them; so the work is spread over many warps with many
// loads in flight, and the tensor cores (m16n8k16, whose 16 rows are the tile) only keep
// the arithmetic out of the way.  A cluster of C CTAs of four warps takes one sequence and
// key head; every warp runs over 16 keys at a time with its own running maximum and sum,
//     S = Q K^T,  P = exp2(c S - m),  l += sum P,  O += P V,
// and the warps' results -- and those of the shared prefix, where it has units of its
// own -- are added up at the end through the cluster's shared memory:
//     M = max_w m_w,  L = sum_w l_w e^{m_w - M},  o = sum_w O_w e^{m_w - M} / L.
//
// Each warp keeps kStages - 1 tiles of 16 keys and values in flight to a ring of its own in
// shared memory (16-byte cp.async, rows past a length filled with zeros; the page numbers a
// tile further ahead): 128 KB an SM.  Loads to registers, two tiles of them, got 2.9 TB/s.
// From there 16-byte loads give the operands, because the order of a product's inner index
// is free, and so is which column an accumulator stands for:
//  - Q K^T: the lane that holds inner indices {2c, 2c+1, 2c+8, 2c+9} of two MMAs reads
//    elements 32 i + 8 c .. + 7 of its key (and of its query row);
//  - P V: a lane reads 8 consecutive columns of 4 keys, and pairs the keys by byte picks;
//    MMA e of 8 then takes column 8 n + e as its column n.
#include <cooperative_groups.h>

#include "common.cuh"
#include "kernels.h"

namespace cg = cooperative_groups;

namespace gdn {
namespace {

constexpr int kRows = kAttendFewRows;
constexpr int kWarps = 4, kThreads = 32 * kWarps;
constexpr int kMaxCluster = 16;  // (over 8: not portable, asked for at the launch)
constexpr int kPerSm = 3;
constexpr int kStages = 2;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

__device__ __forceinline__ void mma_16816(float (&d)[4], uint4 a, uint32_t b0,
                                          uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint4 load16(const __nv_bfloat16* p, bool take) {
  return take ? __ldg(reinterpret_cast<const uint4*>(p)) : make_uint4(0, 0, 0, 0);
}

__device__ __forceinline__ void cp_async16_zfill(void* dst, const void* src, bool take) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(
                   (uint32_t)__cvta_generic_to_shared(dst)),
               "l"(src), "r"(take ? 16u : 0u)
               : "memory");
}

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ bool nonfinite2(uint32_t x) {
  return (x & 0x7f80u) == 0x7f80u || (x & 0x7f800000u) == 0x7f800000u;
}
__device__ __forceinline__ uint32_t finite2(uint32_t x) {
  if ((x & 0x7f80u) == 0x7f80u) x &= 0xffff0000u;
  if ((x & 0x7f800000u) == 0x7f800000u) x &= 0x0000ffffu;
  return x;
}

// The prefix's units run before this kernel, which may start beside their last ones: from
// here on their parts are there.  (Every CTA comes here, so that this kernel never ends
// before theirs.)
__device__ __forceinline__ void prefix_done() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// Where the 16 bytes `chunk` of a row of a K or V tile are: eight lanes that read at once, a
// quarter of two rows (K) or two chunks of every other row (V), then find them in all banks.
__device__ __forceinline__ int place(int row, int chunk) {
  return 8 * (chunk ^ ((row & 6) ^ ((row & 1) << 2)));
}

template <int DP>
struct Shared {
  union {
    __nv_bfloat16 ring[kWarps][kStages][2][16][DP];  // K and V tiles (`place`)
    struct {  // then
      float O[kWarps][kRows][DP + 4];    // the warps' sums; [0] then holds the CTA's
      float wp[kRows][kAttendMaxParts];  // weight of each part of the prefix in the result
    };
  };
  uint4 q[DP / 32][2][32];         // Q as the MMAs take it: a lane's 16 bytes each
  float m[kWarps][kRows], l[kWarps][kRows];
  float cm[kRows], cl[kRows];      // the CTA's maximum and sum
  float w[kRows][kMaxCluster];     // weight of each CTA's sums in the result
  float scale[kRows];              // 1 / L
  uint32_t bad;                    // own nodes whose values hold infinities or NaN
  int32_t parent[kRows];
};

template <int DP>
__global__ void __launch_bounds__(kThreads, kPerSm)
attend_few_kernel(const __nv_bfloat16* __restrict__ q, const __nv_bfloat16* __restrict__ k,
                  const __nv_bfloat16* __restrict__ v, const int32_t* __restrict__ parent,
                  const int32_t* __restrict__ cu, const __nv_bfloat16* __restrict__ k_cache,
                  const __nv_bfloat16* __restrict__ v_cache, const int32_t* __restrict__ table,
                  const int32_t* __restrict__ context_len,
                  const int32_t* __restrict__ prefix_pages, float scale,
                  __nv_bfloat16* __restrict__ o, float* __restrict__ lse, gdn_tree_attend_dims d,
                  int plen, const float* __restrict__ part_o, const float* __restrict__ part_lse,
                  int parts, int32_t* dev_status) {
  extern __shared__ __align__(16) unsigned char smem_raw[];
  Shared<DP>& S = *reinterpret_cast<Shared<DP>*>(smem_raw);
  cg::cluster_group cluster = cg::this_cluster();
  const int C = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  const int unit = blockIdx.x / C;
  const int hk = unit % d.Hkv, b = unit / d.Hkv;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int c = lane & 3, r8 = lane >> 2;  // inner quarter, row (and key, and column block)
  const int G = d.Hq / d.Hkv;

  const int first = cu[b], stop = cu[b + 1], n = stop - first, ctx = context_len[b];
  const long long cap = (long long)d.table_width * d.page_size;
  // (stop < first, not n < 0: of two numbers far apart the difference may wrap)
  if (first < 0 || stop < first || stop > d.T || n > d.N || ctx < 0 || ctx > cap) {
    if (dev_status && tid == 0) atomicMax(dev_status + b, GDN_TREE_STATUS_BAD_LAYOUT);
    prefix_done();
    return;  // (every CTA of the cluster)
  }
  const int rows = n * G;
  if (rows == 0 || rows > kRows) {
    prefix_done();
    return;
  }
  const bool own = k != nullptr, tree = own && parent != nullptr;
  if (tid < n) {
    const int p = tree ? parent[first + tid] : tid - 1;
    const bool bad = p < -1 || p >= tid;
    S.parent[tid] = bad ? -1 : p;
    if (bad && dev_status) atomicMax(dev_status + b, GDN_TREE_STATUS_BAD_TREE);
  }
  if (tid == 0) S.bad = 0u;

  // ---- Q of rows r8 and r8 + 8 of each lane, in the MMAs' order -------------------------
  constexpr int kI = DP / 32;
  for (int i = warp; i < kI; i += kWarps) {
    uint4 x[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int row = r8 + 8 * e;
      const bool take = row < rows && 32 * i + 8 * c < d.D;
      const int node = take ? row / G : 0, g = take ? row - node * G : 0;
      x[e] = load16(q + ((size_t)(first + node) * d.Hq + hk * G + g) * d.D + 32 * i + 8 * c, take);
    }
    S.q[i][0][lane] = make_uint4(x[0].x, x[1].x, x[0].y, x[1].y);
    S.q[i][1][lane] = make_uint4(x[0].z, x[1].z, x[0].w, x[1].w);
  }
  __syncthreads();
  // the own nodes that rows r8 and r8 + 8 see, a bit a node
  uint32_t sees[2] = {0u, 0u};
#pragma unroll
  for (int e = 0; e < 2; ++e)
    if (own && r8 + 8 * e < rows)
      for (int a = (r8 + 8 * e) / G; a >= 0; a = S.parent[a]) sees[e] |= 1u << a;
  __syncwarp();

  // ---- the keys, 16 at a time -------------------------------------------------------------
  const int nP = (plen + 15) >> 4, nC = (ctx + 15) >> 4, all = nP + nC + (own ? 1 : 0);
  const float cs = scale * kLog2e;
  const size_t stride = (size_t)d.Hkv * d.D;
  // lanes 0 .. 15: the row of key `lane` of tile t in its array, -1 where there is none
  auto rows_of = [&](int t) -> int {
    if (t >= all || lane >= 16) return -1;
    const bool pre = t < nP, mine = t >= nP + nC;
    const int j = 16 * (pre ? t : mine ? 0 : t - nP) + lane;
    if (j >= (pre ? plen : mine ? n : ctx)) return -1;
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
  // a warp's copy instruction covers kAtOnce rows of a tile
  constexpr int kChunks = DP / 8, kAtOnce = 32 / kChunks;
  const int ch = lane % kChunks, sub = lane / kChunks;
  auto fetch = [&](int t, int row, int stage) {
    if (t < all) {
      const bool mine = t >= nP + nC;
      const size_t col = (size_t)hk * d.D + 8 * ch;
      const __nv_bfloat16 *kb = (mine ? k : k_cache) + col, *vb = (mine ? v : v_cache) + col;
#pragma unroll
      for (int i = 0; i < 16; i += kAtOnce) {
        const int x = __shfl_sync(0xffffffffu, row, i + sub);
        const bool take = x >= 0 && 8 * ch < d.D;
        const size_t off = take ? x * stride : 0;
        cp_async16_zfill(&S.ring[warp][stage][0][i + sub][place(i + sub, ch)], take ? kb + off : kb, take);
        cp_async16_zfill(&S.ring[warp][stage][1][i + sub][place(i + sub, ch)], take ? vb + off : vb, take);
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };

  float O[DP / 64][8][4];
#pragma unroll
  for (int h = 0; h < DP / 64; ++h)
#pragma unroll
    for (int e = 0; e < 8; ++e)
#pragma unroll
      for (int i = 0; i < 4; ++i) O[h][e][i] = 0.f;
  float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
  const int step = kWarps * C;
  const int t0 = rank * kWarps + warp;
  // rows of the tiles in flight (bit masks of the keys there are), and of the next to fetch
  uint32_t there_of[kStages];
  int next_row = rows_of(t0);
#pragma unroll
  for (int s = 0; s < kStages - 1; ++s) {
    const int row = next_row;
    next_row = rows_of(t0 + (s + 1) * step);
    there_of[s] = __ballot_sync(0xffffffffu, row >= 0);
    fetch(t0 + s * step, row, s);
  }
  int stage = 0;
  for (int t = t0; t < all; t += step) {
    const bool mine = t >= nP + nC;
    asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 2) : "memory");
    __syncwarp();
    const uint32_t there = there_of[0];
    {  // the stage that the last tile was read from takes the next one
      const int ahead = t + (kStages - 1) * step, row = next_row;
      next_row = rows_of(ahead + step);
#pragma unroll
      for (int s = 0; s + 2 < kStages; ++s) there_of[s] = there_of[s + 1];
      there_of[kStages - 2] = __ballot_sync(0xffffffffu, row >= 0);
      fetch(ahead, row, stage == 0 ? kStages - 1 : stage - 1);
    }
    const __nv_bfloat16(*kt)[DP] = S.ring[warp][stage][0];
    const __nv_bfloat16(*vt)[DP] = S.ring[warp][stage][1];
    stage = stage == kStages - 1 ? 0 : stage + 1;
    float s[2][4] = {};
#pragma unroll
    for (int i = 0; i < kI; ++i) {
      const uint4 q0 = S.q[i][0][lane], q1 = S.q[i][1][lane];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const uint4 x = *reinterpret_cast<const uint4*>(&kt[r8 + 8 * e][place(r8, 4 * i + c)]);
        mma_16816(s[e], q0, x.x, x.y);
        mma_16816(s[e], q1, x.z, x.w);
      }
    }
    // s[e][..]: rows r8 (0, 1) and r8 + 8 (2, 3), keys 8 e + 2 c + {0, 1}
    float top[2] = {-INFINITY, -INFINITY};
#pragma unroll
    for (int e = 0; e < 2; ++e)
#pragma unroll
      for (int i = 0; i < 4; ++i) s[e][i] *= cs;
    if (mine || there != 0xffffu) {
#pragma unroll
      for (int e = 0; e < 2; ++e)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int key = 8 * e + 2 * c + (i & 1);
          const bool on = ((mine ? there & sees[i >> 1] : there) >> key) & 1u;
          if (!on) s[e][i] = -INFINITY;
        }
    }
#pragma unroll
    for (int e = 0; e < 2; ++e)
#pragma unroll
      for (int i = 0; i < 4; ++i) top[i >> 1] = fmaxf(top[i >> 1], s[e][i]);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      top[i] = fmaxf(top[i], __shfl_xor_sync(0xffffffffu, top[i], 1));
      top[i] = fmaxf(top[i], __shfl_xor_sync(0xffffffffu, top[i], 2));
      top[i] = fmaxf(top[i], m[i]);
    }
    if (__any_sync(0xffffffffu, top[0] > m[0] || top[1] > m[1])) {
      float keep[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        keep[i] = m[i] == -INFINITY ? 0.f : ex2(m[i] - top[i]);
        m[i] = top[i];
        l[i] *= keep[i];
      }
#pragma unroll
      for (int h = 0; h < DP / 64; ++h)
#pragma unroll
        for (int e = 0; e < 8; ++e)
#pragma unroll
          for (int i = 0; i < 4; ++i) O[h][e][i] *= keep[i >> 1];
    }
#pragma unroll
    for (int e = 0; e < 2; ++e)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        s[e][i] = ex2(s[e][i] - (m[i >> 1] == -INFINITY ? 0.f : m[i >> 1]));
        l[i >> 1] += s[e][i];  // (this lane's keys; the four lanes of a row add up at the end)
      }
    // P as the A operand: its inner index is the key.  (bf16 as V is, at most 2^-8 of a weight;
    // l above is the fp32 weights')
    const uint4 pa = make_uint4(pack_bf16(s[0][0], s[0][1]), pack_bf16(s[0][2], s[0][3]),
                                pack_bf16(s[1][0], s[1][1]), pack_bf16(s[1][2], s[1][3]));
#pragma unroll
    for (int h = 0; h < DP / 64; ++h) {
      uint4 x[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int key = 2 * c + (e & 1) + 8 * (e >> 1);
        x[e] = *reinterpret_cast<const uint4*>(&vt[key][place(key, 8 * h + r8)]);
        // own nodes are masked for some rows only: what is not finite is kept out of the
        // product (0 * inf) and added to the rows that see it at the end
        if (mine && n > 1 &&
            (nonfinite2(x[e].x) || nonfinite2(x[e].y) || nonfinite2(x[e].z) || nonfinite2(x[e].w))) {
          atomicOr(&S.bad, 1u << key);
          x[e] = make_uint4(finite2(x[e].x), finite2(x[e].y), finite2(x[e].z), finite2(x[e].w));
        }
      }
      __syncwarp();
      const uint32_t w[4][4] = {{x[0].x, x[0].y, x[0].z, x[0].w}, {x[1].x, x[1].y, x[1].z, x[1].w},
                                {x[2].x, x[2].y, x[2].z, x[2].w}, {x[3].x, x[3].y, x[3].z, x[3].w}};
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const uint32_t pick = (e & 1) ? 0x7632u : 0x5410u;  // high or low halves
        mma_16816(O[h][e], pa, __byte_perm(w[0][e >> 1], w[1][e >> 1], pick),
                  __byte_perm(w[2][e >> 1], w[3][e >> 1], pick));
      }
    }
    __syncwarp();  // the tile has been read: its stage may be filled again
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
  __syncthreads();  // every ring is done with: the sums take its place

  // ---- the warp's results to shared memory, the CTA's from them ---------------------------
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    l[i] += __shfl_xor_sync(0xffffffffu, l[i], 1);
    l[i] += __shfl_xor_sync(0xffffffffu, l[i], 2);
    if (c == 0) {
      S.m[warp][r8 + 8 * i] = m[i];
      S.l[warp][r8 + 8 * i] = l[i];
    }
    // this lane's columns: 64 h + 16 c + e (accumulator 0 / 2) and + 8 (1 / 3)
#pragma unroll
    for (int h = 0; h < DP / 64; ++h)
#pragma unroll
      for (int x = 0; x < 2; ++x)
#pragma unroll
        for (int e = 0; e < 8; e += 4)
          *reinterpret_cast<float4*>(&S.O[warp][r8 + 8 * i][64 * h + 16 * c + 8 * x + e]) =
              make_float4(O[h][e][2 * i + x], O[h][e + 1][2 * i + x], O[h][e + 2][2 * i + x],
                          O[h][e + 3][2 * i + x]);
  }
  __syncthreads();
  constexpr int kVec = DP / 4;
  for (int e = tid; e < kRows * kVec; e += kThreads) {
    const int r = e / kVec, x = 4 * (e % kVec);
    float M = -INFINITY;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) M = fmaxf(M, S.m[w][r]);
    float L = 0.f;
    float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float f = S.m[w][r] == -INFINITY ? 0.f : ex2(S.m[w][r] - M);
      const float4 z = *reinterpret_cast<const float4*>(&S.O[w][r][x]);
      L = fmaf(f, S.l[w][r], L);
      y.x = fmaf(f, z.x, y.x);
      y.y = fmaf(f, z.y, y.y);
      y.z = fmaf(f, z.z, y.z);
      y.w = fmaf(f, z.w, y.w);
    }
    // (S.O[0][r][x ..] is read by this thread alone)
    *reinterpret_cast<float4*>(&S.O[0][r][x]) = y;
    if (x == 0) {
      S.cm[r] = M;
      S.cl[r] = L;
    }
  }
  if (C > 1) cluster.sync();
  else __syncthreads();

  prefix_done();

  // ---- the rows' weights: the cluster's CTAs and the prefix's parts -----------------------
  const size_t T = (size_t)d.T * d.Hq;
  auto out_row = [&](int r) {
    const int node = r / G;
    return (size_t)(first + node) * d.Hq + hk * G + (r - node * G);
  };
  for (int r = warp; r < rows; r += kWarps) {  // a warp a row, a lane a part
    const size_t at = out_row(r);
    constexpr int kPer = kAttendMaxParts / 32;
    float z[kPer + 1], M = -INFINITY;
    z[kPer] = lane < C ? *cluster.map_shared_rank(&S.cm[r], lane) : -INFINITY;
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      z[i] = lane + 32 * i < parts ? part_lse[(lane + 32 * i) * T + at] * kLog2e : -INFINITY;
#pragma unroll
    for (int i = 0; i <= kPer; ++i) M = fmaxf(M, z[i]);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, off));
    float L = 0.f;
#pragma unroll
    for (int i = 0; i <= kPer; ++i) {
      const float f = z[i] == -INFINITY ? 0.f : ex2(z[i] - M);
      if (i < kPer) {
        S.wp[r][lane + 32 * i] = f;
        L += f;
      } else if (lane < C) {
        S.w[r][lane] = f;
        L = fmaf(f, *cluster.map_shared_rank(&S.cl[r], lane), L);
      }
    }
    L = warp_sum(L);
    if (lane == 0) {
      S.scale[r] = L > 0.f ? 1.f / L : (L == 0.f ? 0.f : L);  // (NaN is kept)
      if (lse && rank == 0) lse[at] = L == 0.f ? -INFINITY : (M + log2f(L)) * kLn2;
    }
  }
  __syncthreads();
  for (int e = rank * kThreads + tid; e < rows * kVec; e += C * kThreads) {
    const int r = e / kVec, x = 4 * (e % kVec);
    if (x >= d.D) continue;
    const size_t at = out_row(r);
    const float f = S.scale[r];
    float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int w = 0; w < C; ++w) {
      const float4 z = *reinterpret_cast<const float4*>(cluster.map_shared_rank(&S.O[0][r][x], w));
      const float g = S.w[r][w];
      y.x = fmaf(g, z.x, y.x);
      y.y = fmaf(g, z.y, y.y);
      y.z = fmaf(g, z.z, y.z);
      y.w = fmaf(g, z.w, y.w);
    }
    // (a part that saw nothing has weight 0 and sums of 0)
#pragma unroll 8
    for (int p = 0; p < parts; ++p) {
      const float4 z = *reinterpret_cast<const float4*>(part_o + (p * T + at) * d.D + x);
      const float g = S.wp[r][p];
      y.x = fmaf(g, z.x, y.x);
      y.y = fmaf(g, z.y, y.y);
      y.z = fmaf(g, z.z, y.z);
      y.w = fmaf(g, z.w, y.w);
    }
    if (f == 0.f) y = make_float4(0.f, 0.f, 0.f, 0.f);
    else { y.x *= f; y.y *= f; y.z *= f; y.w *= f; }
    // the one CTA that holds the own nodes has their bits
    uint32_t bad = 0;
    if (own && n > 1)
      for (int w = 0; w < C; ++w) bad |= *cluster.map_shared_rank(&S.bad, w);
    if (bad) {
      for (int nd = r / G; nd >= 0; nd = S.parent[nd]) {
        if (!((bad >> nd) & 1u)) continue;
        const __nv_bfloat16* vr = v + ((size_t)(first + nd) * d.Hkv + hk) * d.D + x;
        float* ys = &y.x;
        for (int i = 0; i < 4; ++i) {
          const float z = __bfloat162float(vr[i]);
          if (!isfinite(z)) ys[i] += z;
        }
      }
    }
    *reinterpret_cast<uint2*>(o + at * d.D + x) = make_uint2(pack_bf16(y.x, y.y), pack_bf16(y.z, y.w));
  }
  if (C > 1) cluster.sync();  // no CTA leaves while another reads its shared memory
}

template <int DP>
cudaError_t launch_dp(const AttendArgs& a, int plen, const float* part_o, const float* part_lse,
                      int parts, int cluster, cudaStream_t stream) {
  const gdn_tree_attend_dims& d = a.d;
  auto kernel = attend_few_kernel<DP>;
  cudaError_t err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         (int)sizeof(Shared<DP>));
  if (err != cudaSuccess) return err;
  if (cluster > 8)
    err = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (err != cudaSuccess) return err;
  const long long blocks = (long long)d.B * d.Hkv * cluster;
  if (blocks > 0x7fffffffll) return cudaErrorInvalidConfiguration;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)blocks);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = sizeof(Shared<DP>);
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)cluster;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = parts > 0 ? 2 : 1;  // (beside the prefix's units, where there are any)
  typedef const __nv_bfloat16* bf;
  err = cudaLaunchKernelEx(&cfg, kernel, static_cast<bf>(a.q), static_cast<bf>(a.k),
                           static_cast<bf>(a.v), a.parent, a.cu, static_cast<bf>(a.k_cache),
                           static_cast<bf>(a.v_cache), a.page_table, a.context_len, a.prefix_pages,
                           a.scale, static_cast<__nv_bfloat16*>(a.o), a.lse, d, plen, part_o,
                           part_lse, parts, a.dev_status);
  return err != cudaSuccess ? err : cudaGetLastError();
}

}  // namespace

// How many CTAs take a sequence and key head, and about how long that takes in us.  The CTAs
// run in rounds of kPerSm an SM.  64 keys (32 KB of 128-wide heads) take a CTA 1.3, 1.5 or
// 2.4 us where 1, 2 or 3 of them share the SM, and its start and end about twice that.
// Measured with 8 key heads and one of 4096 keys a sequence, in us by CTAs a unit: 16
// sequences 1: 84, 2: 57, 4: 73, 8: 69; 32 sequences 97, 131, 113, 130; 64 sequences 234,
// 205, 192, 238; one sequence of 8192 keys 150, 84, 45, 26, and 21 with 16.
// That is for the longest contexts that the page table holds.  They are rarely all that long,
// and then the longest one is what is waited for; so more CTAs a unit are taken where they
// would cost no more than 1.3 times as much, in three rounds at most and with 8 times 64 keys
// each at least.  Measured with 256 to 8192 keys a sequence: 16 sequences 155, 91, 60, 51 us,
// 32 sequences 163, 99, 79, 90.
int attend_few_cluster(const gdn_tree_attend_dims& d, int prefix_len, float* us) {
  constexpr float kUs[kPerSm + 1] = {0.f, 1.3f, 1.5f, 2.4f}, kMore = 1.3f;
  const long long sms = sm_count() > 0 ? sm_count() : 152, slots = kPerSm * sms;
  const long long units = (long long)d.B * d.Hkv;
  const long long keys = (long long)d.table_width * d.page_size + d.N + prefix_len;
  float least = 0.f;
  int best = 1;
  for (int more = 0; more < 2; ++more)
    for (int C = 1; C <= kMaxCluster; C *= 2) {
      const long long full = units * C / slots, rest = units * C - full * slots;
      const long long rounds = (keys + 16 * kWarps * C - 1) / (16 * kWarps * C);
      const float t = (full * kUs[kPerSm] + kUs[(rest + sms - 1) / sms]) * (rounds + 2);
      const bool take = !more ? C == 1 || t < least
                              : C > best && t <= kMore * least && rounds >= 8 && units * C <= 3 * slots;
      if (!take) continue;
      best = C;
      *us = t;
      if (!more) least = t;
    }
  return best;
}

cudaError_t launch_attend_few(const AttendArgs& a, int prefix_len, const float* part_o,
                              const float* part_lse, int parts, cudaStream_t stream) {
  const gdn_tree_attend_dims& d = a.d;
  float us;
  const int cluster = attend_few_cluster(d, prefix_len, &us);
  return d.D <= 64 ? launch_dp<64>(a, prefix_len, part_o, part_lse, parts, cluster, stream)
                   : launch_dp<128>(a, prefix_len, part_o, part_lse, parts, cluster, stream);
}

}  // namespace gdn
