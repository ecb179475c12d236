// rule_recurrent.cu -- the gated delta rule token by token: prefill of any shape and
// type, and the decoding step of one token.
//
//     S <- alpha (I - beta k k^T) S + beta k v^T,   o = S^T q
// Columns of S do not mix, so the split over dv needs no exchange.  With s = S^T k and
// r = S^T q taken from the state before the token,
//     u = beta (v - alpha s),   S <- alpha S + k u^T,   o = alpha r + (q.k) u,
// so a token costs one reduction over dk (s and r together; q.k does not depend on S).
// All arithmetic is fp32; nothing is rounded below it but o in its own type.
#include <type_traits>

#include "common.cuh"
#include "kernels.h"

namespace gdn {
namespace {

__device__ __forceinline__ void cp_async16(void* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(
                   (uint32_t)__cvta_generic_to_shared(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async4(void* dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(
                   (uint32_t)__cvta_generic_to_shared(dst)), "l"(src) : "memory");
}

// four consecutive elements as fp32, in pairs
__device__ __forceinline__ void load4(const float* p, float2& a, float2& b) {
  const float4 x = *reinterpret_cast<const float4*>(p);
  a = make_float2(x.x, x.y);
  b = make_float2(x.z, x.w);
}
__device__ __forceinline__ void load4(const __nv_bfloat16* p, float2& a, float2& b) {
  const uint2 x = *reinterpret_cast<const uint2*>(p);
  a = make_float2(__uint_as_float(x.x << 16), __uint_as_float(x.x & 0xffff0000u));
  b = make_float2(__uint_as_float(x.y << 16), __uint_as_float(x.y & 0xffff0000u));
}

// ---- many tokens: eight columns a warp ----------------------------------------------------
// Bound by the chain from a token's state to the next one's (products, a reduction, u, the
// update) or, with heads enough for every SM, by its instructions.  A column's dk rows are
// spread over 8 lanes of one warp (lane = 4 * row group + pair of columns) and reduced by three
// shuffles, with no barrier between tokens.  Tokens come 16 at a time, copied (cp.async) while
// the 16 before are computed.  Row 32 i + 4 (row group) + e: a warp's reads of k and q are
// consecutive.  (Two columns a lane: with one, reading k and q takes as long as the chain.)
// 0.21 us a token (fp32, 128 x 128 states, 4 heads); 16 sequences of 500 tokens with 32 heads
// take 0.99 ms, 20 TFLOP/s.  One barrier a token and 32 columns over a CTA took twice as long;
// two tokens a turn, with one round of shuffles for both, 0.26 us a token and 1.14 ms.
constexpr int kStage = 16;

template <typename T, int kI, int kWarps>  // dk <= 32 kI
__global__ void __launch_bounds__(32 * kWarps)
rule_scan_kernel(const T* __restrict__ q, const T* __restrict__ k, const T* __restrict__ v,
                 const float* __restrict__ log_alpha, const float* __restrict__ beta,
                 const float* pool_in, float* pool_out, T* __restrict__ o, gdn_tree_dims d,
                 SeqLayout lay, int32_t* dev_status) {
  constexpr int kD = 32 * kI, kCols = 8 * kWarps, kThreads = 32 * kWarps, kPer = 16 / sizeof(T);
  __shared__ __align__(16) T sK[2][kStage][kD], sQ[2][kStage][kD], sV[2][kStage][kCols];
  __shared__ float sA[2][kStage], sB[2][kStage];
  const int tiles = (d.dv + kCols - 1) / kCols;
  const int tile = blockIdx.x % tiles;
  const int h = (blockIdx.x / tiles) % d.Hv;
  const int b = blockIdx.x / tiles / d.Hv;
  const int tid = threadIdx.x, lane = tid & 31, rg = lane >> 2;
  const int own = 8 * (tid >> 5) + 2 * (lane & 3);  // the lane's columns of the tile
  const int col0 = tile * kCols, col = col0 + own;
  const int hq = h / (d.Hv / d.Hqk);

  const int n = lay.count(b, d.N), st = lay.state(b);
  if (n < 0 || st < 0) {
    if (dev_status && tid == 0) atomicMax(dev_status + b, GDN_TREE_STATUS_BAD_LAYOUT);
    return;
  }
  const size_t row = (size_t)lay.row0(b, d.N);
  const size_t soff = ((size_t)st * d.Hv + h) * d.dk * d.dv;
  const bool mine = col < d.dv;

  const T* kb = k + (row * d.Hqk + hq) * d.dk;
  const T* qb = q + (row * d.Hqk + hq) * d.dk;
  const T* vb = v + (row * d.Hv + h) * d.dv + col0;
  const float* ab = log_alpha + row * d.Hv + h;
  const float* bb = beta + row * d.Hv + h;
  const size_t qstride = (size_t)d.Hqk * d.dk, vstride = (size_t)d.Hv * d.dv;
  auto fetch = [&](int t0, int s) {
    constexpr int kRowChunks = kD / kPer, kVChunks = kCols / kPer;
#pragma unroll
    for (int e = 0; e < kStage * kRowChunks; e += kThreads) {
      const int t = (e + tid) / kRowChunks, c = kPer * ((e + tid) % kRowChunks);
      if (t < kStage && t0 + t < n && c < d.dk) {
        const size_t at = (t0 + t) * qstride + c;
        cp_async16(&sK[s][t][c], kb + at);
        cp_async16(&sQ[s][t][c], qb + at);
      }
    }
#pragma unroll
    for (int e = 0; e < kStage * kVChunks; e += kThreads) {
      const int t = (e + tid) / kVChunks, c = kPer * ((e + tid) % kVChunks);
      if (t < kStage && t0 + t < n && col0 + c < d.dv)
        cp_async16(&sV[s][t][c], vb + (t0 + t) * vstride + c);
    }
    if (tid < kStage && t0 + tid < n) {
      cp_async4(&sA[s][tid], ab + (size_t)(t0 + tid) * d.Hv);
      cp_async4(&sB[s][tid], bb + (size_t)(t0 + tid) * d.Hv);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };

  if (n > 0) fetch(0, 0);
  // rows past dk are zero
  for (int e = tid; e < 2 * kStage * kD; e += kThreads) {
    const int c = e % kD, t = e / kD;
    if (c >= d.dk) {
      sK[0][0][t * kD + c] = from_f32<T>(0.f);
      sQ[0][0][t * kD + c] = from_f32<T>(0.f);
    }
  }
  float2 S[2][2 * kI];  // two columns; pairs of rows
#pragma unroll
  for (int i = 0; i < kI; ++i) {
    float2 x[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int r = 32 * i + 4 * rg + e;
      x[e] = make_float2(0.f, 0.f);
      if (mine && r < d.dk)
        x[e] = *reinterpret_cast<const float2*>(pool_in + soff + (size_t)r * d.dv + col);
    }
    S[0][2 * i] = make_float2(x[0].x, x[1].x);
    S[0][2 * i + 1] = make_float2(x[2].x, x[3].x);
    S[1][2 * i] = make_float2(x[0].y, x[1].y);
    S[1][2 * i + 1] = make_float2(x[2].y, x[3].y);
  }
  auto dot = [&](const float2(&x)[2 * kI], const float2(&y)[2 * kI]) {
    float2 s0 = make_float2(0.f, 0.f), s1 = s0;
#pragma unroll
    for (int i = 0; i < 2 * kI; i += 2) {
      fma2(s0, x[i], y[i]);
      fma2(s1, x[i + 1], y[i + 1]);
    }
    return (s0.x + s0.y) + (s1.x + s1.y);
  };
  auto load_row = [&](const T* from, float2(&x)[2 * kI]) {
#pragma unroll
    for (int i = 0; i < kI; ++i) load4(from + 32 * i + 4 * rg, x[2 * i], x[2 * i + 1]);
  };

  T* ot = o + (row * d.Hv + h) * d.dv + col;
  for (int t0 = 0; t0 < n; t0 += kStage) {
    const int nt = min(kStage, n - t0), s = (t0 / kStage) & 1;
    asm volatile("cp.async.wait_all;" ::: "memory");
    __syncthreads();  // the stage is there, and the one before has been used
    if (t0 + kStage < n) fetch(t0 + kStage, s ^ 1);
    // the next token's k, gates and v are read while this one's sums are added up
    float2 kk[2 * kI], kn[2 * kI];
    float a, bt, an, bn, vt[2], vn[2];
    load_row(sK[s][0], kk);
    a = expf(sA[s][0]);
    bt = sB[s][0];
    vt[0] = to_f32(sV[s][0][own]);
    vt[1] = to_f32(sV[s][0][own + 1]);
#pragma unroll 2
    for (int t = 0; t < nt; ++t) {
      float2 qq[2 * kI];
      float x[2], r[2], u[2];
      load_row(sQ[s][t], qq);
      x[0] = dot(kk, S[0]);
      x[1] = dot(kk, S[1]);
      const int next = min(t + 1, nt - 1);
      load_row(sK[s][next], kn);
      an = expf(sA[s][next]);
      bn = sB[s][next];
      vn[0] = to_f32(sV[s][next][own]);
      vn[1] = to_f32(sV[s][next][own + 1]);
      r[0] = dot(qq, S[0]);
      r[1] = dot(qq, S[1]);
      float qk = dot(qq, kk);
#pragma unroll
      for (int off = 4; off < 32; off <<= 1) {
        x[0] += __shfl_xor_sync(0xffffffffu, x[0], off);
        x[1] += __shfl_xor_sync(0xffffffffu, x[1], off);
      }
      u[0] = bt * fmaf(-a, x[0], vt[0]);
      u[1] = bt * fmaf(-a, x[1], vt[1]);
#pragma unroll
      for (int c = 0; c < 2; ++c)
#pragma unroll
        for (int i = 0; i < 2 * kI; ++i) {
          mul2(S[c][i], a);
          fma2(S[c][i], kk[i], make_float2(u[c], u[c]));
        }
#pragma unroll
      for (int off = 4; off < 32; off <<= 1) {
        r[0] += __shfl_xor_sync(0xffffffffu, r[0], off);
        r[1] += __shfl_xor_sync(0xffffffffu, r[1], off);
        qk += __shfl_xor_sync(0xffffffffu, qk, off);
      }
      if (rg == 0 && mine) {
        ot[0] = from_f32<T>(fmaf(a, r[0], qk * u[0]));
        ot[1] = from_f32<T>(fmaf(a, r[1], qk * u[1]));
      }
      ot += vstride;
#pragma unroll
      for (int i = 0; i < 2 * kI; ++i) kk[i] = kn[i];
      a = an;
      bt = bn;
      vt[0] = vn[0];
      vt[1] = vn[1];
    }
  }
#pragma unroll
  for (int i = 0; i < kI; ++i) {
    const float2 x[4] = {make_float2(S[0][2 * i].x, S[1][2 * i].x),
                         make_float2(S[0][2 * i].y, S[1][2 * i].y),
                         make_float2(S[0][2 * i + 1].x, S[1][2 * i + 1].x),
                         make_float2(S[0][2 * i + 1].y, S[1][2 * i + 1].y)};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int r = 32 * i + 4 * rg + e;
      if (mine && r < d.dk)
        *reinterpret_cast<float2*>(pool_out + soff + (size_t)r * d.dv + col) = x[e];
    }
  }
}

// ---- one token: kCols columns of a state a CTA ---------------------------------------------
// Bound by DRAM: a 64 KB state is read and written whole, 16 bytes a thread with all of a
// thread's loads in flight.  Thread (rg, cl): float4 column chunk cl of the CTA's columns, rows
// rg, rg + kRG, ...; a warp's loads of one row cover kCols * 4 contiguous bytes.  256 sequences
// of 32 heads 162 us (6.7 TB/s, 98 % of a copy's rate), 64 41.9 us, 16 11.8 us, 1 3.1 us; a
// whole state a CTA by bulk copies took 167, 47.8, 17.2 us.
constexpr int kThreads = kMaxD;

template <typename T, int kCols>
__global__ void __launch_bounds__(kThreads)
rule_token_kernel(const T* __restrict__ q, const T* __restrict__ k, const T* __restrict__ v,
                  const float* __restrict__ log_alpha, const float* __restrict__ beta,
                  const float* pool_in, float* pool_out, T* __restrict__ o, gdn_tree_dims d,
                  SeqLayout lay, int32_t* dev_status) {
  constexpr int kCL = kCols / 4;          // float4 lanes a row
  constexpr int kRG = kThreads / kCL;     // row groups
  constexpr int kRows = kMaxD / kRG;      // rows a thread, at most
  constexpr int kWarps = kThreads / 32;
  static_assert(kMaxD % kRG == 0, "rows split evenly");
  const int tiles = (d.dv + kCols - 1) / kCols;
  const int tile = blockIdx.x % tiles;
  const int h = (blockIdx.x / tiles) % d.Hv;
  const int b = blockIdx.x / tiles / d.Hv;
  const int tid = threadIdx.x, warp = tid >> 5;
  const int cl = tid % kCL, rg = tid / kCL;
  const int col = tile * kCols + 4 * cl;
  const int hq = h / (d.Hv / d.Hqk);

  const int st = lay.state(b);
  if (st < 0) {
    if (dev_status && tid == 0) atomicMax(dev_status + b, GDN_TREE_STATUS_BAD_LAYOUT);
    return;
  }
  const size_t soff = ((size_t)st * d.Hv + h) * d.dk * d.dv;
  const size_t unit = (size_t)b * d.Hv + h;

  float4 S[kRows];
  const bool mine = col < d.dv;
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    const int r = rg + kRG * i;
    S[i] = make_float4(0.f, 0.f, 0.f, 0.f);
    if (mine && r < d.dk)
      S[i] = __ldcs(reinterpret_cast<const float4*>(pool_in + soff + (size_t)r * d.dv + col));
  }
  __shared__ float sK[kMaxD], sQ[kMaxD];
  if (tid < kMaxD) {
    const size_t at = ((size_t)b * d.Hqk + hq) * d.dk + tid;
    sK[tid] = tid < d.dk ? to_f32(k[at]) : 0.f;
    sQ[tid] = tid < d.dk ? to_f32(q[at]) : 0.f;
  }
  float vt[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) vt[e] = mine ? to_f32(v[unit * d.dv + col + e]) : 0.f;
  const float a = expf(log_alpha[unit]), bt = beta[unit];
  __syncthreads();

  __shared__ float red[kWarps][kCL][9];  // s (4), r (4), q.k of each warp
  float x[9] = {};
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    const float ki = sK[rg + kRG * i], qi = sQ[rg + kRG * i];
    x[0] = fmaf(ki, S[i].x, x[0]);
    x[1] = fmaf(ki, S[i].y, x[1]);
    x[2] = fmaf(ki, S[i].z, x[2]);
    x[3] = fmaf(ki, S[i].w, x[3]);
    x[4] = fmaf(qi, S[i].x, x[4]);
    x[5] = fmaf(qi, S[i].y, x[5]);
    x[6] = fmaf(qi, S[i].z, x[6]);
    x[7] = fmaf(qi, S[i].w, x[7]);
    x[8] = fmaf(qi, ki, x[8]);
  }
#pragma unroll
  for (int off = kCL; off < 32; off <<= 1)
#pragma unroll
    for (int e = 0; e < 9; ++e) x[e] += __shfl_xor_sync(0xffffffffu, x[e], off);
  if ((tid & 31) < kCL)
#pragma unroll
    for (int e = 0; e < 9; ++e) red[warp][cl][e] = x[e];
  __syncthreads();
#pragma unroll
  for (int e = 0; e < 9; ++e) {
    x[e] = red[0][cl][e];
#pragma unroll
    for (int w = 1; w < kWarps; ++w) x[e] += red[w][cl][e];
  }
  float u[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) u[e] = bt * (vt[e] - a * x[e]);
  if (!mine) return;
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    const int r = rg + kRG * i;
    const float ki = sK[r];
    if (r < d.dk)
      __stcs(reinterpret_cast<float4*>(pool_out + soff + (size_t)r * d.dv + col),
             make_float4(fmaf(ki, u[0], a * S[i].x), fmaf(ki, u[1], a * S[i].y),
                         fmaf(ki, u[2], a * S[i].z), fmaf(ki, u[3], a * S[i].w)));
  }
  if (rg == 0)
#pragma unroll
    for (int e = 0; e < 4; ++e)
      o[unit * d.dv + col + e] = from_f32<T>(fmaf(a, x[4 + e], x[8] * u[e]));
}

template <typename T>
cudaError_t launch_typed(const RuleArgs& a, bool step, cudaStream_t stream) {
  const gdn_tree_dims& d = a.d;
  auto go = [&](auto kernel, int cols, int threads) {
    const long long blocks = (long long)d.B * d.Hv * ((d.dv + cols - 1) / cols);
    if (blocks > 0x7fffffffll) return cudaErrorInvalidConfiguration;
    kernel<<<(unsigned)blocks, threads, 0, stream>>>(
        static_cast<const T*>(a.q), static_cast<const T*>(a.k), static_cast<const T*>(a.v),
        a.log_alpha, a.beta, a.pool_in, a.pool_out, static_cast<T*>(a.o), d, a.lay,
        a.dev_status);
    return cudaGetLastError();
  };
  // 32 columns (128-byte row pieces) unless dv would leave half of the last tile idle
  const bool wide = d.dv % 32 == 0;
  if (step)
    return wide ? go(rule_token_kernel<T, 32>, 32, kThreads)
                : go(rule_token_kernel<T, 16>, 16, kThreads);
  auto scan = [&](auto w) {
    constexpr int kWarps = decltype(w)::value;
    switch ((d.dk + 31) / 32) {
      case 1: return go(rule_scan_kernel<T, 1, kWarps>, 8 * kWarps, 32 * kWarps);
      case 2: return go(rule_scan_kernel<T, 2, kWarps>, 8 * kWarps, 32 * kWarps);
      case 3: return go(rule_scan_kernel<T, 3, kWarps>, 8 * kWarps, 32 * kWarps);
      default: return go(rule_scan_kernel<T, 4, kWarps>, 8 * kWarps, 32 * kWarps);
    }
  };
  return wide ? scan(std::integral_constant<int, 4>{}) : scan(std::integral_constant<int, 2>{});
}

cudaError_t launch_recurrent(const RuleArgs& a, bool step, cudaStream_t stream) {
  return a.d.dtype == GDN_TREE_BF16 ? launch_typed<__nv_bfloat16>(a, step, stream)
                                    : launch_typed<float>(a, step, stream);
}

}  // namespace

// The chunked kernels from kChunkedFrom tokens of the longest sequence on.  Below it their two
// launches and a whole chunk's work cost more than the tokens one by one.  Measured with 32
// heads, chunked and one by one, in us: 1 sequence of 16 tokens 13 and 7.8, of 32 13 and 12.1,
// of 64 13.1 and 20.5; 4 sequences of 32 27 and 26, of 48 27 and 37; 16 sequences of 16 78
// and 45, of 32 78 and 80, of 48 79 and 117.
constexpr int kChunkedFrom = 33;
static bool chunked(const gdn_tree_dims& d, int32_t T) {
  return d.N >= kChunkedFrom && T > 0 && prefill_tc_supported(d);
}

size_t prefill_workspace_bytes(const gdn_tree_dims& d, int32_t T) {
  return chunked(d, T) ? prefill_tc_workspace_bytes(d, T) : 0;
}

cudaError_t launch_prefill(const RuleArgs& a, void* workspace, cudaStream_t stream) {
  return chunked(a.d, a.lay.T) ? launch_prefill_tc(a, workspace, stream)
                               : launch_recurrent(a, false, stream);
}

cudaError_t launch_decode_step(const RuleArgs& a, cudaStream_t stream) {
  return launch_recurrent(a, true, stream);
}

}  // namespace gdn
