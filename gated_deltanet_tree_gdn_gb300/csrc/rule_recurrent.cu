// rule_recurrent.cu -- the gated delta rule token by token: prefill of any shape and
// type, and the decoding step of one token.
//
// One CTA holds kCols columns of one (sequence, v-head) state in registers and runs
//     S <- alpha (I - beta k k^T) S + beta k v^T,   o = S^T q
// over the sequence's tokens.  Columns of S do not mix, so the split over dv needs no
// exchange.  With s = S^T k and r = S^T q taken from the state before the token,
//     u = beta (v - alpha s),   S <- alpha S + k u^T,   o = alpha r + (q.k) u,
// so a token costs one reduction over dk (s, r and q.k together) and one barrier.
// All arithmetic is fp32; nothing is rounded below it but o in its own type.
//
// Thread (rg, cl): float4 column chunk cl of the CTA's columns, rows rg, rg + kRG, ...
// A warp's loads of one row cover kCols * 4 contiguous bytes.
#include "common.cuh"
#include "kernels.h"
#include "sm100.cuh"

namespace gdn {
namespace {

constexpr int kThreads = 128;
constexpr int kStage = 16;  // tokens staged in shared memory at a time

template <typename T, int kCols>
__global__ void __launch_bounds__(kThreads)
rule_recurrent_kernel(const T* __restrict__ q, const T* __restrict__ k, const T* __restrict__ v,
                      const float* __restrict__ log_alpha, const float* __restrict__ beta,
                      const float* pool_in, float* pool_out, T* __restrict__ o,
                      gdn_tree_dims d, SeqLayout lay, int32_t* dev_status) {
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

  const int n = lay.count(b, d.N), st = lay.state(b);
  if (n < 0 || st < 0) {
    if (dev_status && tid == 0) atomicMax(dev_status + b, GDN_TREE_STATUS_BAD_LAYOUT);
    return;
  }
  const size_t row = (size_t)lay.row0(b, d.N);
  const size_t soff = ((size_t)st * d.Hv + h) * d.dk * d.dv;

  float4 S[kRows];
  const bool mine = col < d.dv;
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    const int r = rg + kRG * i;
    S[i] = make_float4(0.f, 0.f, 0.f, 0.f);
    if (mine && r < d.dk)
      S[i] = __ldcs(reinterpret_cast<const float4*>(pool_in + soff + (size_t)r * d.dv + col));
  }

  __shared__ float sK[kStage][kMaxD], sQ[kStage][kMaxD], sV[kStage][kCols];
  __shared__ float sA[kStage], sB[kStage];
  __shared__ float sRed[2][kWarps][kCL][9];  // s (4), r (4), q.k of each warp

  for (int t0 = 0; t0 < n; t0 += kStage) {
    const int nt = min(kStage, n - t0);
    __syncthreads();  // the previous stage has been used
    for (int e = tid; e < nt * d.dk; e += kThreads) {
      const int t = e / d.dk, i = e - t * d.dk;
      const size_t at = ((row + t0 + t) * d.Hqk + hq) * d.dk + i;
      sK[t][i] = to_f32(k[at]);
      sQ[t][i] = to_f32(q[at]);
    }
    for (int e = tid; e < nt * kCols; e += kThreads) {
      const int t = e / kCols, i = e % kCols;
      sV[t][i] = tile * kCols + i < d.dv
                     ? to_f32(v[((row + t0 + t) * d.Hv + h) * d.dv + tile * kCols + i]) : 0.f;
    }
    if (tid < nt) {
      sA[tid] = expf(log_alpha[(row + t0 + tid) * d.Hv + h]);
      sB[tid] = beta[(row + t0 + tid) * d.Hv + h];
    }
    __syncthreads();
    for (int t = 0; t < nt; ++t) {
      float4 s = make_float4(0.f, 0.f, 0.f, 0.f), r = s;
      float qk = 0.f;
      float kk[kRows];
#pragma unroll
      for (int i = 0; i < kRows; ++i) {
        const int ri = rg + kRG * i;
        kk[i] = ri < d.dk ? sK[t][ri] : 0.f;
        const float qi = ri < d.dk ? sQ[t][ri] : 0.f;
        s.x = fmaf(kk[i], S[i].x, s.x);
        s.y = fmaf(kk[i], S[i].y, s.y);
        s.z = fmaf(kk[i], S[i].z, s.z);
        s.w = fmaf(kk[i], S[i].w, s.w);
        r.x = fmaf(qi, S[i].x, r.x);
        r.y = fmaf(qi, S[i].y, r.y);
        r.z = fmaf(qi, S[i].z, r.z);
        r.w = fmaf(qi, S[i].w, r.w);
        qk = fmaf(qi, kk[i], qk);
      }
#pragma unroll
      for (int off = kCL; off < 32; off <<= 1) {
        s.x += __shfl_xor_sync(0xffffffffu, s.x, off);
        s.y += __shfl_xor_sync(0xffffffffu, s.y, off);
        s.z += __shfl_xor_sync(0xffffffffu, s.z, off);
        s.w += __shfl_xor_sync(0xffffffffu, s.w, off);
        r.x += __shfl_xor_sync(0xffffffffu, r.x, off);
        r.y += __shfl_xor_sync(0xffffffffu, r.y, off);
        r.z += __shfl_xor_sync(0xffffffffu, r.z, off);
        r.w += __shfl_xor_sync(0xffffffffu, r.w, off);
        qk += __shfl_xor_sync(0xffffffffu, qk, off);
      }
      // (two buffers: a warp writes token t + 2's sums only after every warp passed the
      // barrier of token t + 1, behind its reads of token t)
      float(*red)[kCL][9] = sRed[t & 1];
      if ((tid & 31) < kCL) {
        float* w = red[warp][cl];
        w[0] = s.x; w[1] = s.y; w[2] = s.z; w[3] = s.w;
        w[4] = r.x; w[5] = r.y; w[6] = r.z; w[7] = r.w;
        w[8] = qk;
      }
      __syncthreads();
      float tot[9];
#pragma unroll
      for (int e = 0; e < 9; ++e) {
        tot[e] = red[0][cl][e];
#pragma unroll
        for (int w = 1; w < kWarps; ++w) tot[e] += red[w][cl][e];
      }
      const float a = sA[t], bt = sB[t];
      const float* vt = &sV[t][4 * cl];
      float4 u;
      u.x = bt * (vt[0] - a * tot[0]);
      u.y = bt * (vt[1] - a * tot[1]);
      u.z = bt * (vt[2] - a * tot[2]);
      u.w = bt * (vt[3] - a * tot[3]);
#pragma unroll
      for (int i = 0; i < kRows; ++i) {
        S[i].x = fmaf(kk[i], u.x, a * S[i].x);
        S[i].y = fmaf(kk[i], u.y, a * S[i].y);
        S[i].z = fmaf(kk[i], u.z, a * S[i].z);
        S[i].w = fmaf(kk[i], u.w, a * S[i].w);
      }
      if (rg == 0 && mine) {
        T* ot = o + ((row + t0 + t) * d.Hv + h) * d.dv + col;
        ot[0] = from_f32<T>(fmaf(a, tot[4], tot[8] * u.x));
        ot[1] = from_f32<T>(fmaf(a, tot[5], tot[8] * u.y));
        ot[2] = from_f32<T>(fmaf(a, tot[6], tot[8] * u.z));
        ot[3] = from_f32<T>(fmaf(a, tot[7], tot[8] * u.w));
      }
    }
  }
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    const int r = rg + kRG * i;
    if (mine && r < d.dk)
      __stcs(reinterpret_cast<float4*>(pool_out + soff + (size_t)r * d.dv + col), S[i]);
  }
}

// ---- one token of many sequences: a state a CTA, by bulk copies ----------------------------
// Bound by DRAM: a 64 KB state (dk rows of 128 columns) is read and written whole.  It comes
// and goes as one contiguous piece each way (cp.async.bulk), three CTAs an SM; four CTAs a
// state with 16-byte accesses of 128-byte row pieces reached 5.5 TB/s, and 5.0 TB/s with
// sixteen CTAs an SM.  Thread (rg, cl): rows 16 rg .., columns 4 cl .. + 3.
constexpr int kBulkThreads = 256;
constexpr int kBulkRows = kMaxD / (kBulkThreads / 32);  // rows a warp

struct BulkShared {
  float k[kMaxD], q[kMaxD], qk[kBulkThreads / 32];
  float4 s[kBulkThreads / 32][32], r[kBulkThreads / 32][32];  // each warp's S^T k and S^T q
  uint64_t bar;
};
constexpr uint32_t kBulkBytes = kMaxD * kMaxD * 4 + sizeof(BulkShared);

template <typename T>
__global__ void __launch_bounds__(kBulkThreads, 3)
rule_step_kernel(const T* __restrict__ q, const T* __restrict__ k, const T* __restrict__ v,
                 const float* __restrict__ log_alpha, const float* __restrict__ beta,
                 const float* pool_in, float* pool_out, T* __restrict__ o, gdn_tree_dims d,
                 SeqLayout lay, int32_t* dev_status, uint64_t limit_ns) {
  extern __shared__ __align__(128) unsigned char smem[];
  float4(*sS)[32] = reinterpret_cast<float4(*)[32]>(smem);  // [dk][128 columns]
  BulkShared& P = *reinterpret_cast<BulkShared*>(smem + kMaxD * kMaxD * 4);
  const int h = blockIdx.x % d.Hv, b = blockIdx.x / d.Hv;
  const int tid = threadIdx.x, rg = tid >> 5, cl = tid & 31;
  const int hq = h / (d.Hv / d.Hqk);
  const int st = lay.state(b);
  if (st < 0) {
    if (dev_status && tid == 0) atomicMax(dev_status + b, GDN_TREE_STATUS_BAD_LAYOUT);
    return;
  }
  const size_t soff = ((size_t)st * d.Hv + h) * d.dk * kMaxD;
  const uint32_t bytes = (uint32_t)d.dk * kMaxD * 4;
  if (tid == 0) {
    sm100::mbar_init(&P.bar, 1);
    sm100::mbar_fence_init();
    sm100::mbar_arrive_expect_tx(&P.bar, bytes);
    sm100::bulk_load(smem, pool_in + soff, bytes, &P.bar);
  }
  if (tid < d.dk) P.k[tid] = to_f32(k[((size_t)b * d.Hqk + hq) * d.dk + tid]);
  if (tid >= kMaxD && tid - kMaxD < d.dk)
    P.q[tid - kMaxD] = to_f32(q[((size_t)b * d.Hqk + hq) * d.dk + tid - kMaxD]);
  const size_t unit = (size_t)b * d.Hv + h;
  const float a = expf(log_alpha[unit]), bt = beta[unit];
  float vv[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) vv[e] = to_f32(v[unit * kMaxD + 4 * cl + e]);
  __syncthreads();
  const bool ok = sm100::mbar_wait(&P.bar, 0, limit_ns);
  float4 S[kBulkRows], s = make_float4(0.f, 0.f, 0.f, 0.f), r = s;
  float qk = 0.f;
#pragma unroll
  for (int i = 0; i < kBulkRows; ++i) {
    const int row = rg * kBulkRows + i;
    if (row < d.dk) {
      S[i] = sS[row][cl];
      const float ki = P.k[row], qi = P.q[row];
      s.x = fmaf(ki, S[i].x, s.x);
      s.y = fmaf(ki, S[i].y, s.y);
      s.z = fmaf(ki, S[i].z, s.z);
      s.w = fmaf(ki, S[i].w, s.w);
      r.x = fmaf(qi, S[i].x, r.x);
      r.y = fmaf(qi, S[i].y, r.y);
      r.z = fmaf(qi, S[i].z, r.z);
      r.w = fmaf(qi, S[i].w, r.w);
      qk = fmaf(qi, ki, qk);
    }
  }
  P.s[rg][cl] = s;
  P.r[rg][cl] = r;
  if (cl == 0) P.qk[rg] = qk;
  // (a timeout leaves the copy in flight: it is waited for once more before the CTA ends)
  if (__syncthreads_or(!ok)) {
    sm100::mbar_wait(&P.bar, 0, limit_ns);
    if (dev_status && tid == 0) atomicMax(dev_status + b, GDN_TREE_STATUS_TIMEOUT);
    return;
  }
  s = P.s[0][cl];
  r = P.r[0][cl];
  qk = P.qk[0];
#pragma unroll
  for (int w = 1; w < kBulkThreads / 32; ++w) {
    const float4 x = P.s[w][cl], y = P.r[w][cl];
    s.x += x.x; s.y += x.y; s.z += x.z; s.w += x.w;
    r.x += y.x; r.y += y.y; r.z += y.z; r.w += y.w;
    qk += P.qk[w];
  }
  const float4 u = make_float4(bt * (vv[0] - a * s.x), bt * (vv[1] - a * s.y),
                               bt * (vv[2] - a * s.z), bt * (vv[3] - a * s.w));
#pragma unroll
  for (int i = 0; i < kBulkRows; ++i) {
    const int row = rg * kBulkRows + i;
    if (row < d.dk) {
      const float ki = P.k[row];
      sS[row][cl] = make_float4(fmaf(ki, u.x, a * S[i].x), fmaf(ki, u.y, a * S[i].y),
                                fmaf(ki, u.z, a * S[i].z), fmaf(ki, u.w, a * S[i].w));
    }
  }
  sm100::fence_proxy_async_smem();
  if (rg == 0) {
    T* ot = o + unit * kMaxD + 4 * cl;
    ot[0] = from_f32<T>(fmaf(a, r.x, qk * u.x));
    ot[1] = from_f32<T>(fmaf(a, r.y, qk * u.y));
    ot[2] = from_f32<T>(fmaf(a, r.z, qk * u.z));
    ot[3] = from_f32<T>(fmaf(a, r.w, qk * u.w));
  }
  __syncthreads();
  if (tid == 0) {
    sm100::bulk_store(pool_out + soff, smem, bytes);
    sm100::bulk_commit_group();
    sm100::bulk_wait_all();
  }
}

template <typename T>
cudaError_t launch_step_bulk(const RuleArgs& a, cudaStream_t stream) {
  const gdn_tree_dims& d = a.d;
  auto kernel = rule_step_kernel<T>;
  cudaError_t err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         (int)kBulkBytes);
  if (err != cudaSuccess) return err;
  kernel<<<(unsigned)(d.B * d.Hv), kBulkThreads, kBulkBytes, stream>>>(
      static_cast<const T*>(a.q), static_cast<const T*>(a.k), static_cast<const T*>(a.v),
      a.log_alpha, a.beta, a.pool_in, a.pool_out, static_cast<T*>(a.o), d, a.lay, a.dev_status,
      wait_hooks().limit_ns);
  return cudaGetLastError();
}

template <typename T>
cudaError_t launch_typed(const RuleArgs& a, cudaStream_t stream) {
  const gdn_tree_dims& d = a.d;
  auto go = [&](auto kernel, int cols) {
    const long long blocks = (long long)d.B * d.Hv * ((d.dv + cols - 1) / cols);
    if (blocks > 0x7fffffffll) return cudaErrorInvalidConfiguration;
    kernel<<<(unsigned)blocks, kThreads, 0, stream>>>(
        static_cast<const T*>(a.q), static_cast<const T*>(a.k), static_cast<const T*>(a.v),
        a.log_alpha, a.beta, a.pool_in, a.pool_out, static_cast<T*>(a.o), d, a.lay,
        a.dev_status);
    return cudaGetLastError();
  };
  // 32 columns (128-byte row pieces) unless dv would leave half of the last tile idle
  return d.dv % 32 == 0 ? go(rule_recurrent_kernel<T, 32>, 32)
                        : go(rule_recurrent_kernel<T, 16>, 16);
}

cudaError_t launch_recurrent(const RuleArgs& a, cudaStream_t stream) {
  return a.d.dtype == GDN_TREE_BF16 ? launch_typed<__nv_bfloat16>(a, stream)
                                    : launch_typed<float>(a, stream);
}

}  // namespace

// The chunked kernels from kChunkedFrom tokens of the longest sequence on.  Below it their two
// launches and a whole chunk's work cost more than the tokens one by one.  Measured with 32
// heads, chunked and one by one: 1 sequence of 8 tokens 16.2 and 9.3 us, of 16 15.6 and 15.7, of
// 24 15.6 and 22.5, of 64 15.8 and 55; 4 sequences of 16 27 and 22, of 24 27 and 31; 16 sequences
// of 16 80 and 66, of 24 81 and 95, of 64 83 and 251.
constexpr int kChunkedFrom = 17;
static bool chunked(const gdn_tree_dims& d, int32_t T) {
  return d.N >= kChunkedFrom && T > 0 && prefill_tc_supported(d);
}

size_t prefill_workspace_bytes(const gdn_tree_dims& d, int32_t T) {
  return chunked(d, T) ? prefill_tc_workspace_bytes(d, T) : 0;
}

cudaError_t launch_prefill(const RuleArgs& a, void* workspace, cudaStream_t stream) {
  return chunked(a.d, a.lay.T) ? launch_prefill_tc(a, workspace, stream)
                               : launch_recurrent(a, stream);
}

cudaError_t launch_decode_step(const RuleArgs& a, cudaStream_t stream) {
  // A state a CTA by bulk copies where there are many rounds of them, else four CTAs a state,
  // which have it sooner.  Measured with 32 heads: 16 sequences 17.2 and 14.3 us, 64 47.8 and
  // 46.0, 96 68.6 and 68.2, 128 87.5 and 90.2, 192 127 and 138, 256 168 and 195.
  const gdn_tree_dims& d = a.d;
  const long long units = (long long)d.B * d.Hv;
  if (d.dv == kMaxD && units >= 24 * (sm_count() > 0 ? sm_count() : 152) && units <= 0x7fffffffll)
    return d.dtype == GDN_TREE_BF16 ? launch_step_bulk<__nv_bfloat16>(a, stream)
                                    : launch_step_bulk<float>(a, stream);
  return launch_recurrent(a, stream);
}

}  // namespace gdn
