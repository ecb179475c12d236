// prefill_tc.cu -- the gated delta rule over whole sequences in chunks of 64 tokens, on the
// tensor cores (bf16, dk = dv = 128).
//
// With g_t the sum of log alpha over the chunk up to token t, S the state before the chunk,
// K, Q, V the chunk's rows (Yang et al., "Gated Delta Networks", the chunkwise form):
//     X[t,s] = beta_t e^{g_t - g_s} k_t.k_s  (s < t),     T = (I + X)^-1,
//     Y[t,s] =        e^{g_t - g_s} q_t.k_s  (s <= t),    Z = Y T,
//     R = diag(beta) (V - diag(e^g) K S),                 U = T R,
//     O = diag(e^g) Q S + Z R,
//     S <- e^{g_C} S + K^T diag(e^{g_C - g}) U.
// T and Z do not depend on the state, so a first kernel computes them for every chunk and
// head at once; a second one runs over each sequence's chunks.  Z (instead of Y U) gives
// U and O from one product, [T; Z] R, as [K; Q] S gives the two products with the state.
//
// The columns of S, V, R, U and O do not mix: the second kernel's CTA takes 32 of the 128
// value columns of one sequence and head (four times the CTAs of a head each, and a quarter
// of the work between two dependent products).  A chunk is three dependent steps,
//     D1 = [K; Q] S,   D2 = [T; Z] R,   D3 = K^T (w U),
// each an MMA of M = 128 and N = 3 x 32: the right-hand operand is an fp32 matrix as three
// bf16 parts side by side, x = hi + mid + lo exactly (8 bits each, by truncation), and the
// three results are added in fp32.  K and Q are exact in bf16; T and Z, computed in fp32,
// are three bf16 parts too; S itself lives in fp32 registers.  The state is within 1e-6 of
// the exact rule on ordinary inputs (two parts a matrix would give 3e-6, and 1e-5 of the
// largest entry where all keys are the same).
//
// What bounds it: the chain of dependent steps (MMA, TMEM to registers, split, shared
// memory, MMA), not bytes or tensor rate.  One sequence of 32768 tokens with 32 heads takes
// 1.27 ms (0.64 TB/s of inputs and outputs), 1.0 ms of it in the second kernel's chains and
// the rest in what of the first kernel does not fit beside them; 16 ragged prompts of 17 to
// 2048 tokens take 418 us.
#include <string.h>

#include "common.cuh"
#include "kernels.h"
#include "sm100.cuh"

namespace gdn {
namespace {

using namespace sm100;

constexpr int kC = 64;        // tokens of a chunk
constexpr int kD = 128;       // dk = dv
constexpr int kW = 32;        // value columns of a chain (a CTA runs one or two)
constexpr uint32_t kTileTZ = 128 * 128;            // [T; Z], one part: 128 rows x 64, 128-byte rows
constexpr uint32_t kTZBytes = 3 * kTileTZ;
constexpr uint32_t kAuxBytes = 1024;               // e^g, beta, e^{gC - g} [64] each, e^gC
constexpr uint32_t kSlotBytes = kTZBytes + kAuxBytes;
constexpr uint32_t kTileKQ = 2 * 128 * 128;        // [K; Q]: 128 rows x 128, two 64-column blocks
// What the workspace is kept to where a segment of at least kMinSegment chunks of every sequence
// fits.  It is a target, not a limit: with 32 heads 41 sequences fit; of more, a segment is
// kMinSegment chunks of each (12.8 MB a sequence), or all chunks packed where that is less.
// Shorter segments would read and write the states too often (64 KB each way a sequence and
// head, against 50 KB of tiles a chunk).
constexpr size_t kWorkspaceTarget = (size_t)512 << 20;
constexpr int kMinSegment = 8;                     // chunks a launch pair, at least

// Chunks [c0, c0 + span) of every sequence are one segment; where all chunks fit the target
// there is one, with slots packed by row position (dense = true), else
// slot = b * span + c - c0.
struct Segment {
  int c0, span;
  bool dense;
  bool by_length = false;  // the second kernel takes the longest sequences first
  bool ahead = false;      // the next segment's first kernel runs beside this one's second
};

__host__ __device__ inline long long dense_slots(long long T, long long B) { return T / kC + B + 1; }

// slot of sequence b's chunk c: cu / 64 + b is past the last slot of sequence b - 1
__device__ __forceinline__ size_t slot_of(const Segment& s, const int32_t* cu, int b, int c) {
  return s.dense ? (size_t)(cu[b] / kC + b + c) : (size_t)b * s.span + (c - s.c0);
}

// ---- waits -----------------------------------------------------------------------------
__device__ __forceinline__ bool wait_bar(uint64_t* bar, uint32_t parity, int* abort,
                                         uint64_t limit) {
  uint64_t t0 = 0;
  bool ok = true;
  for (uint32_t tries = 0; !mbar_try_wait(bar, parity); ++tries) {
    if ((tries & 63u) != 63u) continue;
    if (ld_acquire_shared(abort)) { ok = false; break; }
    const uint64_t now = globaltimer_ns();
    if (t0 == 0) t0 = now;
    if (now - t0 > limit) {
      st_release_shared(abort, 1);
      ok = false;
      break;
    }
  }
  return __all_sync(0xffffffffu, ok);  // (a whole warp waits together)
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
constexpr float kLog2e = 1.4426950408889634f;
// e^{a - b} for log-decay sums
__device__ __forceinline__ float decay(df a, df b) { return ex2(kLog2e * df_diff(a, b)); }

// bits 16 .. 31 of a and b as one word (a below)
__device__ __forceinline__ uint32_t high_halves(uint32_t a, uint32_t b) {
  return __byte_perm(a, b, 0x7632);
}
// (x, y) - (a, b), two fp32 lanes an instruction
__device__ __forceinline__ void sub2(float& x, float& y, uint32_t a, uint32_t b) {
  asm("{\n\t.reg .b64 p, q;\n\t"
      "mov.b64 p, {%0, %1};\n\tmov.b64 q, {%2, %3};\n\t"
      "sub.rn.f32x2 p, p, q;\n\tmov.b64 {%0, %1}, p;\n\t}"
      : "+f"(x), "+f"(y)
      : "r"(a), "r"(b));
}
// a pair as three bf16 pairs, exactly: truncated to 8 bits three times
__device__ __forceinline__ void split3(float a, float b, uint32_t& hi, uint32_t& mid,
                                       uint32_t& lo) {
  uint32_t ua = __float_as_uint(a), ub = __float_as_uint(b);
  hi = high_halves(ua, ub);
  sub2(a, b, ua & 0xffff0000u, ub & 0xffff0000u);
  ua = __float_as_uint(a), ub = __float_as_uint(b);
  mid = high_halves(ua, ub);
  sub2(a, b, ua & 0xffff0000u, ub & 0xffff0000u);
  lo = high_halves(__float_as_uint(a), __float_as_uint(b));
}

// 8 consecutive values of row r of [T; Z] as three parts
__device__ __forceinline__ void store_tz(unsigned char* base, int r, int c8, const float (&x)[8]) {
  uint4 hi, mid, lo;
  split3(x[0], x[1], hi.x, mid.x, lo.x);
  split3(x[2], x[3], hi.y, mid.y, lo.y);
  split3(x[4], x[5], hi.z, mid.z, lo.z);
  split3(x[6], x[7], hi.w, mid.w, lo.w);
  const uint32_t off = sw128_chunk(r, c8);
  *reinterpret_cast<uint4*>(base + off) = hi;
  *reinterpret_cast<uint4*>(base + kTileTZ + off) = mid;
  *reinterpret_cast<uint4*>(base + 2 * kTileTZ + off) = lo;
}

// zero rows [from, 64) of the K half of a [K; Q] tile (whole warp)
__device__ __forceinline__ void zero_k_rows(unsigned char* tile, int from, int lane) {
  for (int e = from * 16 + lane; e < kC * 16; e += 32) {
    const int r = e >> 4, c = e & 15;
    *reinterpret_cast<uint4*>(tile + (c >> 3) * kSw128TileBytes + r * 128 + ((c & 7) << 4)) =
        make_uint4(0, 0, 0, 0);
  }
}

// the [K; Q] tile of a chunk: rows 0-63 K, 64-127 Q, by TMA (one thread)
__device__ __forceinline__ void load_kq(unsigned char* tile, const CUtensorMap* mapK,
                                        const CUtensorMap* mapQ, uint64_t* bar, int hq, int row) {
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    tma_load_3d(tile + c * kSw128TileBytes, mapK, bar, 64 * c, hq, row);
    tma_load_3d(tile + c * kSw128TileBytes + kC * 128, mapQ, bar, 64 * c, hq, row);
  }
}

// ---- first kernel: T and Z of every chunk and head --------------------------------------
// T = (I + X)^-1 by blocks: the four 16 x 16 blocks of the diagonal column by column, then
// twice the block below the diagonal of a pair, T21 = -T22 X21 T11 (16, then 32 rows).
// Z = Y T on the tensor cores.  Bound by shared memory reads and the latency of these short
// steps: three CTAs an SM hide it in one another (one array for X and T, and T over K and Q,
// make them fit).  About 9 us a CTA of which the copies in take 2, the inverse 3; 8192 chunks
// and heads 210 us.
constexpr int kPrepThreads = 256;
constexpr int kWarpTmem = 2;  // the warp that holds the TMEM columns
constexpr int kAld = 72;  // floats a row (8 of a row and 4 rows lie in all banks)

struct PrepShared {
  // below and on the diagonal T, above it X^T (X[t][s] at [s][t]); a diagonal block that is
  // done holds T^T above its diagonal
  float A[kC][kAld];
  float P[kC / 2][kC / 2 + 8];  // a product of blocks on its way
  df g[kC];
  float beta[kC], up[kC], down[kC];  // e^{g - g_mid}, e^{g_mid - g}
  uint64_t bar, mma;
  uint32_t tmem;
  int abort, mild;
};
constexpr uint32_t kPrepTiles = kTZBytes > kTileKQ ? kTZBytes : kTileKQ;  // [K; Q], then [T; Z]
constexpr uint32_t kPrepBytes = kPrepTiles + sizeof(PrepShared) + 1024;

// x as the sum of two numbers of 11 significant bits (and the rest, below 2^-22 of it)
__device__ __forceinline__ void split_tf32(float x, uint32_t& hi, uint32_t& lo) {
  hi = __float_as_uint(x) & 0xffffe000u;
  lo = __float_as_uint(x - __uint_as_float(hi)) + 0x1000u;  // (the product drops the last 13)
}
__device__ __forceinline__ void mma_tf32(float (&d)[4], const uint32_t (&a)[4],
                                         const uint32_t (&b)[2]) {
  asm volatile(
      "mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]));
}

// T21 = -T22 X21 T11 for the pair of n x n blocks at `o`: a warp's 16 rows and 8 columns of
// P = X21 T11, then (kSecond) of T22 P, with d[0], d[1] at row lane / 4 and columns 2 (lane %
// 4), + 1, and d[2], d[3] 8 rows below.  The operands are two parts each and three of their
// four products are kept (2^-22 of a term; fp32 sums).  Shared memory reads bound this
// kernel, and CUDA cores needed three times as many.
template <int n, bool kSecond>
__device__ __forceinline__ void block_product(const PrepShared& S, int o, int po, int mt, int nt,
                                              int lane, float (&d)[4]) {
  const int g = lane >> 2, t = lane & 3, j = 8 * nt + g;
#pragma unroll
  for (int e = 0; e < 4; ++e) d[e] = 0.f;
#pragma unroll
  for (int s = 0; s < n / 8; ++s) {
    // T11 and T22 are triangular
    if (kSecond ? 8 * s > 16 * mt + 15 : 8 * s + 7 < 8 * nt) continue;
    uint32_t ah[4], al[4], bh[2], bl[2];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int i = 16 * mt + g + 8 * (e & 1), k = 8 * s + t + 4 * (e >> 1);
      float x = kSecond ? S.A[o + n + k][o + n + i] : S.A[o + k][o + n + i];
      if (kSecond && k > i) x = 0.f;
      split_tf32(x, ah[e], al[e]);
    }
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int k = 8 * s + t + 4 * e;
      float x = kSecond ? S.P[po + k][j] : S.A[o + k][o + j];
      if (!kSecond && j > k) x = 0.f;
      split_tf32(x, bh[e], bl[e]);
    }
    mma_tf32(d, al, bh);
    mma_tf32(d, ah, bl);
    mma_tf32(d, ah, bh);
  }
}

// One CTA of a first kernel that began beside the second kernel of the segment before waits for
// that one's end, so that whatever follows this kernel follows both.
__device__ __forceinline__ void scan_done() {
  if (blockIdx.x == 0) asm volatile("griddepcontrol.wait;" ::: "memory");
}

__global__ void __launch_bounds__(kPrepThreads, 3)
prefill_prep_kernel(const __grid_constant__ CUtensorMap mapK,
                    const __grid_constant__ CUtensorMap mapQ, const float* __restrict__ log_alpha,
                    const float* __restrict__ beta, gdn_tree_dims d, SeqLayout lay, Segment seg,
                    unsigned char* ws, int32_t* dev_status, WaitHooks hooks) {
  const uint64_t limit_ns = hooks.limit_ns;
  extern __shared__ unsigned char smem_raw[];
  unsigned char* smem = reinterpret_cast<unsigned char*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  unsigned char* sKQ = smem;
  unsigned char* sTZ = smem;
  PrepShared& P = *reinterpret_cast<PrepShared*>(smem + kPrepTiles);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int h = blockIdx.x % d.Hv, slot = blockIdx.x / d.Hv;
  const int hq = h / (d.Hv / d.Hqk);
  if (tid == 0) {
    tma_prefetch_desc(&mapK);
    tma_prefetch_desc(&mapQ);
    mbar_init(&P.bar, 1);
    mbar_init(&P.mma, 1);
    P.abort = 0;
    mbar_fence_init();
  }
  if (warp == kWarpTmem) tmem_alloc(&P.tmem, 128);
  int b, c;
  if (seg.dense) {  // the last sequence whose first slot is not past this one, 32 a probe
    int lo = 0, hi = d.B;
    while (hi - lo > 1) {
      const int step = (hi - lo + 31) >> 5, m = lo + lane * step;
      const bool not_past = m < hi && lay.cu[m] / kC + m <= slot;
      lo += max(__popc(__ballot_sync(0xffffffffu, not_past)) - 1, 0) * step;
      hi = min(hi, lo + step);
    }
    b = lo;
    c = slot - (lay.cu[b] / kC + b);
  } else {
    b = slot / seg.span;
    c = seg.c0 + slot % seg.span;
  }
  const int n = lay.count(b, d.N);
  // (an invalid sequence is reported by the second kernel; its offset may give any c)
  if (n < 0 || c < 0 || n <= (long long)c * kC) {
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    if (warp == kWarpTmem) tmem_dealloc(P.tmem, 128);
    scan_done();
    return;
  }
  const int nc = min(kC, n - c * kC);
  const size_t row = (size_t)lay.cu[b] + (size_t)c * kC;
  if (tid == 0) {
    mbar_arrive_expect_tx(&P.bar, kTileKQ);
    if (b != hooks.withhold_copy_seq) load_kq(sKQ, &mapK, &mapQ, &P.bar, hq, (int)row);
  }
  float la[2] = {0.f, 0.f}, be[2] = {0.f, 0.f};  // the gates of rows 2 lane and 2 lane + 1
  if (warp == 1) {
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      if (2 * lane + e >= nc) continue;
      // (past L1, where the lines of cu are to stay)
      la[e] = __ldcg(log_alpha + (row + 2 * lane + e) * d.Hv + h);
      be[e] = __ldcg(beta + (row + 2 * lane + e) * d.Hv + h);
    }
  }

  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = P.tmem;
  unsigned char* out = ws + ((size_t)slot * d.Hv + h) * kSlotBytes;
  if (warp == 1) {
    // g by a scan of pairs; -inf (alpha = 0) becomes -1e4: e^-1e4 is 0 as well, and
    // differences of sums stay defined
    df x[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      x[e] = df{la[e] < -1e4f ? -1e4f : la[e], 0.f};
      P.beta[2 * lane + e] = be[e];
    }
    x[1] = df_add(x[0], x[1]);
    df run = x[1];
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const df y = {__shfl_up_sync(0xffffffffu, run.hi, off), __shfl_up_sync(0xffffffffu, run.lo, off)};
      if (lane >= off) run = df_add(y, run);
    }
    const df before = {__shfl_up_sync(0xffffffffu, run.hi, 1), __shfl_up_sync(0xffffffffu, run.lo, 1)};
    const df g0 = lane > 0 ? df_add(before, x[0]) : x[0];
    P.g[2 * lane] = g0;
    P.g[2 * lane + 1] = run;
    // within e^+-40 of the middle every weight is a product of two factors
    const df mid = {__shfl_sync(0xffffffffu, run.hi, 15), __shfl_sync(0xffffffffu, run.lo, 15)};
    const float d0 = df_diff(g0, mid), d1 = df_diff(run, mid);
    P.up[2 * lane] = ex2(kLog2e * d0);
    P.up[2 * lane + 1] = ex2(kLog2e * d1);
    P.down[2 * lane] = ex2(-kLog2e * d0);
    P.down[2 * lane + 1] = ex2(-kLog2e * d1);
    const bool mild = fabsf(d0) <= 40.f && fabsf(d1) <= 40.f;
    const bool all = __all_sync(0xffffffffu, mild);
    if (lane == 0) P.mild = all;
    const df last = {__shfl_sync(0xffffffffu, run.hi, 31), __shfl_sync(0xffffffffu, run.lo, 31)};
    float* aux = reinterpret_cast<float*>(out + kTZBytes);
#pragma unroll
    for (int e = 0; e < 2; ++e) {  // (rows past the sequence add nothing to g)
      const int i = 2 * lane + e;
      const df gi = e ? run : g0;
      aux[i] = ex2(kLog2e * df_value(gi));
      aux[kC + i] = be[e];
      aux[2 * kC + i] = i < nc ? decay(last, gi) : 0.f;
    }
    if (lane == 0) aux[3 * kC] = ex2(kLog2e * df_value(last));
  }
  // [K; Q] K^T: lanes 0-63 the rows k_t.k_s, lanes 64-127 q_t.k_s
  if (warp == 0) {
    if (wait_bar(&P.bar, 0, &P.abort, limit_ns) && elect_one()) {
      constexpr uint32_t id = idesc_bf16_f32(128, kC);
      const uint64_t a = desc_sw128_kmajor(smem_addr(sKQ));
#pragma unroll
      for (int s = 0; s < kD / 16; ++s) {
        const uint32_t off = ((s >> 2) * kSw128TileBytes + (s & 3) * 32) >> 4;
        if (s == 0) umma_ss<false>(tmem, a + off, a + off, id);
        else umma_ss<true>(tmem, a + off, a + off, id);
      }
      umma_commit(&P.mma);
    }
    __syncwarp();
  }
  // thread: TMEM lane 32 (warp & 3) + lane, columns 32 half ..
  const int half = warp >> 2, ln = 32 * (warp & 3) + lane, t = ln & (kC - 1);
  const bool isq = ln >= kC;
  const uint32_t tl = tmem + ((uint32_t)(32 * (warp & 3)) << 16);
  bool ok = wait_bar(&P.mma, 0, &P.abort, limit_ns);
  tc_fence_after_sync();
  ok = __syncthreads_and(ok);  // (every warp goes on, or none)
  if (ok) {
    float gram[32];
    tmem_ld_32cols(tl + 32 * half, gram);
    {  // X^T in fp32 above the diagonal; Y in rows 64-127 of the [T; Z] tiles
      const bool live = t < nc;
      if (P.mild) {
        const float f = (isq ? 1.f : P.beta[t]) * P.up[t];
#pragma unroll
        for (int e = 0; e < 32; e += 4) {
          const float4 w = *reinterpret_cast<const float4*>(&P.down[32 * half + e]);
          gram[e] *= f * w.x;
          gram[e + 1] *= f * w.y;
          gram[e + 2] *= f * w.z;
          gram[e + 3] *= f * w.w;
        }
      } else {
        const df gt = P.g[t];
        const float f = isq ? 1.f : P.beta[t];
#pragma unroll
        for (int e = 0; e < 32; ++e) {
          const int s = 32 * half + e;
          gram[e] *= s <= t ? f * decay(gt, P.g[s]) : 0.f;
        }
      }
      if (!isq) {
#pragma unroll
        for (int e = 0; e < 32; ++e) {
          const int s = 32 * half + e;
          if (s < t) P.A[s][t] = live ? gram[e] : 0.f;
        }
      } else {
#pragma unroll
        for (int c8 = 0; c8 < 4; ++c8) {
          float y[8];
#pragma unroll
          for (int e = 0; e < 8; ++e)
            y[e] = live && 32 * half + 8 * c8 + e <= t ? gram[8 * c8 + e] : 0.f;
          store_tz(sTZ, ln, 4 * half + c8, y);
        }
      }
    }
    __syncthreads();
    if (tid < kC) {  // the diagonal blocks: a thread a column
      const int o = tid & ~15, j = tid & 15;
      float u[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) u[i] = i == j ? 1.f : 0.f;
#pragma unroll
      for (int s = 0; s < 15; ++s) {
        float x[16];  // column s of X, 16-byte pieces (those that hold rows past s)
#pragma unroll
        for (int i = 4 * ((s + 1) / 4); i < 16; i += 4)
          *reinterpret_cast<float4*>(x + i) = *reinterpret_cast<const float4*>(&P.A[o + s][o + i]);
#pragma unroll
        for (int i = s + 1; i < 16; ++i) u[i] = fmaf(-x[i], u[s], u[i]);
      }
      __syncwarp();
#pragma unroll
      for (int i = 0; i < 16; ++i)
        if (i >= j) P.A[o + i][o + j] = P.A[o + j][o + i] = u[i];
    }
    __syncthreads();
    {  // pairs of 16-row blocks: two warps a pair
      const int pr = warp >> 1, nt = warp & 1, o = 32 * pr, i = lane >> 2, j = 8 * nt + 2 * (lane & 3);
      float x[4];
      if (warp < 4) {
        block_product<16, false>(P, o, 16 * pr, 0, nt, lane, x);
        *reinterpret_cast<float2*>(&P.P[16 * pr + i][j]) = make_float2(x[0], x[1]);
        *reinterpret_cast<float2*>(&P.P[16 * pr + i + 8][j]) = make_float2(x[2], x[3]);
      }
      __syncthreads();
      if (warp < 4) {
        block_product<16, true>(P, o, 16 * pr, 0, nt, lane, x);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int ie = i + 8 * (e >> 1), je = j + (e & 1);
          P.A[o + 16 + ie][o + je] = -x[e];
          if (pr == 1) P.A[o + je][o + 16 + ie] = -x[e];
        }
      }
    }
    __syncthreads();
    {  // the pair of 32-row blocks
      const int mt = warp & 1, nt = warp >> 1, i = 16 * mt + (lane >> 2), j = 8 * nt + 2 * (lane & 3);
      float x[4];
      block_product<32, false>(P, 0, 0, mt, nt, lane, x);
      *reinterpret_cast<float2*>(&P.P[i][j]) = make_float2(x[0], x[1]);
      *reinterpret_cast<float2*>(&P.P[i + 8][j]) = make_float2(x[2], x[3]);
      __syncthreads();
      block_product<32, true>(P, 0, 0, mt, nt, lane, x);
      *reinterpret_cast<float2*>(&P.A[32 + i][j]) = make_float2(-x[0], -x[1]);
      *reinterpret_cast<float2*>(&P.A[32 + i + 8][j]) = make_float2(-x[2], -x[3]);
    }
    __syncthreads();
    // T in rows 0-63 of the tiles
#pragma unroll
    for (int e = tid; e < kC * 8; e += kPrepThreads) {
      const int r = e >> 3, c8 = e & 7;
      float x[8];
      *reinterpret_cast<float4*>(x) = *reinterpret_cast<const float4*>(&P.A[r][8 * c8]);
      *reinterpret_cast<float4*>(x + 4) = *reinterpret_cast<const float4*>(&P.A[r][8 * c8 + 4]);
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = 8 * c8 + i <= r ? x[i] : 0.f;
      store_tz(sTZ, r, c8, x);
    }
    fence_proxy_async_smem();
    tc_fence_before_sync();
    __syncthreads();
    // the tiles go to the workspace as they lie, T's rows now and Z's when they are there
    if (tid == 32) {
#pragma unroll
      for (int p = 0; p < 3; ++p) bulk_store(out + p * kTileTZ, sTZ + p * kTileTZ, kTileTZ / 2);
      bulk_commit_group();
    }
    // Z = Y T: lanes 64-127 of [T; Y] T (T as an operand whose rows are the inner index)
    if (warp == 0) {
      tc_fence_after_sync();
      if (elect_one()) {
        constexpr uint32_t id = idesc_bf16_f32_bmn(128, kC);
        const uint64_t a = desc_sw128_kmajor(smem_addr(sTZ));
        const uint64_t bt = desc_sw128_mnmajor(smem_addr(sTZ), kSw128TileBytes, 1024);
#pragma unroll
        for (int p = 0; p < 6; ++p) {  // the products of parts above 2^-24
          constexpr int kA[6] = {0, 0, 1, 1, 0, 2}, kB[6] = {0, 1, 0, 1, 2, 0};
          const uint64_t ap = a + kA[p] * (kTileTZ >> 4), bp = bt + kB[p] * (kTileTZ >> 4);
#pragma unroll
          for (int s = 0; s < kC / 16; ++s) {
            if (p == 0 && s == 0) umma_ss<false>(tmem + 64, ap + ((s * 32) >> 4), bp + ((s * 2048) >> 4), id);
            else umma_ss<true>(tmem + 64, ap + ((s * 32) >> 4), bp + ((s * 2048) >> 4), id);
          }
        }
        umma_commit(&P.mma);
      }
      __syncwarp();
    }
    ok = wait_bar(&P.mma, 1, &P.abort, limit_ns);
    tc_fence_after_sync();
    if (ok && isq) {
      tmem_ld_32cols(tl + 64 + 32 * half, gram);
#pragma unroll
      for (int c8 = 0; c8 < 4; ++c8) {
        float y[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) y[e] = gram[8 * c8 + e];
        store_tz(sTZ, ln, 4 * half + c8, y);
      }
    }
    fence_proxy_async_smem();
    __syncthreads();
    // (the second kernel may set up now, where its launch says so)
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (tid == 32) {
      if (ok) {
#pragma unroll
        for (int p = 0; p < 3; ++p)
          bulk_store(out + p * kTileTZ + kTileTZ / 2, sTZ + p * kTileTZ + kTileTZ / 2, kTileTZ / 2);
        bulk_commit_group();
      }
      bulk_wait_read_all();  // (the kernel's end is what the reader waits for)
    }
  }
  // (after a timeout: the copies and MMAs in flight end, or their bounded waits do)
  if (P.abort && warp == 0) {
    mbar_wait(&P.bar, 0, limit_ns);
    mbar_wait(&P.mma, 0, limit_ns);
    mbar_wait(&P.mma, 1, limit_ns);
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  if (tid == 0 && P.abort && dev_status) atomicMax(dev_status + b, GDN_TREE_STATUS_TIMEOUT);
  if (warp == kWarpTmem) tmem_dealloc(tmem, 128);
  scan_done();
}

// ---- second kernel: the chunks of a sequence, 32 value columns a chain ---------------------
// A CTA runs one chain of dependent steps (3800 cycles a chunk, of which its MMAs are 1250),
// or two, over the same keys, queries and [T; Z], whose steps fill one another's waits (6300
// cycles for both): two where that takes the SMs fewer cycles in all.  Measured, one and two a
// CTA: 2048 tokens of 32 heads (128 chains) 103 and 149 us, of 40 heads (160) 167 and 150.
constexpr int kChainThreads = 256;   // two threads a TMEM lane, 16 columns each
constexpr int kStages = 2;
// right-hand operands: rows of 3 x 32 bf16 (hi, mid | lo, unused) in two 64-column atoms; S
// for the first product, then R, then w U (64 rows) in the same place
constexpr uint32_t kOperand = kD * 256;

struct ChainBars {
  uint64_t d1, d2, d3, r_ready, u_ready, s_ready, drain;
};
struct ScanBars {
  uint64_t raw, full[kStages], empty[kStages];
  ChainBars chain[2];
  uint32_t tmem;
  int abort;
  int unit;  // the sequence
};
static_assert(sizeof(ScanBars) <= 256, "the barriers fit their place");

template <int kChains>
struct Scan {
  static constexpr int kSlices = kD / kW / kChains;
  static constexpr int kCompute = kChains * kChainThreads;
  // + a loading warp and an issuing one for each chain
  static constexpr int kThreads = kCompute + 32 + 32 * kChains;
  static constexpr int kWarpLoad = kCompute / 32, kWarpMma = kWarpLoad + 1;
  static constexpr uint32_t kTmemColumns = 256 * kChains;
  static constexpr uint32_t OFF_KQ = 0;
  static constexpr uint32_t OFF_TZ = OFF_KQ + kStages * kTileKQ;
  static constexpr uint32_t OFF_X = OFF_TZ + kStages * kSlotBytes;  // ([T; Z] and weights)
  static constexpr uint32_t OFF_BAR = OFF_X + kChains * kOperand;
  static constexpr uint32_t kBytes = OFF_BAR + 256;
};

// two fp32 lanes an instruction: (a, b) * w; (a, b) * x + (c, d); (a, b) + (c, d)
__device__ __forceinline__ void mul2(float& a, float& b, float w) {
  asm("{\n\t.reg .b64 p, q;\n\t"
      "mov.b64 p, {%0, %1};\n\tmov.b64 q, {%2, %2};\n\t"
      "mul.rn.f32x2 p, p, q;\n\tmov.b64 {%0, %1}, p;\n\t}"
      : "+f"(a), "+f"(b)
      : "f"(w));
}
__device__ __forceinline__ void mad2(float& a, float& b, float x, float c, float d) {
  asm("{\n\t.reg .b64 p, q, r;\n\t"
      "mov.b64 p, {%0, %1};\n\tmov.b64 q, {%2, %2};\n\tmov.b64 r, {%3, %4};\n\t"
      "fma.rn.f32x2 p, p, q, r;\n\tmov.b64 {%0, %1}, p;\n\t}"
      : "+f"(a), "+f"(b)
      : "f"(x), "f"(c), "f"(d));
}
__device__ __forceinline__ void add2(float& a, float& b, float c, float d) {
  asm("{\n\t.reg .b64 p, q;\n\t"
      "mov.b64 p, {%0, %1};\n\tmov.b64 q, {%2, %3};\n\t"
      "add.rn.f32x2 p, p, q;\n\tmov.b64 {%0, %1}, p;\n\t}"
      : "+f"(a), "+f"(b)
      : "f"(c), "f"(d));
}

// 16 consecutive values of a row as three parts; `at`: the shared address of their first
// chunk (mn_chunk(row, 2 ch) of an operand; the swizzle makes the next chunk bit 4 of it and
// the middle part bit 6, the third part lies an atom further)
__device__ __forceinline__ void store_parts(uint32_t at, const float (&x)[16]) {
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    uint4 hi, mid, lo;
    split3(x[8 * e + 0], x[8 * e + 1], hi.x, mid.x, lo.x);
    split3(x[8 * e + 2], x[8 * e + 3], hi.y, mid.y, lo.y);
    split3(x[8 * e + 4], x[8 * e + 5], hi.z, mid.z, lo.z);
    split3(x[8 * e + 6], x[8 * e + 7], hi.w, mid.w, lo.w);
    const uint32_t to = at ^ (16u * e);
    auto st = [](uint32_t p, uint4 w) {
      asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(p), "r"(w.x), "r"(w.y),
                   "r"(w.z), "r"(w.w)
                   : "memory");
    };
    st(to, hi);
    st(to ^ 64u, mid);
    st(to + kMnLbo, lo);
  }
}

// the sum of the three results of 16 columns of a row (8 columns at a time: 24 registers)
template <bool kOnce>
__device__ __forceinline__ void load_sum(uint32_t taddr, float (&x)[16]) {
  if constexpr (kOnce) {  // all at once, where there are registers for it: one wait
    float y[16], z[16];
#pragma unroll
    for (int p = 0; p < 3; ++p) {
      float(&r)[16] = p == 0 ? x : p == 1 ? y : z;
      asm volatile(
          "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
          "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
          : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3]), "=f"(r[4]), "=f"(r[5]), "=f"(r[6]),
            "=f"(r[7]), "=f"(r[8]), "=f"(r[9]), "=f"(r[10]), "=f"(r[11]), "=f"(r[12]), "=f"(r[13]),
            "=f"(r[14]), "=f"(r[15])
          : "r"(taddr + p * kW));
    }
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
    for (int i = 0; i < 16; i += 2) {
      add2(y[i], y[i + 1], z[i], z[i + 1]);
      add2(x[i], x[i + 1], y[i], y[i + 1]);
    }
  } else {
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      float r[24];
#pragma unroll
      for (int p = 0; p < 3; ++p)
        asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                     : "=f"(r[8 * p]), "=f"(r[8 * p + 1]), "=f"(r[8 * p + 2]), "=f"(r[8 * p + 3]),
                       "=f"(r[8 * p + 4]), "=f"(r[8 * p + 5]), "=f"(r[8 * p + 6]), "=f"(r[8 * p + 7])
                     : "r"(taddr + p * kW + 8 * e));
      asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
      for (int i = 0; i < 8; i += 2) {
        add2(r[8 + i], r[9 + i], r[16 + i], r[17 + i]);
        add2(r[i], r[i + 1], r[8 + i], r[9 + i]);
        x[8 * e + i] = r[i];
        x[8 * e + i + 1] = r[i + 1];
      }
    }
  }
}

// From here on the first kernel's results are there.  (Every CTA comes here, so that this
// kernel never ends before that one.)
__device__ __forceinline__ void prep_done() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

template <int kChains>
__global__ void __launch_bounds__(Scan<kChains>::kThreads, 1)
prefill_scan_kernel(const __grid_constant__ CUtensorMap mapK,
                    const __grid_constant__ CUtensorMap mapQ,
                    const __grid_constant__ CUtensorMap mapV, const __nv_bfloat16* __restrict__ v,
                    const float* pool_in, float* pool_out, __nv_bfloat16* __restrict__ o,
                    gdn_tree_dims d, SeqLayout lay, Segment seg, const unsigned char* ws,
                    int32_t* dev_status, WaitHooks hooks) {
  using L = Scan<kChains>;
  const uint64_t limit_ns = hooks.limit_ns;
  extern __shared__ __align__(1024) unsigned char smem[];
  ScanBars* B = reinterpret_cast<ScanBars*>(smem + L::OFF_BAR);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int slice = blockIdx.x % L::kSlices;
  const int h = (blockIdx.x / L::kSlices) % d.Hv;
  const int hq = h / (d.Hv / d.Hqk);
  int b = blockIdx.x / L::kSlices / d.Hv;
  if (seg.by_length) {  // (found by one warp)
    if (warp == 0) {
      const int x0 = lane < d.B ? lay.cu[lane + 1] - lay.cu[lane] : kNoRank;
      const int x1 = lane + 32 < d.B ? lay.cu[lane + 33] - lay.cu[lane + 32] : kNoRank;
      b = nth_largest(x0, x1, d.B, b, lane);
      if (lane == 0) B->unit = b;
    }
    __syncthreads();
    b = B->unit;
  }
  const int n = lay.count(b, d.N), st = lay.state(b);
  if (n < 0 || st < 0) {
    if (dev_status && tid == 0) atomicMax(dev_status + b, GDN_TREE_STATUS_BAD_LAYOUT);
    prep_done();
    return;
  }
  const int chunks = (n + kC - 1) / kC;
  const int c_end = min(chunks, seg.c0 + seg.span);
  if (seg.c0 > 0 && c_end <= seg.c0) {  // this sequence ended in an earlier segment
    prep_done();
    return;
  }
  const size_t row0 = (size_t)lay.cu[b];

  if (tid == 0) {
    mbar_init(&B->raw, 1);
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&B->full[s], 1);
      mbar_init(&B->empty[s], kChains);
    }
    for (int x = 0; x < kChains; ++x) {
      ChainBars& C = B->chain[x];
      mbar_init(&C.d1, 1);
      mbar_init(&C.d2, 1);
      mbar_init(&C.d3, 1);
      mbar_init(&C.drain, 1);
      mbar_init(&C.r_ready, kChainThreads / 32);  // (warps)
      mbar_init(&C.u_ready, kChainThreads / 64);
      mbar_init(&C.s_ready, kChainThreads / 32);
    }
    // (the swizzled tiles need their 1024-byte boundary)
    B->abort = (smem_addr(smem) & 1023u) != 0;
    mbar_fence_init();
  }
  if (warp == L::kWarpMma) tmem_alloc(&B->tmem, L::kTmemColumns);
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem0 = B->tmem;
  // TMEM columns of a chain; D3 takes D1's place (all have read D1 before U is there)
  constexpr uint32_t kD1 = 0, kD2 = 3 * kW, kD3 = 0;
  const bool run = B->abort == 0;

  if (warp == L::kWarpLoad) {
    prep_done();
    // (the next segment's first kernel, where its launch asks for it, may start now)
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const unsigned char* tz = ws + (slot_of(seg, lay.cu, b, seg.c0) * d.Hv + h) * (size_t)kSlotBytes;
    for (int c = seg.c0; run && c < c_end; ++c) {
      const int i = c - seg.c0, s = i % kStages;
      if (i >= kStages && !wait_bar(&B->empty[s], ((i / kStages) & 1) ^ 1, &B->abort, limit_ns)) break;
      const int nc = min(kC, n - c * kC);
      unsigned char* kq = smem + L::OFF_KQ + s * kTileKQ;
      // (the last chunk's tile passes through this warp: rows past the sequence are not
      // its own, and a zero weight must not meet what they hold)
      uint64_t* bar = nc < kC ? &B->raw : &B->full[s];
      if (elect_one()) {
        mbar_arrive_expect_tx(bar, kTileKQ + kSlotBytes);
        load_kq(kq, &mapK, &mapQ, bar, hq, (int)(row0 + (size_t)c * kC));
        bulk_load(smem + L::OFF_TZ + s * kSlotBytes, tz, kSlotBytes, bar);
        // (v goes straight to the compute threads' registers, a chunk ahead: from L2)
        tma_prefetch_l2_3d(&mapV, slice * kChains * kW, h, (int)(row0 + (size_t)(c + 1) * kC));
      }
      __syncwarp();
      tz += (size_t)d.Hv * kSlotBytes;
      if (nc < kC) {
        if (!wait_bar(&B->raw, 0, &B->abort, limit_ns)) break;
        zero_k_rows(kq, nc, lane);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&B->full[s]);
      }
    }
  } else if (warp >= L::kWarpMma) {
    const int x = warp - L::kWarpMma;
    ChainBars& C = B->chain[x];
    const uint32_t tmem = tmem0 + 256 * x;
    constexpr uint32_t id1 = idesc_bf16_f32_bmn(128, 3 * kW), id2 = idesc_bf16_f32_bmn(128, 2 * kW),
                       id4 = idesc_bf16_f32_bmn(128, kW);
    constexpr uint32_t id3 = idesc_bf16_f32_amn_bmn(128, 3 * kW);
    const uint64_t dKQ = desc_sw128_kmajor(smem_addr(smem + L::OFF_KQ));
    const uint64_t dKt = desc_sw128_mnmajor(smem_addr(smem + L::OFF_KQ), kSw128TileBytes, 1024);
    const uint64_t dTZ = desc_sw128_kmajor(smem_addr(smem + L::OFF_TZ));
    const uint64_t dX = desc_sw128_mnmajor(smem_addr(smem + L::OFF_X + x * kOperand), kMnLbo, kMnSbo);
    constexpr uint32_t kStep = (2 * kMnSbo) >> 4;  // 16 rows of the right-hand operand
    // (the operands that the compute warps wrote reach the tensor cores' proxy by this warp's
    // fence, one for all of them, behind the barrier: a fence in each of their warps took a
    // third of their time)
    bool ok = run;
    for (int c = seg.c0; ok && c < c_end; ++c) {
      const int i = c - seg.c0, s = i % kStages;
      const uint64_t kq = dKQ + s * (kTileKQ >> 4), kt = dKt + s * (kTileKQ >> 4),
                     tz = dTZ + s * (kSlotBytes >> 4);
      ok = wait_bar(&B->full[s], (i / kStages) & 1, &B->abort, limit_ns) &&
           wait_bar(&C.s_ready, i & 1, &B->abort, limit_ns);
      if (!ok) break;
      tc_fence_after_sync();
      fence_proxy_async_smem();
      if (elect_one()) {
#pragma unroll
        for (int e = 0; e < kD / 16; ++e) {
          const uint32_t off = ((e >> 2) * kSw128TileBytes + (e & 3) * 32) >> 4;
          if (e == 0) umma_ss<false>(tmem + kD1, kq + off, dX + e * kStep, id1);
          else umma_ss<true>(tmem + kD1, kq + off, dX + e * kStep, id1);
        }
        umma_commit(&C.d1);
      }
      __syncwarp();
      ok = wait_bar(&C.r_ready, i & 1, &B->abort, limit_ns);
      if (!ok) break;
      tc_fence_after_sync();
      fence_proxy_async_smem();
      if (elect_one()) {
#pragma unroll
        for (int e = 0; e < kC / 16; ++e) {  // hi (hi, mid, lo)
          if (e == 0) umma_ss<false>(tmem + kD2, tz + ((e * 32) >> 4), dX + e * kStep, id1);
          else umma_ss<true>(tmem + kD2, tz + ((e * 32) >> 4), dX + e * kStep, id1);
        }
#pragma unroll
        for (int e = 0; e < kC / 16; ++e)    // mid (hi, mid)
          umma_ss<true>(tmem + kD2, tz + ((kTileTZ + e * 32) >> 4), dX + e * kStep, id2);
#pragma unroll
        for (int e = 0; e < kC / 16; ++e)    // lo (hi)
          umma_ss<true>(tmem + kD2, tz + ((2 * kTileTZ + e * 32) >> 4), dX + e * kStep, id4);
        umma_commit(&C.d2);
      }
      __syncwarp();
      ok = wait_bar(&C.u_ready, i & 1, &B->abort, limit_ns);
      if (!ok) break;
      tc_fence_after_sync();
      fence_proxy_async_smem();
      if (elect_one()) {
#pragma unroll
        for (int e = 0; e < kC / 16; ++e) {
          if (e == 0) umma_ss<false>(tmem + kD3, kt + ((e * 2048) >> 4), dX + e * kStep, id3);
          else umma_ss<true>(tmem + kD3, kt + ((e * 2048) >> 4), dX + e * kStep, id3);
        }
        umma_commit(&C.d3);
        umma_commit(&B->empty[s]);
      }
      __syncwarp();
    }
    // whatever was issued is done before TMEM and the operands go
    if (elect_one()) umma_commit(&C.drain);
    __syncwarp();
    mbar_wait(&C.drain, 0, limit_ns);
  } else {
    // ---- compute: thread (chain, TMEM lane ln, column half ch) --------------------------------
    const int x0 = warp / (kChainThreads / 32), ch = (warp >> 2) & 1, ln = 32 * (warp & 3) + lane;
    ChainBars& C = B->chain[x0];
    const uint32_t tl = tmem0 + 256 * x0 + ((uint32_t)(32 * (warp & 3)) << 16) + 16 * ch;
    const bool isq = ln >= kC;
    const int t = ln & (kC - 1);
    const int col = (slice * kChains + x0) * kW + 16 * ch;  // first value column
    const size_t soff = ((size_t)st * d.Hv + h) * kD * kD + (size_t)ln * kD + col;
    // where this thread's parts go: row ln of S, row t of R and w U
    const uint32_t sX = smem_addr(smem + L::OFF_X + x0 * kOperand);
    const uint32_t to_s = sX + mn_chunk(ln, 2 * ch), to_r = sX + mn_chunk(t, 2 * ch);
    // row ln of the state, 16 columns
    float S[16];
    const float* src = (seg.c0 == 0 ? pool_in : pool_out) + soff;
#pragma unroll
    for (int e = 0; e < 4; ++e)
      *reinterpret_cast<float4*>(S + 4 * e) = *reinterpret_cast<const float4*>(src + 4 * e);
    bool ok = run;
    if (seg.c0 < c_end) {
      store_parts(to_s, S);
      if (!(b * d.Hv + h == hooks.withhold_unit && warp == hooks.withhold_node))
        mbar_arrive_warp(&C.s_ready);
    }
    // this token's v (16 columns) and weights, a chunk ahead (the pointers go along: nothing
    // is looked up on the way)
    uint4 vn[2];
    const size_t v_step = (size_t)kC * d.Hv * kD;
    const size_t first = ((row0 + (size_t)seg.c0 * kC + t) * d.Hv + h) * kD + col;
    const __nv_bfloat16* vp = v + first;
    __nv_bfloat16* op = o + first;
    int left = n - seg.c0 * kC - t;  // > 0: the token is there
    auto fetch_v = [&](bool live) {
      vn[0] = vn[1] = make_uint4(0, 0, 0, 0);
      if (!isq && live) {
        vn[0] = __ldg(reinterpret_cast<const uint4*>(vp));
        vn[1] = __ldg(reinterpret_cast<const uint4*>(vp) + 1);
      }
      vp += v_step;
    };
    if (seg.c0 < c_end) fetch_v(left > 0);
    for (int c = seg.c0; ok && c < c_end; ++c) {
      const int i = c - seg.c0, s = i % kStages;
      ok = wait_bar(&B->full[s], (i / kStages) & 1, &B->abort, limit_ns);
      if (!ok) break;
      const float* aux = reinterpret_cast<const float*>(smem + L::OFF_TZ + s * kSlotBytes + kTZBytes);
      const float gam = aux[t], bt = aux[kC + t], w = aux[2 * kC + t], gC = aux[3 * kC];
      ok = wait_bar(&C.d1, i & 1, &B->abort, limit_ns);
      if (!ok) break;
      tc_fence_after_sync();
      float x[16];
      load_sum<kChains == 1>(tl + kD1, x);
      if (!isq) {
        const uint32_t* vw = reinterpret_cast<const uint32_t*>(vn);
#pragma unroll
        for (int e = 0; e < 16; e += 2) {  // (rows past the sequence: k = v = beta = 0)
          const uint32_t v2 = vw[e >> 1];
          mad2(x[e], x[e + 1], -gam, __uint_as_float(v2 << 16), __uint_as_float(v2 & 0xffff0000u));
          mul2(x[e], x[e + 1], bt);
        }
        store_parts(to_r, x);
      }
      tc_fence_before_sync();
      mbar_arrive_warp(&C.r_ready);
      if (c + 1 < c_end) fetch_v(left > kC);  // (the next chunk's, a chunk ahead of its use)
      ok = wait_bar(&C.d2, i & 1, &B->abort, limit_ns);
      if (!ok) break;
      tc_fence_after_sync();
      float y[16];
      load_sum<kChains == 1>(tl + kD2, y);
      if (!isq) {
#pragma unroll
        for (int e = 0; e < 16; e += 2) mul2(y[e], y[e + 1], w);
        store_parts(to_r, y);
        tc_fence_before_sync();
        mbar_arrive_warp(&C.u_ready);
      } else if (left > 0) {
        uint32_t p[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const __nv_bfloat162 q2 = __floats2bfloat162_rn(fmaf(gam, x[2 * e], y[2 * e]),
                                                          fmaf(gam, x[2 * e + 1], y[2 * e + 1]));
          p[e] = *reinterpret_cast<const uint32_t*>(&q2);
        }
        uint4* to = reinterpret_cast<uint4*>(op);
        to[0] = make_uint4(p[0], p[1], p[2], p[3]);
        to[1] = make_uint4(p[4], p[5], p[6], p[7]);
      }
      __syncwarp();
      ok = wait_bar(&C.d3, i & 1, &B->abort, limit_ns);
      if (!ok) break;
      tc_fence_after_sync();
      load_sum<kChains == 1>(tl + kD3, x);
#pragma unroll
      for (int e = 0; e < 16; e += 2) mad2(S[e], S[e + 1], gC, x[e], x[e + 1]);
      if (c + 1 < c_end) {
        store_parts(to_s, S);
        tc_fence_before_sync();
        mbar_arrive_warp(&C.s_ready);
      }
      op += v_step;
      left -= kC;
    }
    if (ok) {
      float* to = pool_out + soff;
#pragma unroll
      for (int e = 0; e < 4; ++e)
        *reinterpret_cast<float4*>(to + 4 * e) = *reinterpret_cast<const float4*>(S + 4 * e);
    }
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  if (B->abort) {
    // the copies in flight end (or their bounded waits do) before this CTA does
    if (warp == L::kWarpLoad)
      for (uint32_t ph = 0; ph < 2; ++ph) {
        for (int s = 0; s < kStages; ++s) mbar_wait(&B->full[s], ph, 1000000);
        mbar_wait(&B->raw, ph, 1000000);
      }
    __syncthreads();
    if (tid == 0 && dev_status) atomicMax(dev_status + b, GDN_TREE_STATUS_TIMEOUT);
  }
  if (warp == L::kWarpMma) tmem_dealloc(tmem0, L::kTmemColumns);
}

// The segments for these dims: chunks a launch pair, and whether one pair does for all.  Where
// the second kernel leaves SMs idle and runs for long, its segments are short, so that the next
// one's T and Z are computed on those SMs meanwhile, in the other half of the workspace.
// Measured with 32 heads (24 SMs idle), so and in as few segments as fit: 32768 tokens 1266 and
// 1377 us, 16384 660 and 688, 8192 342 and 353; with 2 heads, where the chains are all, 16384
// tokens 519 and 518.  Segments of 64 chunks 1301 us (32768 tokens), of 32 1376.
constexpr int kAheadChunks = 128;
Segment plan(const gdn_tree_dims& d, long long T) {
  const size_t head = (size_t)d.Hv * kSlotBytes;
  const long long longest = ((long long)d.N + kC - 1) / kC;
  const int sms = sm_count() > 0 ? sm_count() : 152;
  if ((long long)d.B * d.Hv * Scan<1>::kSlices <= sms - 8 && longest >= kAheadChunks &&
      2 * kAheadChunks * d.B * head <= kWorkspaceTarget) {
    long long count = (longest + kAheadChunks - 1) / kAheadChunks;
    if (count < 2) count = 2;
    Segment s{0, (int)((longest + count - 1) / count), false};
    s.ahead = true;
    return s;
  }
  if (dense_slots(T, d.B) * head <= kWorkspaceTarget) return Segment{0, (int)longest, true};
  long long span = (long long)(kWorkspaceTarget / head) / d.B;
  if (span < kMinSegment) span = kMinSegment;
  if (span > longest) span = longest;
  if (span > 0) {  // (segments of equal length)
    const long long count = (longest + span - 1) / span;
    span = (longest + count - 1) / count;
  }
  // (long batches of short sequences: packing may still be the smaller)
  if (dense_slots(T, d.B) <= span * d.B) return Segment{0, (int)longest, true};
  return Segment{0, (int)span, false};
}

}  // namespace

bool prefill_tc_supported(const gdn_tree_dims& d) {
  return d.dtype == GDN_TREE_BF16 && d.dk == kD && d.dv == kD && verify_tc_supported(
             gdn_tree_dims{1, 1, d.Hqk, d.Hv, kD, kD, GDN_TREE_BF16});
}

size_t prefill_tc_workspace_bytes(const gdn_tree_dims& d, int32_t T) {
  const Segment s = plan(d, T);
  return (size_t)(s.dense ? dense_slots(T, d.B) : (long long)s.span * d.B * (s.ahead ? 2 : 1)) *
         d.Hv * kSlotBytes;
}

cudaError_t launch_prefill_tc(const RuleArgs& a, void* workspace, cudaStream_t stream) {
  const gdn_tree_dims& d = a.d;
  CUtensorMap mapK, mapQ, mapV;
  if (!encode_head_rows_map(&mapK, a.k, a.lay.T, d.Hqk, kD, kC) ||
      !encode_head_rows_map(&mapQ, a.q, a.lay.T, d.Hqk, kD, kC) ||
      !encode_head_rows_map(&mapV, a.v, a.lay.T, d.Hv, kD, kC))
    return cudaErrorInvalidValue;
  cudaError_t err = cudaFuncSetAttribute(prefill_prep_kernel,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize, kPrepBytes);
  if (err == cudaSuccess)
    err = cudaFuncSetAttribute(prefill_scan_kernel<1>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                               Scan<1>::kBytes);
  if (err == cudaSuccess)
    err = cudaFuncSetAttribute(prefill_scan_kernel<2>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                               Scan<2>::kBytes);
  if (err != cudaSuccess) return err;
  Segment s = plan(d, a.lay.T);
  const long long slots = s.dense ? dense_slots(a.lay.T, d.B) : (long long)s.span * d.B;
  // One chain a CTA or two: the rounds of the SMs, as if the rows were T / N sequences of the
  // longest's length, times 3800 or 6300 cycles a chunk.  Sequences of one length take whole
  // rounds; others, the longest first, fill them up.  Measured, one and two, with 32 heads: 2 and
  // 3 sequences of 1000 tokens 101 and 88, 148 and 152 us, 16 of them 677 and 587; 16 of 17 to
  // 2048 496 and 421; 8 of 17 to 4096 243 and 282; 4 of 627 to 3354 441 and 402; with 16 heads 3
  // of 4 to 12220 468 and 711.
  const int sms = sm_count() > 0 ? sm_count() : 152;
  const float full = d.N > 0 ? fminf((float)a.lay.T / d.N, (float)d.B) : (float)d.B;
  auto rounds = [&](int slices) {
    const float x = full * d.Hv * slices / sms;
    return full >= 0.9f * d.B ? ceilf(x) : fmaxf(x, 1.f);
  };
  const bool two = 63.f * rounds(Scan<2>::kSlices) < 38.f * rounds(Scan<1>::kSlices);
  const long long scan = (long long)d.B * d.Hv * (two ? Scan<2>::kSlices : Scan<1>::kSlices);
  if (slots * d.Hv > 0x7fffffffll || scan > 0x7fffffffll) return cudaErrorInvalidConfiguration;
  // in more than a round of the SMs the long sequences go first, so that the SMs end closer
  // together (16 ragged prompts 492 to 463 us)
  s.by_length = scan > sms && d.B > 1 && d.B <= kMaxRanked;
  const WaitHooks hooks = wait_hooks();
  unsigned char* ws = static_cast<unsigned char*>(workspace);
  const int longest = (int)(((long long)d.N + kC - 1) / kC);
  // The second kernel starts beside the first one's last CTAs, unless the sequences are long.
  // Measured with 32 heads, so and one after the other: 512 tokens 38.0 and 41.4 us, 4 times
  // 512 105 and 109, 4096 200 and 203, but 16384 790 and 744, 32768 1566 and 1486: the chains
  // that start first then run slower to the end.  (Not with segments made ahead: the states
  // that it reads first are then the second kernel's of the segment before, which may run.)
  const int beside = longest > 0 && longest <= kAheadChunks && !s.ahead;
  for (s.c0 = 0; s.c0 == 0 || s.c0 < longest; s.c0 += s.span) {
    if (longest > 0) {
      cudaLaunchConfig_t cfg = {};
      cfg.gridDim = dim3((unsigned)(slots * d.Hv));
      cfg.blockDim = dim3(kPrepThreads);
      cfg.dynamicSmemBytes = kPrepBytes;
      cfg.stream = stream;
      cudaLaunchAttribute attr[1];
      attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
      attr[0].val.programmaticStreamSerializationAllowed = 1;
      cfg.attrs = attr;
      cfg.numAttrs = s.ahead && s.c0 > 0;
      err = cudaLaunchKernelEx(&cfg, prefill_prep_kernel, mapK, mapQ, a.log_alpha, a.beta, d, a.lay,
                               s, ws, a.dev_status, hooks);
      if (err != cudaSuccess || (err = cudaGetLastError()) != cudaSuccess) return err;
    }
    auto run = [&](auto kernel, int threads, uint32_t bytes) {
      cudaLaunchConfig_t cfg = {};
      cfg.gridDim = dim3((unsigned)scan);
      cfg.blockDim = dim3(threads);
      cfg.dynamicSmemBytes = bytes;
      cfg.stream = stream;
      cudaLaunchAttribute attr[1];
      attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
      attr[0].val.programmaticStreamSerializationAllowed = 1;
      cfg.attrs = attr;
      cfg.numAttrs = beside;
      const cudaError_t e = cudaLaunchKernelEx(
          &cfg, kernel, mapK, mapQ, mapV, static_cast<const __nv_bfloat16*>(a.v), a.pool_in,
          a.pool_out, static_cast<__nv_bfloat16*>(a.o), d, a.lay, s,
          static_cast<const unsigned char*>(ws), a.dev_status, hooks);
      return e != cudaSuccess ? e : cudaGetLastError();
    };
    err = two ? run(prefill_scan_kernel<2>, Scan<2>::kThreads, Scan<2>::kBytes)
              : run(prefill_scan_kernel<1>, Scan<1>::kThreads, Scan<1>::kBytes);
    if (err != cudaSuccess) return err;
    if (s.ahead)  // the halves by turns
      ws = static_cast<unsigned char*>(workspace) +
           (ws == workspace ? (size_t)slots * d.Hv * kSlotBytes : 0);
    if (s.span == 0) break;  // (no tokens at all: the states are copied)
  }
  return cudaSuccess;
}

}  // namespace gdn
