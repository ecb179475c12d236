// attend_tc.cu -- attention over a paged cache on the tensor cores (bf16, D <= 128):
// blocks of 256 query rows against 128 keys at a time, and the joining of parts.
//
// A unit is one key head, up to 256 query rows (two tiles of 128: row = node * G + g) and
// a range of key tiles; it computes, with the running maximum and sum of a softmax,
//     S = Q K^T,  P = exp2(c S - m),  l += sum P,  O += P V        (c = scale log2 e)
// and writes O / l, or, where the keys of the rows are cut into parts, the part's O / l
// and lse, which attend_join_kernel adds up:
//     lse = log sum_s e^{lse_s},   o = sum_s e^{lse_s - lse} o_s.
// Two kinds of units:
//   - a sequence's: the rows of one sequence against its own context and tree (and, where
//     a sequence has rows enough to fill the tiles, the shared prefix);
//   - the prefix's: 256 rows of the whole batch, whatever sequence they are of, against
//     the shared prefix, which is then read once for every 256 rows of the batch and not
//     once for every sequence.
// A unit of one row tile (kFork) lends the other's warps and columns to every second key tile.
//
// Roles (19 warps): warps 0-7 and 8-15 the softmax of row tile 0 and 1, two threads a row
// (one for keys 0-63 of a tile, one for 64-127); warp 16 brings K tiles, warp 17 V tiles;
// warp 18 issues the MMAs.  Tiles come by TMA, a box a page (a box a tile where pages are
// larger, and for the tree's own rows); pages that do not fit the tiles, and head sizes
// other than 64 and 128, come by 16-byte cp.async row by row.
// S and O are fp32 in TMEM; P goes back to TMEM as bf16 over the S it came from, each thread
// of a row its half in columns that only it reads, and is the A operand of P V.  Issue order
// P0 V, S0', P1 V, S1': one tile's MMAs (1030 cycles for D = 128) run while the other's
// softmax does.  That softmax, 1500 cycles, is what bounds a tile of keys (3000 cycles; one
// thread a row: 4100).  Making the next S in two halves around P V, so that half of the
// softmax starts sooner, was slower (4100: products of 64 keys cost more than they free).
// So was P in columns of its own beside S of 96 keys, which lets the next S come during the
// softmax: the 16 warps then share the issue slots (193 us for 32 trees of 128 nodes, against
// 166), although a unit of one row tile gained by it (112 to 94 us for 20 smaller trees).
//
// Measured: those 32 trees over 256 to 4096 rows and a prefix of 1024, 32 heads of 128: 159 us,
// 1.1 PFLOP/s; causal prompts of 4096 and 16384 rows 180 and 2373 us, 0.77 and 0.93 PFLOP/s.
//
// O is rescaled only when a row's maximum has grown by more than 2^8 over the one its
// sums use (exact either way: P and l stay far below the overflow of their types).
#include <string.h>

#include "common.cuh"
#include "kernels.h"
#include "sm100.cuh"

namespace gdn {
namespace {

using namespace sm100;

constexpr int kTile = 128;               // rows of a tile, keys of a tile
constexpr int kSoftmax = 512;             // softmax threads: two a row
constexpr int kThreads = kSoftmax + 3 * 32;
constexpr int kWarpK = kSoftmax / 32, kWarpV = kWarpK + 1, kWarpMma = kWarpK + 2;
constexpr int kHalf = kTile / 2;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kGrow = 8.f;             // log2 of the growth that is left in P

struct TcArgs {
  const __nv_bfloat16 *q, *k, *v;
  const int32_t *parent, *cu;
  const __nv_bfloat16 *k_cache, *v_cache;
  const int32_t *table, *ctx, *prefix_pages;
  float scale;
  __nv_bfloat16* o;
  float* lse;
  gdn_tree_attend_dims d;
  int32_t* dev_status;
  float* part_o;    // [slots][T * Hq][D] or null
  float* part_lse;  // [slots][T * Hq]
  int slot0;        // first slot of this launch's parts
  int splits;       // parts of a row's keys in this launch
  int tiles;        // 256-row blocks a sequence (a batch, for prefix units)
  bool prefix_units;   // units of the shared prefix over the whole batch
  bool with_prefix;    // a sequence's units include the prefix
  bool few;            // sequences of at most kAttendFewRows rows are attend_few.cu's
  int box_rows;        // rows of a TMA box of the cache (0: cache rows come by cp.async)
  bool own_box;        // the tree's own rows come by TMA
  bool q_box;          // Q too: G divides a tile, and the scale is not negative
  bool by_length;      // units of long contexts first (more units than SMs, kMaxRanked sequences at most)
  int rank0;           // then the first sequence of this launch, by length
  bool before_rest;    // a launch of the other sequences follows, and may start
  bool rest;           // this is that launch
};

constexpr uint32_t kBarBytes = 6144;

template <int DP>
struct Smem {
  static constexpr uint32_t kQ = kTile * DP * 2;   // one row tile
  static constexpr uint32_t kKV = kTile * DP * 2;  // one K or V tile
  static constexpr uint32_t OFF_Q = 0;
  static constexpr uint32_t OFF_K = OFF_Q + 2 * kQ;
  static constexpr uint32_t OFF_V = OFF_K + 2 * kKV;
  static constexpr uint32_t OFF_PARENT = OFF_V + 2 * kKV;
  static constexpr uint32_t OFF_BAR = OFF_PARENT + kMaxNLong * 4;
  static constexpr uint32_t kBytes = OFF_BAR + kBarBytes + 1024;  // + alignment slack
};

struct Bars {
  uint64_t kfull[2], kempty[2], vfull[2], vempty[2], sfull[2], pready[2], pvdone[2], lsum[2];
  uint64_t vraw, ready, qfull, drain;
  int4 unit;  // the sequence, its first row and the one after its last, its context
  uint32_t tmem;
  int abort;
  float top[2][2][kTile];  // a row's maximum over each half of a tile; at the end its sums
  float mref[2][kTile];     // at the end: what a row's sums are over
  int poison[2][2][kTile];  // whether the half saw values that are not finite
  uint32_t badv[2][4];  // own rows of a V tile that hold infinities or NaN (by stage)
};

__device__ __forceinline__ bool wait_bar(uint64_t* bar, uint32_t parity, Bars* s,
                                         uint64_t limit) {
  // (the clock is read once in a while: reading it takes longer than most of these waits)
  uint64_t t0 = 0;
  for (uint32_t tries = 0; !mbar_try_wait(bar, parity); ++tries) {
    if ((tries & 63u) != 63u) continue;
    if (ld_acquire_shared(&s->abort)) return false;
    const uint64_t now = globaltimer_ns();
    if (t0 == 0) t0 = now;
    if (now - t0 > limit) {
      st_release_shared(&s->abort, 1);
      return false;
    }
  }
  return true;
}

// the same for a whole warp: every lane gets the same answer
__device__ __forceinline__ bool wait_warp(uint64_t* bar, uint32_t parity, Bars* s,
                                          uint64_t limit) {
  return __all_sync(0xffffffffu, wait_bar(bar, parity, s, limit));
}

__device__ __forceinline__ void tmem_st_16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]),
      "r"(r[15])
      : "memory");
}

// starts loading 32 consecutive fp32 columns of this warp's 32 lanes; tmem_ld_wait before use
__device__ __forceinline__ void tmem_ld_start(uint32_t taddr, float (&v)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]),
        "=f"(v[7]), "=f"(v[8]), "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]),
        "=f"(v[14]), "=f"(v[15]), "=f"(v[16]), "=f"(v[17]), "=f"(v[18]), "=f"(v[19]),
        "=f"(v[20]), "=f"(v[21]), "=f"(v[22]), "=f"(v[23]), "=f"(v[24]), "=f"(v[25]),
        "=f"(v[26]), "=f"(v[27]), "=f"(v[28]), "=f"(v[29]), "=f"(v[30]), "=f"(v[31])
      : "r"(taddr));
}
// (the values pass through the wait, so that nothing uses them before it)
__device__ __forceinline__ void tmem_ld_wait(float (&v)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3]), "+f"(v[4]), "+f"(v[5]),
                 "+f"(v[6]), "+f"(v[7]), "+f"(v[8]), "+f"(v[9]), "+f"(v[10]), "+f"(v[11]),
                 "+f"(v[12]), "+f"(v[13]), "+f"(v[14])
               :: "memory");
  asm volatile(""
               : "+f"(v[15]), "+f"(v[16]), "+f"(v[17]), "+f"(v[18]), "+f"(v[19]), "+f"(v[20]),
                 "+f"(v[21]), "+f"(v[22]), "+f"(v[23]), "+f"(v[24]), "+f"(v[25]), "+f"(v[26]),
                 "+f"(v[27]), "+f"(v[28]), "+f"(v[29])
               :: "memory");
  asm volatile("" : "+f"(v[30]), "+f"(v[31])::"memory");
}

__device__ __forceinline__ void cp_async16_zfill(uint32_t dst, const void* src, bool take) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
               "r"(take ? 16u : 0u)
               : "memory");
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// (x, y) <- c (x, y) + b, and (s, t) += (x, y): two fp32 lanes an instruction
__device__ __forceinline__ void fma2(float& x, float& y, float c, float b) {
  asm("{\n\t.reg .b64 p, q, r;\n\t"
      "mov.b64 p, {%0, %1};\n\tmov.b64 q, {%2, %2};\n\tmov.b64 r, {%3, %3};\n\t"
      "fma.rn.f32x2 p, p, q, r;\n\tmov.b64 {%0, %1}, p;\n\t}"
      : "+f"(x), "+f"(y)
      : "f"(c), "f"(b));
}
__device__ __forceinline__ void add2(float& s, float& t, float x, float y) {
  asm("{\n\t.reg .b64 p, q;\n\t"
      "mov.b64 p, {%0, %1};\n\tmov.b64 q, {%2, %3};\n\t"
      "add.rn.f32x2 p, p, q;\n\tmov.b64 {%0, %1}, p;\n\t}"
      : "+f"(s), "+f"(t)
      : "f"(x), "f"(y));
}

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// One thread's 64 weights of a tile: exp2(c s - base) of 64 TMEM columns as bf16 pairs in
// pk, their fp32 sum, and the largest c s - base.  192 instructions where nothing is
// masked (the masked form, 64 selections more, is a branch of its own: folded into one by
// the compiler the selections would run for every tile).  bf16, because the product's other
// operand, V, is and the MMA takes one type: at most 2^-8 of a weight, 2^-8 sum_j p_j |v_j|
// of o.  A second part a weight would take that away for twice the products of P V and half
// as many stores again; o is rounded to bf16 anyhow.
template <bool kMasked>
__device__ __forceinline__ void weights(uint32_t tS, float c, float base, const uint32_t (&w)[2],
                                        float& top, float& total, uint32_t (&pk)[2][16]) {
  float x[2][32], mx[2] = {-INFINITY, -INFINITY}, sum[2] = {0.f, 0.f};
  tmem_ld_start(tS, x[0]);
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    tmem_ld_wait(x[e]);
    if (e == 0) tmem_ld_start(tS + 32, x[1]);  // (comes while the first half is worked on)
#pragma unroll
    for (int j = 0; j < 32; j += 2) fma2(x[e][j], x[e][j + 1], c, -base);
    if (kMasked) {
#pragma unroll
      for (int j = 0; j < 32; ++j) x[e][j] = (w[e] >> j) & 1u ? x[e][j] : -INFINITY;
    }
#pragma unroll
    for (int j = 0; j < 32; j += 4) {
      mx[0] = fmaxf(mx[0], fmaxf(x[e][j], x[e][j + 1]));
      mx[1] = fmaxf(mx[1], fmaxf(x[e][j + 2], x[e][j + 3]));
    }
#pragma unroll
    for (int j = 0; j < 32; j += 2) {
      x[e][j] = ex2(x[e][j]);
      x[e][j + 1] = ex2(x[e][j + 1]);
      add2(sum[0], sum[1], x[e][j], x[e][j + 1]);
      pk[e][j / 2] = pack_bf16(x[e][j], x[e][j + 1]);
    }
  }
  top = fmaxf(mx[0], mx[1]);
  total = sum[0] + sum[1];
}

// the largest c s of 64 TMEM columns
template <bool kMasked>
__device__ __forceinline__ float largest(uint32_t tS, float c, const uint32_t (&w)[2]) {
  float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    float x[32];
    tmem_ld_32cols(tS + 32 * e, x);
#pragma unroll
    for (int j = 0; j < 32; ++j)
      if (!kMasked || ((w[e] >> j) & 1u)) mx[j & 1] = fmaxf(mx[j & 1], c * x[j]);
  }
  return fmaxf(mx[0], mx[1]);
}

// bits of a packed pair of bf16 that are infinities or NaN
__device__ __forceinline__ bool nonfinite2(uint32_t x) {
  return (x & 0x7f80u) == 0x7f80u || (x & 0x7f800000u) == 0x7f800000u;
}
__device__ __forceinline__ uint32_t finite2(uint32_t x) {
  if ((x & 0x7f80u) == 0x7f80u) x &= 0xffff0000u;
  if ((x & 0x7f800000u) == 0x7f800000u) x &= 0x0000ffffu;
  return x;
}

static_assert(sizeof(Bars) <= kBarBytes, "the barriers fit their place");

// The sequence that comes `want`-th when the longest contexts come first (ties in order), and
// its rows and length.  Long units first, the SMs end closer together.
__device__ __forceinline__ int ranked(const int32_t* ctx, const int32_t* cu, int B, int want,
                                      int lane, int& first, int& stop, int& len) {
  const bool on0 = lane < B, on1 = lane + 32 < B;
  const int f0 = on0 ? cu[lane] : 0, e0 = on0 ? cu[lane + 1] : 0;
  const int f1 = on1 ? cu[lane + 32] : 0, e1 = on1 ? cu[lane + 33] : 0;
  const int x0 = on0 ? ctx[lane] : kNoRank, x1 = on1 ? ctx[lane + 32] : kNoRank;
  const int at = nth_largest(x0, x1, B, want, lane), l = at & 31;
  first = __shfl_sync(0xffffffffu, at < 32 ? f0 : f1, l);
  stop = __shfl_sync(0xffffffffu, at < 32 ? e0 : e1, l);
  len = __shfl_sync(0xffffffffu, at < 32 ? x0 : x1, l);
  return at;
}

enum Segment { kPrefix = 0, kContext = 1, kOwn = 2 };

// a page number out of range: the sequence's error, every sequence's for the prefix
__device__ __noinline__ void report_page(const TcArgs& a, bool prefix, int b) {
  if (!a.dev_status) return;
  if (!prefix) atomicMax(a.dev_status + b, GDN_TREE_STATUS_BAD_LAYOUT);
  else
    for (int i = 0; i < a.d.B; ++i) atomicMax(a.dev_status + i, GDN_TREE_STATUS_BAD_LAYOUT);
}

// adds the infinities and NaN of the values on a row's path to columns [c0, c1) of its
// result (they were kept out of the product, which masks by zero weights)
__device__ __noinline__ void add_nonfinite(const TcArgs& a, size_t out, size_t slot, int first,
                                           int node, int hk, int c0, int c1) {
  for (int col = c0; col < min(c1, a.d.D); ++col) {
    float x = 0.f;
    for (int nd = node, up; nd >= 0; nd = up) {
      up = a.parent ? a.parent[first + nd] : nd - 1;
      if (up >= nd) up = -1;  // (a bad tree, reported)
      const float v = __bfloat162float(a.v[((size_t)(first + nd) * a.d.Hkv + hk) * a.d.D + col]);
      if (!isfinite(v)) x += v;
    }
    if (isfinite(x)) continue;
    if (a.part_o) a.part_o[slot * a.d.D + col] += x;
    else a.o[out * a.d.D + col] = __float2bfloat16_rn(__bfloat162float(a.o[out * a.d.D + col]) + x);
  }
}

// After a wait that ran out: the tiles still on their way arrive (or these bounded waits end)
// before the CTA, and with it the place that they are written to, goes.  Both phases of each
// barrier, as the one that is open is not known.  All threads come here.
__device__ __noinline__ void await_tiles(Bars* S, int warp) {
  constexpr uint64_t kArrivalNs = 1000000;
  for (uint32_t ph = 0; ph < 2; ++ph) {
    for (int s = 0; s < 2; ++s)
      if (warp == kWarpK) mbar_wait(&S->kfull[s], ph, kArrivalNs);
      else if (warp == kWarpV) mbar_wait(&S->vfull[s], ph, kArrivalNs);
    if (warp == kWarpV) mbar_wait(&S->vraw, ph, kArrivalNs);
    if (warp == kWarpMma) mbar_wait(&S->qfull, ph, kArrivalNs);
  }
  __syncthreads();
}

template <int DP, bool kFork>
__global__ void __launch_bounds__(kThreads, 1)
attend_tc_kernel(TcArgs a, const __grid_constant__ CUtensorMap mapK,
                 const __grid_constant__ CUtensorMap mapV,
                 const __grid_constant__ CUtensorMap mapKo,
                 const __grid_constant__ CUtensorMap mapVo,
                 const __grid_constant__ CUtensorMap mapQ, WaitHooks hooks) {
  using L = Smem<DP>;
  const uint64_t limit_ns = hooks.limit_ns;
  extern __shared__ unsigned char smem_raw[];
  unsigned char* smem = reinterpret_cast<unsigned char*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  Bars* S = reinterpret_cast<Bars*>(smem + L::OFF_BAR);
  int32_t* sParent = reinterpret_cast<int32_t*>(smem + L::OFF_PARENT);
  const gdn_tree_attend_dims& d = a.d;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int G = d.Hq / d.Hkv;

  // ---- the unit: rows [r0, r1) of key head hk, key tiles [i0, i1) -------------------
  const int split = blockIdx.x % a.splits;
  int u = blockIdx.x / a.splits;
  const int hk = u % d.Hkv;
  u /= d.Hkv;
  const int t = a.tiles - 1 - u % a.tiles;  // (a chain's last rows see the most keys)
  // the sequence is found by one warp while others set up
  if (warp == 0 && !a.prefix_units) {
    int b = u / a.tiles, first, stop, ctx;
    if (a.by_length) {
      b = ranked(a.ctx, a.cu, d.B, a.rank0 + b, lane, first, stop, ctx);
    } else {
      stop = a.cu[b + 1];
      first = a.cu[b];
      ctx = a.ctx[b];
    }
    if (lane == 0) S->unit = make_int4(b, first, stop, ctx);
  }
  if (tid == 32) {
    if (a.prefix_units) S->unit = make_int4(0, 0, 0, 0);
    for (int s = 0; s < 2; ++s) {
      mbar_init(&S->kfull[s], 1);
      mbar_init(&S->kempty[s], 1);
      mbar_init(&S->vfull[s], 1);
      mbar_init(&S->vempty[s], 1);
      mbar_init(&S->sfull[s], 1);
      mbar_init(&S->pready[s], kSoftmax / 64);  // (warps)
      mbar_init(&S->pvdone[s], 1);
      mbar_init(&S->lsum[s], kSoftmax / 64);
    }
    mbar_init(&S->vraw, 1);
    mbar_init(&S->qfull, 1);
    mbar_init(&S->ready, kSoftmax / 32);  // Q and the tree are in shared memory
    mbar_init(&S->drain, 1);
    S->abort = 0;
    mbar_fence_init();
  }
  if (warp == kWarpMma) tmem_alloc(&S->tmem, 512);
  // (attend_few.cu may start; it waits for this kernel's end before it reads its parts.  So may
  // the launch of the rest, one CTA of which waits for this one's end before its own)
  if (a.prefix_units || a.before_rest) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = S->tmem;
  constexpr uint32_t kStage = L::kKV;
  const int b = S->unit.x, first = S->unit.y, stop = S->unit.z, n = stop - first, ctx = S->unit.w;
  bool mine = true;  // the unit has rows, and they are this kernel's
  if (!a.prefix_units) {
    const long long cap = (long long)d.table_width * d.page_size;
    // (stop < first, not n < 0: of two numbers far apart the difference may wrap)
    if (first < 0 || stop < first || stop > d.T || n > d.N || ctx < 0 || ctx > cap) {
      if (a.dev_status && tid == 0) atomicMax(a.dev_status + b, GDN_TREE_STATUS_BAD_LAYOUT);
      mine = false;
    } else {
      mine = !a.few || n * G > kAttendFewRows;  // (else attend_few.cu's)
    }
  }
  constexpr int kUnitRows = kFork ? kTile : 2 * kTile;
  // (units past the sequence's rows, whose row numbers may be past 32 bits)
  const long long unit0 = (long long)t * kUnitRows;
  if (!mine || unit0 >= (long long)(a.prefix_units ? d.T : n) * G) {
    if (warp == kWarpMma) tmem_dealloc(tmem, 512);
    if (a.rest && blockIdx.x == 0) asm volatile("griddepcontrol.wait;" ::: "memory");
    return;
  }
  const int rows_end = a.prefix_units ? d.T * G : (first + n) * G;
  const int r0 = first * G + (int)unit0;
  const int rows = min(kUnitRows, rows_end - r0);
  const bool two = !kFork && rows > kTile;
  const bool own = a.k != nullptr && !a.prefix_units;
  const bool tree = own && a.parent != nullptr;
  const int plen = a.prefix_units || a.with_prefix ? d.prefix_len : 0;
  const int nP = (plen + kTile - 1) / kTile, nC = (ctx + kTile - 1) / kTile;
  // own keys past the last row's node are seen by none of these rows
  const int seen = own ? (r0 + rows - 1) / G - first + 1 : 0;
  const int nO = (seen + kTile - 1) / kTile;
  const int all = nP + nC + nO;
  const int i0 = (int)((long long)all * split / a.splits);
  const int i1 = (int)((long long)all * (split + 1) / a.splits);
  const int ntiles = i1 - i0;
  // rows for one tile only: the two groups of softmax warps take its key tiles by turns, with
  // sums of their own (S and O of row tile 1), which are added up at the end
  const bool fork = kFork && ntiles > 1;
  // key tile i: its segment, first key and keys (own tiles from the last to the first, so
  // that a row follows its path upwards once)
  auto tile_of = [&](int i, int& seg, int& j0, int& len) {
    if (i < nP) { seg = kPrefix; j0 = i * kTile; len = plen; }
    else if (i < nP + nC) { seg = kContext; j0 = (i - nP) * kTile; len = ctx; }
    else { seg = kOwn; j0 = (all - 1 - i) * kTile; len = seen; }
  };

  if (warp == kWarpK || warp == kWarpV) {
    // ---- producers: K or V --------------------------------------------------------------
    const bool isV = warp == kWarpV;
    uint64_t* full = isV ? S->vfull : S->kfull;
    uint64_t* empty = isV ? S->vempty : S->kempty;
    unsigned char* stage0 = smem + (isV ? L::OFF_V : L::OFF_K);
    constexpr int kChunks = DP / 8;             // 16-byte chunks a row
    constexpr int kRowsAtOnce = 32 / kChunks;   // rows a warp instruction covers
    const int c8 = lane % kChunks;
    const bool in_row = 8 * c8 < d.D;
    uint32_t raw_phase = 0;
    auto row_of = [&](int seg, int j) -> int {  // key j's row in the cache, -1: a bad page
      const int pi = j / d.page_size;
      const int pg = seg == kPrefix ? a.prefix_pages[pi] : a.table[(size_t)b * d.table_width + pi];
      if (pg >= 0 && pg < d.n_pages) return pg * d.page_size + (j - pi * d.page_size);
      report_page(a, seg == kPrefix, b);
      return -1;
    };
    for (int i = i0; i < i1; ++i) {
      const int at = i - i0, st = at & 1;
      int seg, j0, len;
      tile_of(i, seg, j0, len);
      const int valid = min(len - j0, kTile);
      unsigned char* stage = stage0 + st * kStage;
      // V rows that are masked for every row (past a length) or for some (the tree's) must
      // not meet a zero weight with an infinity or a NaN: they pass through this warp
      const bool fix = isV && (seg == kOwn || valid < kTile);
      if (seg == kOwn ? a.own_box : a.box_rows != 0) {
        const int box = seg == kOwn ? kTile : a.box_rows;
        const int boxes = (valid + box - 1) / box;
        int crow = 0;
        if (lane < boxes) {
          crow = seg == kOwn ? first + j0 : row_of(seg, j0 + lane * box);
          if (crow < 0) crow = d.n_pages * d.page_size;  // (past the last row: reads zeros)
        }
        if (at >= 2 && !wait_warp(&empty[st], ((at >> 1) & 1) ^ 1, S, limit_ns)) break;
        uint64_t* bar = fix ? &S->vraw : &full[st];
        if (lane == 0) mbar_arrive_expect_tx(bar, (uint32_t)(boxes * box * DP * 2));
        __syncwarp();
        if (lane < boxes) {
          const CUtensorMap* map = seg == kOwn ? (isV ? &mapVo : &mapKo) : (isV ? &mapV : &mapK);
#pragma unroll
          for (int c = 0; c < DP / 64; ++c)
            tma_load_3d(stage + c * kSw128TileBytes + lane * box * 128, map, bar, 64 * c, hk, crow);
        }
        __syncwarp();
        if (!fix) continue;
        if (!wait_warp(&S->vraw, raw_phase, S, limit_ns)) break;
        raw_phase ^= 1u;
      } else {
        // lane l looks up rows l, 32 + l, 64 + l, 96 + l of the tile
        int row[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int j = 32 * e + lane;
          row[e] = j >= valid ? -1 : seg == kOwn ? first + j0 + j : row_of(seg, j0 + j);
        }
        if (at >= 2 && !wait_warp(&empty[st], ((at >> 1) & 1) ^ 1, S, limit_ns)) break;
        const __nv_bfloat16* src = (seg == kOwn ? (isV ? a.v : a.k) : (isV ? a.v_cache : a.k_cache)) +
                                   (size_t)hk * d.D + 8 * c8;
        const size_t stride = (size_t)d.Hkv * d.D;
        const uint32_t dst = smem_addr(stage);
#pragma unroll
        for (int e = 0; e < 4; ++e)
#pragma unroll 8
          for (int rr = 0; rr < 32; rr += kRowsAtOnce) {
            const int r = rr + lane / kChunks;
            const int x = __shfl_sync(0xffffffffu, row[e], r);
            const bool take = x >= 0 && in_row;
            cp_async16_zfill(dst + sw128_chunk(32 * e + r, c8), take ? src + x * stride : src, take);
          }
        asm volatile("cp.async.wait_all;" ::: "memory");
      }
      if (fix) {
        for (int key = valid + lane / kChunks; key < kTile; key += kRowsAtOnce)
          *reinterpret_cast<uint4*>(stage + sw128_chunk(key, c8)) = make_uint4(0, 0, 0, 0);
        if (seg == kOwn) {
          // what is not finite is kept out of the product and added to the rows that see
          // it at the end; a multiple of zero tells whether there is any
          if (lane < 4) S->badv[st][lane] = 0u;
          __syncwarp();
          const __nv_bfloat162 zero = __floats2bfloat162_rn(0.f, 0.f);
          __nv_bfloat162 acc[4] = {zero, zero, zero, zero};
#pragma unroll 8
          for (int key = lane / kChunks; key < valid; key += kRowsAtOnce) {
            const uint4 w = *reinterpret_cast<const uint4*>(stage + sw128_chunk(key, c8));
            acc[0] = __hfma2(reinterpret_cast<const __nv_bfloat162&>(w.x), zero, acc[0]);
            acc[1] = __hfma2(reinterpret_cast<const __nv_bfloat162&>(w.y), zero, acc[1]);
            acc[2] = __hfma2(reinterpret_cast<const __nv_bfloat162&>(w.z), zero, acc[2]);
            acc[3] = __hfma2(reinterpret_cast<const __nv_bfloat162&>(w.w), zero, acc[3]);
          }
          const float2 t0 = __bfloat1622float2(__hadd2(__hadd2(acc[0], acc[1]), __hadd2(acc[2], acc[3])));
          if (__any_sync(0xffffffffu, isnan(t0.x + t0.y))) {
            for (int key = lane / kChunks; key < valid; key += kRowsAtOnce) {
              uint4* at16 = reinterpret_cast<uint4*>(stage + sw128_chunk(key, c8));
              const uint4 w = *at16;
              if (nonfinite2(w.x) || nonfinite2(w.y) || nonfinite2(w.z) || nonfinite2(w.w)) {
                atomicOr(&S->badv[st][key >> 5], 1u << (key & 31));
                *at16 = make_uint4(finite2(w.x), finite2(w.y), finite2(w.z), finite2(w.w));
              }
            }
          }
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&full[st]);
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
  } else if (warp == kWarpMma) {
    // ---- MMAs: the warp waits together, one lane issues ---------------------------------
    if (ntiles > 0) {
      if (a.q_box && elect_one()) {  // (rows past the unit's are somebody's, and not used)
        mbar_arrive_expect_tx(&S->qfull, (two ? 2 : 1) * L::kQ);
        for (int x = 0; x < (two ? 2 : 1); ++x)
#pragma unroll
          for (int c = 0; c < DP / 64; ++c)
            tma_load_3d(smem + L::OFF_Q + x * L::kQ + c * kSw128TileBytes, &mapQ, &S->qfull, 64 * c,
                        hk * G, (r0 + x * kTile) / G);
      }
      __syncwarp();
      constexpr uint32_t idS = idesc_bf16_f32(kTile, kTile);
      constexpr uint32_t idO = idesc_bf16_f32_bmn(kTile, DP);
      const uint64_t dQ = desc_sw128_kmajor(smem_addr(smem + L::OFF_Q));
      const uint64_t dK = desc_sw128_kmajor(smem_addr(smem + L::OFF_K));
      // (V: keys are K rows, D contiguous; 8-key groups 1 KB apart, 64-column blocks 16 KB)
      const uint64_t dV = desc_sw128_mnmajor(smem_addr(smem + L::OFF_V), kSw128TileBytes, 1024);
      auto issue_s = [&](int tile, int st, bool last_of_k) {
        if (elect_one()) {
          const uint32_t to = tmem + tile * kTile;
          const uint64_t q = dQ + (fork ? 0 : tile) * (L::kQ >> 4), k = dK + st * (kStage >> 4);
#pragma unroll
          for (int s = 0; s < DP / 16; ++s) {
            const uint32_t off = ((s >> 2) * kSw128TileBytes + (s & 3) * 32) >> 4;
            if (s == 0) umma_ss<false>(to, q + off, k + off, idS);
            else umma_ss<true>(to, q + off, k + off, idS);
          }
          umma_commit(&S->sfull[tile]);
          if (last_of_k) umma_commit(&S->kempty[st]);
        }
        __syncwarp();
      };
      auto issue_pv = [&](int tile, int st, bool first_tile, bool last_of_v) {
        if (elect_one()) {
          const uint32_t to = tmem + 2 * kTile + tile * kTile, p = tmem + tile * kTile;
          const uint64_t v = dV + st * (kStage >> 4);
          if (first_tile) umma_ts<false>(to, p, v, idO);
          else umma_ts<true>(to, p, v, idO);
#pragma unroll
          for (int s = 1; s < kTile / 16; ++s)
            umma_ts<true>(to, p + (s >> 2) * kHalf + 8 * (s & 3), v + ((s * 2048) >> 4), idO);
          umma_commit(&S->pvdone[tile]);
          if (last_of_v) umma_commit(&S->vempty[st]);
        }
        __syncwarp();
      };
      bool ok = wait_warp(a.q_box ? &S->qfull : &S->ready, 0, S, limit_ns) &&
                wait_warp(&S->kfull[0], 0, S, limit_ns);
      if (ok) {
        issue_s(0, 0, !two);
        if (two) issue_s(1, 0, true);
      }
      // (both tiles written out: a loop over them takes the descriptors out of the uniform
      // registers, and 8 % longer)
      if (fork) {
        ok = ok && wait_warp(&S->kfull[1], 0, S, limit_ns);
        if (ok) issue_s(1, 1, true);
        // (key tiles at and at + 1, written out as well)
        for (int at = 0; ok && at < ntiles; at += 2) {
          const uint32_t ph = (at >> 1) & 1;
          ok = wait_warp(&S->vfull[0], ph, S, limit_ns) && wait_warp(&S->pready[0], ph, S, limit_ns);
          if (!ok) break;
          tc_fence_after_sync();
          issue_pv(0, 0, at == 0, true);
          if (at + 2 < ntiles) {
            ok = wait_warp(&S->kfull[0], ph ^ 1, S, limit_ns);
            if (!ok) break;
            issue_s(0, 0, true);
          }
          if (at + 1 < ntiles) {
            ok = wait_warp(&S->vfull[1], ph, S, limit_ns) && wait_warp(&S->pready[1], ph, S, limit_ns);
            if (!ok) break;
            tc_fence_after_sync();
            issue_pv(1, 1, at == 0, true);
          }
          if (at + 3 < ntiles) {
            ok = wait_warp(&S->kfull[1], ph ^ 1, S, limit_ns);
            if (!ok) break;
            issue_s(1, 1, true);
          }
        }
      }
      for (int at = 0; !fork && ok && at < ntiles; ++at) {
        const int st = at & 1, nx = (at + 1) & 1;
        const bool more = at + 1 < ntiles;
        ok = wait_warp(&S->vfull[st], (at >> 1) & 1, S, limit_ns) &&
             wait_warp(&S->pready[0], at & 1, S, limit_ns);
        if (!ok) break;
        tc_fence_after_sync();
        issue_pv(0, st, at == 0, !two);
        if (more) {
          ok = wait_warp(&S->kfull[nx], ((at + 1) >> 1) & 1, S, limit_ns);
          if (!ok) break;
          issue_s(0, nx, !two);
        }
        if (two) {
          ok = wait_warp(&S->pready[1], at & 1, S, limit_ns);
          if (!ok) break;
          tc_fence_after_sync();
          issue_pv(1, st, at == 0, true);
          if (more) issue_s(1, nx, true);
        }
      }
      // whatever was issued is done before TMEM and the operands go
      if (elect_one()) umma_commit(&S->drain);
      __syncwarp();
      mbar_wait(&S->drain, 0, limit_ns);
    }
    __syncwarp();
  } else {
    // Q, negated where the scale is negative (the maximum is then taken with c >= 0), and
    // the tree (a parent that is not earlier is an error; taken as a root meanwhile)
    const uint32_t flip = a.scale < 0.f ? 0x80008000u : 0u;
#pragma unroll 4
    for (int e = tid; !a.q_box && e < 2 * kTile * (DP / 8); e += kSoftmax) {
      const int r = e / (DP / 8), c8 = e % (DP / 8);
      uint4 x = make_uint4(0, 0, 0, 0);
      if (r < rows && 8 * c8 < d.D) {
        const int rho = r0 + r, tok = rho / G, g = rho - tok * G;
        x = *reinterpret_cast<const uint4*>(a.q + ((size_t)tok * d.Hq + hk * G + g) * d.D + 8 * c8);
        x.x ^= flip; x.y ^= flip; x.z ^= flip; x.w ^= flip;
      }
      *reinterpret_cast<uint4*>(smem + L::OFF_Q + (r / kTile) * L::kQ + sw128_chunk(r % kTile, c8)) = x;
    }
    if (tree)
      for (int i = tid; i < n; i += kSoftmax) {
        const int p = a.parent[first + i];
        const bool bad = p < -1 || p >= i;
        sParent[i] = bad ? -1 : p;
        if (bad && a.dev_status) atomicMax(a.dev_status + b, GDN_TREE_STATUS_BAD_TREE);
      }
    fence_proxy_async_smem();
    __syncwarp();
    if (!(b * d.Hkv + hk == hooks.withhold_unit && warp == hooks.withhold_node))
      mbar_arrive_warp(&S->ready);
    bool ok = wait_warp(&S->ready, 0, S, limit_ns);
    // ---- softmax: two threads a row --------------------------------------------------------
    const int tile = warp >> 3, half = (warp >> 2) & 1, lr = (warp & 3) * 32 + lane;
    const int r = fork ? lr : tile * kTile + lr;
    const uint32_t tl = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const uint32_t tS = tl + tile * kTile + kHalf * half, tO = tl + 2 * kTile + tile * kTile;
    // The two warps of a row, w and w + 4, meet at a named barrier (an mbarrier, with its
    // limit on waiting, made a tile of keys 13 % longer).  It cannot be left waiting: a warp
    // whose wait runs out goes on through all tiles, with every wait at once given up, and
    // writes nothing.
    const int pair = 1 + tile * 4 + (warp & 3);
    auto meet = [&]() { asm volatile("bar.sync %0, 64;" ::"r"(pair) : "memory"); };
    const float c = fabsf(a.scale) * kLog2e;
    const int rho = min(r0 + r, rows_end - 1), tok = rho / G, node = tok - first;
    const bool live = r < rows;
    int walk = node;                   // the next node of the path that is not yet masked
    float mref = -INFINITY, l = 0.f;   // of c s; l: this half's
    bool poison = false;
    if (tile == 0 || two || fork) {
      const int step = fork ? 2 : 1;
      const int mine_of = fork ? (ntiles + 1 - tile) >> 1 : ntiles;  // this group's key tiles
      for (int at = 0; at < mine_of; ++at) {
        const int i = i0 + (fork ? tile : 0) + step * at;
        int seg, j0, len;
        tile_of(i, seg, j0, len);
        ok = wait_warp(&S->sfull[tile], at & 1, S, limit_ns) && ok;
        tc_fence_after_sync();
        const int valid = len - j0;
        const bool masked = seg == kOwn || valid < kTile;
        uint32_t w[2];  // the keys of this half of the tile that the row sees, a bit a key
        if (masked) {
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int left = (seg == kOwn && !tree ? min(valid, node - j0 + 1) : valid) -
                             kHalf * half - 32 * e;
            w[e] = left >= 32 ? 0xffffffffu : left <= 0 ? 0u : (1u << left) - 1u;
          }
          if (seg == kOwn && tree) {
            uint64_t on = 0;
            // (a part that begins below the row's node first walks up to its own tiles)
            while (walk >= j0 + kTile) walk = sParent[walk];
            for (; walk >= j0; walk = sParent[walk]) {
              const int off = walk - j0 - kHalf * half;
              if (off >= 0 && off < kHalf) on |= 1ull << off;
            }
            w[0] &= (uint32_t)on;
            w[1] &= (uint32_t)(on >> 32);
          }
          __syncwarp();
        }
        if (at == 0) {  // the first tile's own maximum, so that its weights are made once
          const float mine = masked ? largest<true>(tS, c, w) : largest<false>(tS, c, w);
          S->top[tile][half][lr] = mine;
          meet();
          mref = fmaxf(mine, S->top[tile][half ^ 1][lr]);
          meet();
        }
        uint32_t pk[2][16];
        float sum;
        // the weights for the maximum that the sums use; where the row's own maximum turns
        // out to have grown by too much, O and l are rescaled and the weights made again
        for (bool again = false;; again = true) {
          const float base = mref == -INFINITY ? 0.f : mref;
          float mine;
          if (masked) weights<true>(tS, c, base, w, mine, sum, pk);
          else weights<false>(tS, c, base, w, mine, sum, pk);
          if (again) break;
          // the row's maximum, over base: the other half's beside this one's
          // (NaN scores: fmaxf drops them here; their weights and sums are NaN)
          S->top[tile][half][lr] = mine;
          meet();
          const float top = fmaxf(mine, S->top[tile][half ^ 1][lr]);
          const bool grow = top > (mref == -INFINITY ? -INFINITY : kGrow);
          if (!__any_sync(0xffffffffu, grow)) break;
          const float to = grow ? base + top : mref;
          const float keep = grow ? (mref == -INFINITY ? 0.f : ex2(-top)) : 1.f;
          if (at > 0) {
            // O of the tiles before is complete once their last product is
            ok = wait_warp(&S->pvdone[tile], (at - 1) & 1, S, limit_ns) && ok;
            tc_fence_after_sync();
#pragma unroll 1
            for (int e = 0; e < DP / 32; ++e) {  // this half's columns of O, 16 at a time
              float y[16];
              uint32_t z[16];
              const uint32_t at16 = tO + DP / 2 * half + 16 * e;
              tmem_ld_16cols(at16, y);
#pragma unroll
              for (int j = 0; j < 16; ++j) z[j] = __float_as_uint(y[j] * keep);
              tmem_st_16(at16, z);
            }
            asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
          }
          l *= keep;
          mref = to;
        }
        tmem_st_16(tS, pk[0]);
        tmem_st_16(tS + 16, pk[1]);
        l += sum;
        if (seg == kOwn) {
          // (the V tile is read behind its barrier: its bits are written by then)
          const int st = (i - i0) & 1;
          ok = wait_warp(&S->vfull[st], ((i - i0) >> 1) & 1, S, limit_ns) && ok;
#pragma unroll
          for (int e = 0; e < 2; ++e) poison |= (w[e] & S->badv[st][2 * half + e]) != 0u;
        }
        asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
        tc_fence_before_sync();
        mbar_arrive_warp(&S->pready[tile]);
      }
      if (ok && ntiles > 0) {
        ok = wait_warp(&S->pvdone[tile], (mine_of - 1) & 1, S, limit_ns);
        tc_fence_after_sync();
      }
      // the row's sum: both halves'
      S->top[tile][half][lr] = l;
      S->poison[tile][half][lr] = poison;
      if (half == 0) S->mref[tile][lr] = mref;
      mbar_arrive_warp(&S->lsum[tile]);
      ok = wait_warp(&S->lsum[tile], 0, S, limit_ns) && ok;
      l = S->top[tile][0][lr] + S->top[tile][1][lr];
      // both groups' sums, over the larger maximum: weights f of O and f2 of the other group's
      float f = 1.f, f2 = 0.f;
      if (fork) {
        ok = wait_warp(&S->lsum[tile ^ 1], 0, S, limit_ns) && ok;
        // (its last product as well)
        ok = wait_warp(&S->pvdone[tile ^ 1], (((ntiles + tile) >> 1) - 1) & 1, S, limit_ns) && ok;
        tc_fence_after_sync();
        const float m2 = S->mref[tile ^ 1][lr], top = fmaxf(mref, m2);
        f = mref == -INFINITY ? 0.f : ex2(mref - top);
        f2 = m2 == -INFINITY ? 0.f : ex2(m2 - top);
        l = f * l + f2 * (S->top[tile ^ 1][0][lr] + S->top[tile ^ 1][1][lr]);
        mref = top;
      }
      const float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);  // (l NaN: kept)
      const int out = tok * d.Hq + hk * G + (rho - tok * G);
      const size_t slot0 = (size_t)(a.slot0 + split) * d.T * d.Hq, slot = slot0 + out;
      if (ok) {
        // 32 columns of a warp's 32 rows at a time through shared memory (Q and the first K
        // tiles, which every product has read by now), so that a store covers whole pieces
        // of rows; a lane a row would touch 32 lines an instruction
        unsigned char* stage = smem + L::OFF_Q + warp * 4096;
        const int row0 = (fork ? 0 : tile * kTile) + 32 * (warp & 3);  // the warp's first row of the unit
        const int e0 = fork ? tile : 0, e1 = fork ? min(tile + 1, DP / 64) : DP / 64;
#pragma unroll 1
        for (int e = e0; e < e1; ++e) {
          const int col = DP / 2 * half + 32 * e;
          float y[32];
          if (fork) {
            float z[32];
            tmem_ld_32cols(tO + col, y);
            tmem_ld_32cols(tl + 2 * kTile + (tile ^ 1) * kTile + col, z);
#pragma unroll
            for (int j = 0; j < 32; ++j) y[j] = fmaf(f, y[j], f2 * z[j]);
          } else if (ntiles > 0) {
            tmem_ld_32cols(tO + col, y);
          } else {
#pragma unroll
            for (int j = 0; j < 32; ++j) y[j] = 0.f;
          }
#pragma unroll
          for (int j = 0; j < 32; ++j) y[j] *= inv;
          if (a.part_o) {
#pragma unroll
            for (int j = 0; j < 8; ++j)
              *reinterpret_cast<float4*>(stage + lane * 128 + ((j ^ (lane & 7)) << 4)) =
                  make_float4(y[4 * j], y[4 * j + 1], y[4 * j + 2], y[4 * j + 3]);
            __syncwarp();
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const int rr = 4 * i + (lane >> 3), j = lane & 7;
              const int to = __shfl_sync(0xffffffffu, out, rr);
              if (row0 + rr < rows && col + 4 * j < d.D)
                *reinterpret_cast<float4*>(a.part_o + (slot0 + to) * d.D + col + 4 * j) =
                    *reinterpret_cast<const float4*>(stage + rr * 128 + ((j ^ (rr & 7)) << 4));
            }
          } else {
#pragma unroll
            for (int j = 0; j < 4; ++j)
              *reinterpret_cast<uint4*>(stage + lane * 64 + ((j ^ ((lane >> 1) & 3)) << 4)) =
                  make_uint4(pack_bf16(y[8 * j], y[8 * j + 1]), pack_bf16(y[8 * j + 2], y[8 * j + 3]),
                             pack_bf16(y[8 * j + 4], y[8 * j + 5]), pack_bf16(y[8 * j + 6], y[8 * j + 7]));
            __syncwarp();
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int rr = 8 * i + (lane >> 2), j = lane & 3;
              const int to = __shfl_sync(0xffffffffu, out, rr);
              if (row0 + rr < rows && col + 8 * j < d.D)
                *reinterpret_cast<uint4*>(a.o + (size_t)to * d.D + col + 8 * j) =
                    *reinterpret_cast<const uint4*>(stage + rr * 64 + ((j ^ ((rr >> 1) & 3)) << 4));
            }
          }
          __syncwarp();
        }
        // (either half may have seen them)
        int bad = S->poison[tile][0][lr] | S->poison[tile][1][lr];
        if (fork) bad |= S->poison[tile ^ 1][0][lr] | S->poison[tile ^ 1][1][lr];
        if (bad != 0 && live && e0 < e1)
          add_nonfinite(a, out, slot, first, node, hk, DP / 2 * half + 32 * e0, DP / 2 * half + 32 * e1);
        if (live && half == 0 && (tile == 0 || !fork)) {
          const float z = l == 0.f ? -INFINITY : (mref + log2f(l)) * kLn2;
          if (a.part_o) a.part_lse[slot] = z;
          else if (a.lse) a.lse[out] = z;
        }
      }
    }
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  if (S->abort) await_tiles(S, warp);
  if (warp == kWarpMma) tmem_dealloc(tmem, 512);
  if (a.rest && blockIdx.x == 0) asm volatile("griddepcontrol.wait;" ::: "memory");
  if (tid == 0 && S->abort && a.dev_status) {
    if (a.prefix_units)
      for (int bb = 0; bb < d.B; ++bb) atomicMax(a.dev_status + bb, GDN_TREE_STATUS_TIMEOUT);
    else
      atomicMax(a.dev_status + b, GDN_TREE_STATUS_TIMEOUT);
  }
}

// ---- joining the parts: a warp a row (node * Hq + h of sequence b) -----------------------
__global__ void __launch_bounds__(256)
attend_join_kernel(const float* __restrict__ part_o, const float* __restrict__ part_lse, int slots,
                   const int32_t* __restrict__ cu, gdn_tree_attend_dims d, int groups, bool few,
                   __nv_bfloat16* __restrict__ o, float* __restrict__ lse) {
  const int b = blockIdx.x / groups, lane = threadIdx.x & 31, D = d.D;
  const int first = cu[b], stop = cu[b + 1];
  const long long at = (long long)(blockIdx.x % groups) * 8 + (threadIdx.x >> 5);
  // (a sequence whose rows are out of range was reported, and has no parts)
  if (first < 0 || stop < first || stop > d.T || stop - first > d.N || at >= (long long)(stop - first) * d.Hq ||
      (few && (stop - first) * (d.Hq / d.Hkv) <= kAttendFewRows))  // (attend_few.cu adds those up itself)
    return;
  const size_t rows = (size_t)d.T * d.Hq, row = (size_t)first * d.Hq + at;
  float top = -INFINITY;
  for (int s = lane; s < slots; s += 32) top = fmaxf(top, part_lse[s * rows + row]);
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
  float sum = 0.f;
  for (int s = lane; s < slots; s += 32) {
    const float z = part_lse[s * rows + row];
    if (z != -INFINITY) sum += expf(z - top);  // (a NaN is kept, which fmaxf drops)
  }
  sum = warp_sum(sum);
  const float inv = sum > 0.f ? 1.f / sum : 0.f;
  float x[4] = {0.f, 0.f, 0.f, 0.f};
  if (4 * lane < D)
    for (int s = 0; s < slots; ++s) {
      const float z = part_lse[s * rows + row];
      if (z == -INFINITY) continue;  // a part that saw nothing
      const float w = expf(z - top) * inv;
      const float4 y = *reinterpret_cast<const float4*>(part_o + ((size_t)s * rows + row) * D + 4 * lane);
      x[0] = fmaf(w, y.x, x[0]);
      x[1] = fmaf(w, y.y, x[1]);
      x[2] = fmaf(w, y.z, x[2]);
      x[3] = fmaf(w, y.w, x[3]);
    }
  if (4 * lane < D)
    *reinterpret_cast<uint2*>(o + row * D + 4 * lane) =
        make_uint2(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]));
  if (lse && lane == 0) lse[row] = sum > 0.f ? top + logf(sum) : (sum == 0.f ? -INFINITY : sum);
}

// ---- the plan: what runs for these dims --------------------------------------------------
struct Plan {
  bool tc = false;
  bool shared = false;     // the prefix as units of its own
  int prefix_splits = 0, prefix_tiles = 0;
  bool many = false;       // some sequence may have more rows than attend_few.cu takes
  int seq_splits = 0, seq_tiles = 0;
  int slots = 0;           // parts of a row (0: the kernel writes o itself)
};

// Which units there are, by an estimate of the time.  A unit takes 1.6 us for each key tile,
// 0.95 where it has at most 128 rows, and 8 for its start and end, and each SM has one at a
// time; a part's sums are written and read again, and joined by a launch of its own.
//  - Into how many parts a unit's keys are split: what makes the last round full, as long as
//    the ends and the join do not eat it up.  Measured: 8 units of 33 tiles in 4, 8, 12 (taken),
//    16 and 24 parts 27.7, 23.0, 21.2, 22.5 and 32.1 us.
//  - Whether the prefix has units of its own, with 256 rows from several sequences each, or
//    every sequence reads it.  Measured (32 query and 8 key heads, 512 own rows; with / without,
//    the prefix of 1024, 4096 and 16384 rows): 32 sequences of 1 row 24 / 41, 35 / 106 and 44 /
//    344 us; of 8 nodes 59 / 44, 69 / 88 and 106 / 262; of 31 nodes 79 / 46, 116 / 90 and 263 /
//    264; of 64 nodes, whose units are full, 115 / 61, 188 / 134 and 481 / 429; 4 sequences of
//    8 nodes 25 / 16, 29 / 22 and 40 / 46, of 31 nodes 28 / 18, 34 / 24 and 56 / 48.
Plan plan_of(const gdn_tree_attend_dims& d) {
  constexpr float kTileUs = 1.6f, kTileUs1 = 0.95f, kEndsUs = 8.f, kJoinUs = 5.f;
  constexpr float kPartBytesPerUs = 6e6f;
  Plan p;
  p.tc = d.dtype == GDN_TREE_BF16;
  if (!p.tc) return p;
  const int sms = sm_count() > 0 ? sm_count() : 152;
  const int G = d.Hq / d.Hkv;
  const float part_us = 8.f * d.T * d.Hq * d.D / kPartBytesPerUs;
  auto row_tiles = [](long long r) { return (int)((r + 2 * kTile - 1) / (2 * kTile)); };
  // n units of so many rows and keys: the parts, and the time; joined: whether there are others
  auto split = [&](long long n, long long rows, long long keys, bool joined, int& parts) {
    const float tile_us = rows <= kTile ? kTileUs1 : kTileUs;
    const long long tiles = (keys + kTile - 1) / kTile;
    float best = 0.f;
    parts = 1;
    for (int s = 1; s <= kAttendMaxParts && (s == 1 || s <= tiles); ++s) {
      const float us = (float)((n * s + sms - 1) / sms) * ((tiles + s - 1) / s * tile_us + kEndsUs) +
                       (s > 1 || joined ? s * part_us : 0.f) + (s > 1 && !joined ? kJoinUs : 0.f);
      if (s > 1 && us >= best) continue;
      best = us;
      parts = s;
    }
    return best;
  };
  p.many = (long long)d.N * G > kAttendFewRows;
  p.seq_tiles = row_tiles((long long)d.N * G);
  const long long units = (long long)d.B * d.Hkv * p.seq_tiles;
  const long long own = (long long)d.table_width * d.page_size + d.N;
  float us = 0.f;  // the sequences' units read the prefix too
  if (p.many) us = split(units, (long long)d.N * G, own + d.prefix_len, false, p.seq_splits);
  if (d.prefix_len > 0 && d.B > 1) {
    if (!p.many) attend_few_cluster(d, d.prefix_len, &us);
    int prefix_splits, seq_splits = 0;
    const int prefix_tiles = row_tiles((long long)d.T * G);
    float with = split((long long)d.Hkv * prefix_tiles, (long long)d.T * G, d.prefix_len, true,
                       prefix_splits), rest;
    if (p.many) rest = split(units, (long long)d.N * G, own, true, seq_splits) + kJoinUs;
    else attend_few_cluster(d, 0, &rest);
    if (with + rest < us) {
      p.shared = true;
      p.prefix_tiles = prefix_tiles;
      p.prefix_splits = prefix_splits;
      p.seq_splits = seq_splits;
    }
  }
  p.slots = p.prefix_splits + p.seq_splits;
  if (!p.shared && p.seq_splits <= 1) p.slots = 0;
  return p;
}

size_t part_floats(const gdn_tree_attend_dims& d, const Plan& p) {
  return (size_t)p.slots * d.T * d.Hq * d.D;
}

template <int DP, bool kFork>
cudaError_t launch_units(const TcArgs& t, const CUtensorMap (&map)[5], long long blocks,
                         cudaStream_t stream) {
  if (blocks > 0x7fffffffll) return cudaErrorInvalidConfiguration;
  cudaError_t err = cudaFuncSetAttribute(attend_tc_kernel<DP, kFork>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         Smem<DP>::kBytes);
  if (err != cudaSuccess) return err;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)blocks);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = Smem<DP>::kBytes;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = t.rest ? 1 : 0;
  err = cudaLaunchKernelEx(&cfg, attend_tc_kernel<DP, kFork>, t, map[0], map[1], map[2], map[3],
                           map[4], wait_hooks());
  return err != cudaSuccess ? err : cudaGetLastError();
}

}  // namespace

size_t attend_workspace_bytes(const gdn_tree_attend_dims& d) {
  const Plan p = plan_of(d);
  if (!p.slots) return 0;
  return (part_floats(d, p) + (size_t)p.slots * d.T * d.Hq) * sizeof(float);
}

cudaError_t launch_attend(const AttendArgs& a, cudaStream_t stream) {
  const gdn_tree_attend_dims& d = a.d;
  const Plan p = plan_of(d);
  if (!p.tc) return launch_attend_f32(a, stream);
  typedef const __nv_bfloat16* bf;
  TcArgs t{};
  t.q = static_cast<bf>(a.q);
  t.k = static_cast<bf>(a.k);
  t.v = static_cast<bf>(a.v);
  t.parent = a.parent;
  t.cu = a.cu;
  t.k_cache = static_cast<bf>(a.k_cache);
  t.v_cache = static_cast<bf>(a.v_cache);
  t.table = a.page_table;
  t.ctx = a.context_len;
  t.prefix_pages = a.prefix_pages;
  t.scale = a.scale;
  t.o = static_cast<__nv_bfloat16*>(a.o);
  t.lse = a.lse;
  t.d = d;
  t.dev_status = a.dev_status;
  if (p.slots) {
    t.part_o = static_cast<float*>(a.workspace);
    t.part_lse = t.part_o + part_floats(d, p);
  }
  // cache tiles by TMA where pages and tiles divide one another
  CUtensorMap map[5];
  memset(map, 0, sizeof map);
  const int box = d.page_size < kTile ? d.page_size : kTile;
  const long long cache_rows = (long long)d.n_pages * d.page_size;
  if (d.D % 64 == 0 && box % 8 == 0 && kTile % box == 0 && d.page_size % box == 0 &&
      cache_rows > 0 && cache_rows < 0x7fffffffll && a.k_cache &&
      encode_head_rows_map(&map[0], a.k_cache, cache_rows, d.Hkv, d.D, box) &&
      encode_head_rows_map(&map[1], a.v_cache, cache_rows, d.Hkv, d.D, box))
    t.box_rows = box;
  t.own_box = d.D % 64 == 0 && a.k &&
              encode_head_rows_map(&map[2], a.k, d.T, d.Hkv, d.D, kTile) &&
              encode_head_rows_map(&map[3], a.v, d.T, d.Hkv, d.D, kTile);
  const int G = d.Hq / d.Hkv;
  t.q_box = d.D % 64 == 0 && kTile % G == 0 && a.scale >= 0.f &&
            encode_q_map(&map[4], a.q, d.T, d.Hq, d.D, G, kTile / G);
  // Units of at most 128 rows (`rows`: the most that one can have) have their key tiles taken by
  // turns.  Measured against one group of warps for all: 32 trees of 32 nodes 68.6 and 78.1 us,
  // 8 of them 37.5 and 45.0, 64-node trees with one query head a key head 70.1 and 73.9.
  auto units = [&](const TcArgs& x, long long blocks, long long rows) {
    if (rows <= kTile)
      return d.D <= 64 ? launch_units<64, true>(x, map, blocks, stream)
                       : launch_units<128, true>(x, map, blocks, stream);
    return d.D <= 64 ? launch_units<64, false>(x, map, blocks, stream)
                     : launch_units<128, false>(x, map, blocks, stream);
  };
  cudaError_t err = cudaSuccess;
  if (p.shared) {
    t.prefix_units = true;
    t.splits = p.prefix_splits;
    t.tiles = p.prefix_tiles;
    err = units(t, (long long)d.Hkv * p.prefix_tiles * p.prefix_splits, (long long)d.T * G);
    if (err != cudaSuccess) return err;
  }
  // Sequences of few rows, with the prefix's parts added up on the spot.  Where there are rows for
  // a batch of N each, that launch is saved and the units take all sequences: then all have N
  // rows, which are many, or the arrays are larger than what is in them.  Measured with 32 trees
  // of 128 nodes on 256 to 4096 rows, and with 16 of them single tokens: so 162 and 120 us, with
  // the launch 165 and 137.
  t.few = !p.many || d.T < (long long)d.B * d.N;
  if (t.few)
    err = launch_attend_few(a, p.shared ? 0 : d.prefix_len, t.part_o, t.part_lse, p.prefix_splits,
                            stream);
  if (err != cudaSuccess || !p.many) return err;
  t.prefix_units = false;
  t.with_prefix = !p.shared;
  t.slot0 = p.prefix_splits;
  t.splits = p.seq_splits;
  t.tiles = p.seq_tiles;
  t.by_length = d.B > 1 && d.B <= kMaxRanked && p.seq_splits == 1 &&
                (long long)d.B * d.Hkv * p.seq_tiles > sm_count();
  // What a last round of the SMs would be too few for goes in units of half the rows, beside
  // the others' last ones: 32 trees of 128 nodes (512 units, 56 in the last round) 164.8 to
  // 161.5 us, with 4096 own rows each 290 to 273 us.
  const long long each = (long long)d.Hkv * p.seq_tiles, sms = sm_count() > 0 ? sm_count() : 152;
  const long long half_tiles = ((long long)d.N * G + kTile - 1) / kTile;
  int halved = 0;
  if (t.by_length && half_tiles > 1) {
    const long long left = d.B * each % sms;
    halved = (int)((left + each - 1) / each);
    if (halved * d.Hkv * half_tiles > sms) halved = 0;
  }
  t.before_rest = halved > 0;
  err = units(t, (d.B - halved) * each * p.seq_splits, (long long)d.N * G);
  if (err == cudaSuccess && halved > 0) {
    t.before_rest = false;
    t.rest = true;
    t.rank0 = d.B - halved;
    t.tiles = (int)half_tiles;
    err = units(t, halved * d.Hkv * half_tiles, kTile);
  }
  if (err != cudaSuccess || !p.slots) return err;
  const int groups = (int)(((long long)d.N * d.Hq + 7) / 8);
  if ((long long)d.B * groups > 0x7fffffffll) return cudaErrorInvalidConfiguration;
  attend_join_kernel<<<(unsigned)(d.B * groups), 256, 0, stream>>>(
      t.part_o, t.part_lse, p.slots, t.cu, d, groups, t.few, t.o, t.lse);
  return cudaGetLastError();
}

}  // namespace gdn
