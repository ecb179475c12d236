// norm_rope.cuh -- heads normalised and rotated, and rows that join the cache on the way.
//
// For a head's row x of D elements at position p, y = x * w * r with r = 1 / sqrt(sum x^2 * a +
// eps) (a = 1 / D or 1), then pair i of the first R elements is turned by p f_i.  f_i comes as
// turns a position in units of 2^-64: the product with the position, mod 2^64, is the angle's
// fraction of a turn, exact to p 2^-65 for every p, and one multiplication where a reduction of
// p f_i in floating point would need more bits than fp32 has (p = 10^6 leaves 2^-4 of a radian).
//
// Everything is read once and written once, so the call is bound by DRAM, or by latency where
// there are few rows.  A warp takes the heads of one row, or some of them: a head's elements lie
// over a few lanes (8 for 128 of bf16, 5 for 80), two 16-byte vectors a lane, and lane c of every head holds
// the same elements, so that the cosines and sines of a row are made once (a pair a lane, through
// shared memory) for all heads that a warp takes, and a pair's elements are in one lane.
//
// Measured on one GB300, twelve calls or more in a CUDA graph over inputs that do not fit the L2
// (an elementwise kernel over as many bytes in brackets): 32768 rows of 32 + 8 heads of 128 in bf16,
// every second 128 elements read, 99.6 us, 6.7 TB/s (96.2); 16384 rows of 16 + 16 heads made unit
// vectors 42.1 (40.1); 8191 rows of 16 + 16 heads rotated 22.4 (21.3); 4096 rows of 32 + 8 heads
// 15.8 (14.3: they are one round of the SMs, so that every warp's way from its first load to its
// last store counts); 16 prompts of 17 to 4096 rows into the cache and beside it 81.5, 6.4 TB/s
// (75.8); one row 2.0, into the cache 2.7.
//
// What that took, on the 32768 rows (one call a graph here and below, 4 us of which are the graph's
// start): vectors by plain loads, one or two passes ahead in registers,
// 130 to 149 us (loads in flight then cost registers, and with them warps); by cp.async, three
// passes ahead, 120; a lane's weights in registers and not from L1 in every pass, 106; fewer
// instructions (packed fp32 arithmetic; addresses by steps; lanes a head known to the compiler) and
// frequencies read before the position is there 104, and more where heads are small: 16384 rows of
// 32 + 8 heads of 80 elements 56 to 38 us, of 64 32.5 to 27.5.
#pragma once

#include <algorithm>
#include <type_traits>

#include "common.cuh"
#include "kernels.h"

namespace gdn {
namespace {

// (32768 rows: 106 us with 4 stages, 108 to 110 with 2, 3 or 5; 8 leave room for fewer warps)
constexpr int kWarps = 4, kStages = 4;

// How the pairs of a rotation lie in a lane's two vectors of E elements, number va and vb of the
// head's D / E (16384 rows of 32 + 8 heads of 128 in bf16: 52 us, 52, and 56 to 76):
//   kNeighbours  elements 2 i and 2 i + 1 are in the same vector
//   kHalves      R a multiple of 2 E (0 included): vb = va + R / 2 E holds va's partners
//   kCrossed     elements i and i + R / 2 for any other R: rotated in the ring, two pairs a lane
enum Pairs { kNeighbours, kHalves, kCrossed };

// cos and sin of the angle at position p of a pair of this frequency, times the scale
__device__ __forceinline__ float2 turn(long long p, uint64_t freq, float scale) {
  const uint64_t phase = (uint64_t)p * freq + (1ull << 31);
  float s, c;
  sincospif((float)(int32_t)(phase >> 32) * 4.656612873077392578125e-10f, &s, &c);  // 2^-31
  return {c * scale, s * scale};
}

__device__ __forceinline__ uint32_t smem_u32(const void* p) {
  return (uint32_t)__cvta_generic_to_shared(p);
}
__device__ __forceinline__ void copy16(uint32_t to, const void* from) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
}

// two elements at once: a * b and a * b + c
__device__ __forceinline__ float2 mul(float2 a, float2 b) {
  float2 d;
  asm("{.reg .b64 x, y; mov.b64 x, {%2, %3}; mov.b64 y, {%4, %5};\n"
      "mul.rn.f32x2 x, x, y; mov.b64 {%0, %1}, x;}"
      : "=f"(d.x), "=f"(d.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
__device__ __forceinline__ float2 fma(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{.reg .b64 x, y, z; mov.b64 x, {%2, %3}; mov.b64 y, {%4, %5}; mov.b64 z, {%6, %7};\n"
      "fma.rn.f32x2 x, x, y, z; mov.b64 {%0, %1}, x;}"
      : "=f"(d.x), "=f"(d.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}

// a 16-byte vector of E elements as E / 2 pairs of neighbours
template <typename T>
struct Vec;
template <>
struct Vec<float> {
  static constexpr int kSize = 4;
  static __device__ __forceinline__ void open(const uint4& v, float2* x) {
    x[0] = {__uint_as_float(v.x), __uint_as_float(v.y)};
    x[1] = {__uint_as_float(v.z), __uint_as_float(v.w)};
  }
  static __device__ __forceinline__ float2 two(const float* p) {
    return *reinterpret_cast<const float2*>(p);
  }
  static __device__ __forceinline__ void put(float* p, float2 x) {
    *reinterpret_cast<float2*>(p) = x;
  }
  // the first n elements (even) of one vector, the others of another
  static __device__ __forceinline__ uint4 mix(const uint4& a, const uint4& b, int n) {
    return {a.x, a.y, n > 2 ? a.z : b.z, n > 2 ? a.w : b.w};
  }
  static __device__ __forceinline__ uint4 close(const float2* x) {
    return {__float_as_uint(x[0].x), __float_as_uint(x[0].y), __float_as_uint(x[1].x),
            __float_as_uint(x[1].y)};
  }
};
template <>
struct Vec<__nv_bfloat16> {
  static constexpr int kSize = 8;
  static __device__ __forceinline__ void open(const uint4& v, float2* x) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i)
      x[i] = {__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u)};
  }
  static __device__ __forceinline__ float2 two(const __nv_bfloat16* p) {
    return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(p));
  }
  static __device__ __forceinline__ void put(__nv_bfloat16* p, float2 x) {
    *reinterpret_cast<__nv_bfloat162*>(p) = __floats2bfloat162_rn(x.x, x.y);
  }
  static __device__ __forceinline__ uint4 mix(const uint4& a, const uint4& b, int n) {
    return {a.x, n > 2 ? a.y : b.y, n > 4 ? a.z : b.z, n > 6 ? a.w : b.w};
  }
  static __device__ __forceinline__ uint4 close(const float2* x) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 p = __floats2bfloat162_rn(x[i].x, x[i].y);
      w[i] = reinterpret_cast<const uint32_t&>(p);
    }
    return {w[0], w[1], w[2], w[3]};
  }
};

// Rows of sequence b, its context and its place in the table are in range.
__device__ __forceinline__ bool in_range(const gdn_tree_attend_dims& d, int first, int stop,
                                         int ctx) {
  return first >= 0 && stop >= first && stop <= d.T && stop - first <= d.N && ctx >= 0 &&
         ctx <= (long long)d.table_width * d.page_size;
}

// Which sequence row t belongs to: the last b with cu[b] <= t, found by a warp, 32 offsets a
// round.  (-1 or B: none.  Whatever cu holds, every probe is within it.)  ctx: b's, read beside
// the last round's offsets where it can be.
__device__ __forceinline__ int sequence_of(const int32_t* cu, const int32_t* context_len, int B,
                                           int t, int lane, int* ctx) {
  int lo = -1, hi = B + 1;
  bool known = false;
  while (hi - lo > 1) {
    const int step = (hi - lo - 1 + 31) / 32, at = lo + (lane + 1) * step;
    const bool here = at < hi && cu[at] <= t;
    const int c = step == 1 && at < hi && at < B ? context_len[at] : -1;
    const int n = __popc(__ballot_sync(0xffffffffu, here));
    known = step == 1 && n > 0;
    if (known) *ctx = __shfl_sync(0xffffffffu, c, n - 1);
    lo += n * step;
    hi = min(hi, lo + step);
  }
  if (!known) *ctx = lo >= 0 && lo < B ? context_len[lo] : -1;
  return lo;
}

// How a row is divided: 32 / kLanes heads of q, of k or of v a pass (kLanes lanes have the D elements
// of a head), of_q and of_k passes; `splits` warps a row of `per` passes each.
struct Plan {
  int of_q, of_k, splits, per;
};

// A lane's way through the heads of a row that its passes take: the address of its own, how far it
// is to the one of the next pass, the head and how many there are.
struct Walk {
  char* at;
  long long step;
  int h, of;
  __device__ __forceinline__ bool on() const { return h < of; }
};

// CTAs an SM that the registers are to allow: 7 for rows alone (4096 rows 16.1 us, of 8 16.5, of 5
// 17.6); 5 for kCrossed (16384 rows, of 4, 5, 6 and 7: 40 of 80 elements 63, 56, 56 and 60 us, 126 of
// 128 75, 77, 79 and 80, 20 of 80 in fp32 78, 75, 69 and 70); 4 for rows for the cache, whose walks
// want more (2048 tokens 12.3 us, of 5 13.6, of 6 13.9)
constexpr int ctas(Pairs pairs, bool append) { return append ? 4 : pairs == kCrossed ? 5 : 7; }

template <typename T, int kLanes, Pairs kPairs, bool kAppend>
__global__ void __launch_bounds__(32 * kWarps, ctas(kPairs, kAppend))
norm_rope_kernel(const RopeArgs a, const Plan plan) {
  constexpr int E = Vec<T>::kSize, P = E / 2;  // elements and pairs of neighbours of a vector
  // vectors on their way: each lane's its own, head by head for kCrossed
  __shared__ uint4 ring[kWarps][kStages][64];
  __shared__ float4 turns[kWarps][kMaxD / 4];     // cos and sin of the row's pairs, two by two
  const int lane = threadIdx.x & 31, warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0);
  constexpr int D = 2 * E * kLanes;
  const int Hq = a.d.Hq, Hkv = a.d.Hkv, R = a.rope.rotary_dim;
  int t = blockIdx.x * kWarps + warp, i0 = 0;
  if (plan.splits > 1) {
    const int unit = t;
    t = unit / plan.splits;
    i0 = (unit - t * plan.splits) * plan.per;
  }
  const bool any = t < a.d.T;
  if (!kAppend && !any) return;
  // (where kLanes does not divide 32, the lanes behind the last whole head have none)
  constexpr int each = 32 / kLanes;
  const int g = lane / kLanes, c = lane % kLanes;
  const int k0 = plan.of_q, v0 = k0 + plan.of_k;  // the first passes of k and of v
  const int i1 = min(i0 + plan.per, kAppend ? v0 + plan.of_k : v0);
  constexpr int nv = kLanes;
  const int nr = R / (2 * E);
  const int va = kPairs == kHalves && c >= nr ? c + nr : c;
  const int vb = kPairs != kHalves ? c + nv : c < nr ? c + nr : va + nv - nr;
  const int to_b = (vb - va) * 16;  // bytes
  // the way of pass i and the ones after it of the same kind
  const auto walk = [&](int i, const void* q, const void* k, const void* v,
                        const gdn_tree_strides& sq, const gdn_tree_strides& sk,
                        const gdn_tree_strides& sv) {
    const bool is_q = i < k0, is_k = !kAppend || i < v0;
    const char* from = static_cast<const char*>(is_q ? q : is_k ? k : v);
    const gdn_tree_strides s = is_q ? sq : is_k ? sk : sv;
    const int h = (i - (is_q ? 0 : is_k ? k0 : v0)) * each + g;
    return Walk{const_cast<char*>(from) + (t * s.row + h * s.head) * (long long)sizeof(T) + va * 16,
                s.head * each * (long long)sizeof(T), h, g < each ? (is_q ? Hq : Hkv) : 0};
  };
  const int slot_a = kPairs != kCrossed ? lane : g < each ? g * 2 * kLanes + c : 0;
  const int slot_b = kPairs != kCrossed ? lane + 32 : slot_a + nv;
  // The vectors of passes i0, i0 + 1, ... are copied to the stages of the ring in turn (one group
  // a pass, empty or not).
  constexpr int kStage = sizeof(ring[0][0]);
  const uint32_t ring_a = smem_u32(&ring[warp][0][slot_a]);
  const uint32_t ring_b = smem_u32(&ring[warp][0][slot_b]);
  Walk in = walk(i0, a.q, a.k, a.v, a.s.q, a.s.k, a.s.v);
  int coming = any ? i0 : i1;  // the pass that is copied next
  uint32_t stage_in = 0;
  const auto fetch = [&] {
    if (coming < i1) {
      if (in.on()) {
        copy16(ring_a + stage_in, in.at);
        copy16(ring_b + stage_in, in.at + to_b);
      }
      in.at += in.step, in.h += each;
      ++coming;
      if (coming == k0 || (kAppend && coming == v0))
        in = walk(coming, a.q, a.k, a.v, a.s.q, a.s.k, a.s.v);
      stage_in = stage_in + kStage == kStages * kStage ? 0 : stage_in + kStage;
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
#pragma unroll
  for (int i = 0; i < kStages - 1; ++i) fetch();

  // the weights of this lane's elements: of q's, then of k's
  float2 w[2 * P];
  const auto load_weights = [&](const float* from) {
#pragma unroll
    for (int j = 0; j < 2 * P; j += 2) {
      const float4 v = from ? __ldg(reinterpret_cast<const float4*>(from + E * (j < P ? va : vb) +
                                                                    2 * (j & (P - 1))))
                            : float4{1.f, 1.f, 1.f, 1.f};
      w[j] = {v.x, v.y}, w[j + 1] = {v.z, v.w};
    }
  };
  load_weights(i0 < k0 ? a.q_weight : a.k_weight);

  // the frequencies of the pairs that this lane makes the cosines and sines of: of kCrossed, where
  // `wide` lanes take a head, its own pairs m0 and m1 (neighbours where R / 2 is even, so that they
  // are read and written together), else two of the row's
  const bool even = R % 4 == 0;
  const int need = even ? R / 4 : R / 2, wide = need > 16 ? 32 : need > 8 ? 16 : 8;
  const int m0 = kPairs == kCrossed ? (lane & (wide - 1)) << even : lane;
  const int m1 = kPairs == kCrossed && even ? m0 + 1 : m0 + 32;
  const uint64_t f0 = m0 < R / 2 ? a.freq[m0] : 0, f1 = m1 < R / 2 ? a.freq[m1] : 0;

  // The row's position, and its page and row there (-1: none).  (What is read here depends on one
  // another; everything above is on its way meanwhile.)
  long long p = 0;
  int b = -1, page = -1, page_row = 0;
  if (kAppend) {
    // a sequence to be looked at (in 64 bits: a row alone has 32 threads)
    const long long mine = (long long)blockIdx.x * (32 * kWarps) + threadIdx.x;
    if (mine < a.d.B) {
      const int first = a.cu[mine], stop = a.cu[mine + 1], ctx = a.context_len[mine];
      const bool ok = in_range(a.d, first, stop, ctx);
      if (a.new_len) a.new_len[mine] = ok ? (int)((unsigned)ctx + (unsigned)(stop - first)) : ctx;
      if (!ok && a.dev_status) atomicMax(a.dev_status + mine, GDN_TREE_STATUS_BAD_LAYOUT);
    }
    if (!any) return;  // (nothing was copied)
    int ctx;
    b = sequence_of(a.cu, a.context_len, a.d.B, t, lane, &ctx);
    const bool some = b >= 0 && b < a.d.B;
    const int first = some ? a.cu[b] : 0, stop = some ? a.cu[b + 1] : 0;
    if (!some || !in_range(a.d, first, stop, ctx) || t < first || t >= stop) {
      asm volatile("cp.async.wait_all;" ::: "memory");
      return;
    }
    const long long at = (long long)ctx + (t - first);
    p = a.d.prefix_len + at;
    if (i1 > k0 && at < (long long)a.d.table_width * a.d.page_size) {
      // (at fits 32 bits here)
      const unsigned entry = (unsigned)at / (unsigned)a.d.page_size;
      page = a.page_table[(size_t)b * a.d.table_width + entry];
      page_row = (int)((unsigned)at - entry * a.d.page_size);
    }
  } else if (R > 0) {
    p = a.positions[t];
  }

  // The row's cosines and sines, each made by one lane; then those of this lane's pairs (of
  // kNeighbours, pairs j of both vectors).
  constexpr int kMine = kPairs == kCrossed ? 1 : P;
  float2 co[kMine], si[kMine];
  if constexpr (kPairs == kCrossed) {
    const float2 f = turn(p, f0, a.rope.scale), h = turn(p, f1, a.rope.scale);
    co[0] = {f.x, h.x}, si[0] = {f.y, h.y};
  } else if (R > 0) {
    float2* const row = reinterpret_cast<float2*>(turns[warp]);
    if (m0 < R / 2) row[m0] = turn(p, f0, a.rope.scale);
    if (m1 < R / 2) row[m1] = turn(p, f1, a.rope.scale);
    __syncwarp();
#pragma unroll
    for (int j = 0; j < P; ++j) {
      if constexpr (kPairs == kHalves) {
        [[maybe_unused]] const float4 two =
            c < nr ? turns[warp][P * c + j] : float4{1.f, 0.f, 1.f, 0.f};
        co[j] = {two.x, two.z}, si[j] = {two.y, two.w};
      } else {
        const int m = P * va + j, n = P * vb + j;
        [[maybe_unused]] const float2 f = m < R / 2 ? row[m] : float2{1.f, 0.f};
        [[maybe_unused]] const float2 h = n < R / 2 ? row[n] : float2{1.f, 0.f};
        co[j] = {f.x, h.x}, si[j] = {f.y, h.y};
      }
    }
  }
  // the weights of kCrossed's pairs: of their first elements and of their second
  float2 w1 = {1.f, 1.f}, w2 = {1.f, 1.f};
  const auto cross_weights = [&](const float* from) {
    if (kPairs != kCrossed || from == nullptr) return;
    if (m0 < R / 2) w1.x = from[m0], w2.x = from[m0 + R / 2];
    if (m1 < R / 2) w1.y = from[m1], w2.y = from[m1 + R / 2];
  };
  cross_weights(i0 < k0 ? a.q_weight : a.k_weight);

  // the place in the cache (-1: none)
  long long place = -1;
  if (kAppend && i1 > k0) {
    if (page >= 0 && page < a.d.n_pages) place = (long long)page * a.d.page_size + page_row;
    else if (a.dev_status && lane == 0) atomicMax(a.dev_status + b, GDN_TREE_STATUS_BAD_LAYOUT);
  }

  const float share = a.rope.norm == GDN_TREE_NORM_RMS ? 1.f / D : 1.f;
  // where a pass's heads go: an output's (at NULL: none), and the cache's
  const auto walk_out = [&](int i) {
    Walk w = walk(i, a.q_out, a.k_out, a.v_out, a.s.q_out, a.s.k_out, a.s.v_out);
    if (kAppend && (i < k0 ? a.q_out : i < v0 ? a.k_out : a.v_out) == nullptr) w.at = nullptr;
    return w;
  };
  const auto walk_cache = [&](int i) {
    if (!kAppend || i < k0 || place < 0) return static_cast<char*>(nullptr);
    const int h = (i - (i < v0 ? k0 : v0)) * each + g;
    return static_cast<char*>(i < v0 ? a.k_cache : a.v_cache) +
           (place * Hkv + h) * D * (long long)sizeof(T) + va * 16;
  };
  Walk out = walk_out(i0);
  char* cached = walk_cache(i0);
  int now = 0;  // the stage
  for (int i = i0; i < i1; ++i) {
    const bool value = kAppend && i >= v0;
    // (kCrossed: the stage that is filled next was read by other lanes, this one is)
    if constexpr (kPairs == kCrossed) __syncwarp();
    fetch();
    asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 1) : "memory");
    if constexpr (kPairs == kCrossed) __syncwarp();
    uint4* const stage = ring[warp][now];
    now = now + 1 == kStages ? 0 : now + 1;
    uint4 y[2] = {stage[slot_a], stage[slot_b]};
    float2 x[2 * P];
    Vec<T>::open(y[0], x);
    Vec<T>::open(y[1], x + P);
    float r = 1.f;
    // (not of values: with theirs 16 prompts took 83.4 us, not 82.9, keys and values alone 33.0, not
    // 31.8, a few calls a graph)
    if (!value && a.rope.norm != GDN_TREE_NORM_NONE) {
      float2 two = {0.f, 0.f};
#pragma unroll
      for (int j = 0; j < 2 * P; ++j) two = fma(x[j], x[j], two);
      float square = two.x + two.y;
      if constexpr ((kLanes & (kLanes - 1)) == 0) {
#pragma unroll
        for (int o = kLanes / 2; o > 0; o >>= 1) square += __shfl_xor_sync(0xffffffffu, square, o);
      } else {  // (in one order, so that all lanes of a head have the same)
        float sum = 0.f;
#pragma unroll
        for (int n = 0; n < kLanes; ++n) sum += __shfl_sync(0xffffffffu, square, lane - c + n);
        square = sum;
      }
      r = rsqrtf(square * share + a.rope.eps);
    }
    if (!value && a.rope.norm != GDN_TREE_NORM_NONE) {
#pragma unroll
      for (int j = 0; j < 2 * P; ++j) x[j] = mul(x[j], mul(w[j], float2{r, r}));
    }
    if (kPairs == kHalves && !value && c < nr) {
#pragma unroll
      for (int j = 0; j < P; ++j) {
        const float2 u = x[j], v = x[P + j];
        x[j] = fma(u, co[j], mul(v, float2{-si[j].x, -si[j].y}));
        x[P + j] = fma(v, co[j], mul(u, si[j]));
      }
    }
    if (kPairs == kNeighbours && !value && R > 0) {
#pragma unroll
      for (int j = 0; j < P; ++j) {
        // (what is not rotated is left alone, not turned by 0: its pair may not be finite)
        const float2 u = x[j], v = x[P + j];
        if (P * va + j < R / 2)
          x[j] = {u.x * co[j].x - u.y * si[j].x, u.y * co[j].x + u.x * si[j].x};
        if (P * vb + j < R / 2)
          x[P + j] = {v.x * co[j].y - v.y * si[j].y, v.y * co[j].y + v.x * si[j].y};
      }
    }
    if (kPairs == kCrossed && !value) {
      __syncwarp();  // (every lane has its vectors)
      // (out.h - g is the pass's first head)
      const int heads = min(each, (i < k0 ? Hq : Hkv) - (out.h - g));
      for (int n0 = 0; n0 < heads; n0 += 32 / wide) {
        const int n = min(n0 + lane / wide, heads - 1);
        const float rn = __shfl_sync(0xffffffffu, r, n * kLanes);
        T* const head = reinterpret_cast<T*>(stage + n * 2 * kLanes);
        if (n0 + lane / wide < heads && m0 < R / 2) {
          const auto cross = [&](float2& u, float2& v) {
            u = mul(u, mul(w1, float2{rn, rn})), v = mul(v, mul(w2, float2{rn, rn}));
            const float2 t = u;
            u = fma(u, co[0], mul(v, float2{-si[0].x, -si[0].y}));
            v = fma(v, co[0], mul(t, si[0]));
          };
          if (even) {
            float2 u = Vec<T>::two(head + m0), v = Vec<T>::two(head + m0 + R / 2);
            cross(u, v);
            Vec<T>::put(head + m0, u), Vec<T>::put(head + m0 + R / 2, v);
          } else {
            const bool both = m1 < R / 2;
            const int m = both ? m1 : m0;
            float2 u = {to_f32(head[m0]), to_f32(head[m])};
            float2 v = {to_f32(head[m0 + R / 2]), to_f32(head[m + R / 2])};
            cross(u, v);
            head[m0] = from_f32<T>(u.x), head[m0 + R / 2] = from_f32<T>(v.x);
            if (both) head[m1] = from_f32<T>(u.y), head[m1 + R / 2] = from_f32<T>(v.y);
          }
        }
      }
      __syncwarp();
    }
    if (i + 1 == k0) {  // (ahead of the first pass that takes them)
      load_weights(a.k_weight);
      w1 = w2 = {1.f, 1.f};
      cross_weights(a.k_weight);
    }
    if (out.on()) {
      if (kPairs == kCrossed && !value) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int left = R - E * (j ? vb : va);  // rotated elements of the vector
          const uint4 own = Vec<T>::close(x + j * P), turned = stage[j ? slot_b : slot_a];
          y[j] = left >= E ? turned : left <= 0 ? own : Vec<T>::mix(turned, own, left);
        }
      } else if (!value) {
        y[0] = Vec<T>::close(x), y[1] = Vec<T>::close(x + P);
      }
      if (!kAppend || out.at) {
        *reinterpret_cast<uint4*>(out.at) = y[0];
        *reinterpret_cast<uint4*>(out.at + to_b) = y[1];
      }
      if (kAppend && cached) {
        *reinterpret_cast<uint4*>(cached) = y[0];
        *reinterpret_cast<uint4*>(cached + to_b) = y[1];
      }
    }
    if (i + 1 == k0 || (kAppend && i + 1 == v0)) {
      out = walk_out(i + 1);
      cached = walk_cache(i + 1);
    } else {
      if (!kAppend || out.at) out.at += out.step;
      out.h += each;
      if (kAppend && cached) cached += each * D * (int)sizeof(T);
    }
  }
}

template <typename T, bool kAppend>
cudaError_t launch(const RopeArgs& a, cudaStream_t stream) {
  constexpr int E = Vec<T>::kSize;
  const int R = a.rope.rotary_dim;
  Plan plan{};
  const int each = 32 / (a.d.D / (2 * E));
  plan.of_q = (a.d.Hq + each - 1) / each;
  plan.of_k = (a.d.Hkv + each - 1) / each;
  const int passes = plan.of_q + (kAppend ? 2 : 1) * plan.of_k;
  const int sms = sm_count();
  // Warps a row: one where the rows alone fill the SMs (what a warp makes once for its row is then
  // made once), more where they do not (a warp's passes follow one another).  Measured with 32 + 8
  // heads of 128 in bf16, a warp a row against this rule: 1 row 6.5 and 2.1 us, 256 rows 6.8 and
  // 3.0, 1024 rows 8.6 and 6.7, 2048 rows 9.8 and 9.1; four warps a row at 4096 rows 22 us against
  // 16.3.  Rows for the cache take longer to begin: 1024 tokens 10.9 us at 16 warps an SM, 8.9 at 12.
  const int want = (kAppend ? 12 : 14) * sms;
  int splits = 1;
  if (a.d.T > 0 && a.d.T <= want) splits = std::min(passes, want / a.d.T + 1);
  plan.per = (passes + splits - 1) / splits;
  plan.splits = (passes + plan.per - 1) / plan.per;
  long long blocks = ((long long)a.d.T * plan.splits + kWarps - 1) / kWarps;
  if (kAppend) blocks = std::max(blocks, ((long long)a.d.B + 32 * kWarps - 1) / (32 * kWarps));
  if (blocks == 0) return cudaSuccess;
  const auto go = [&](auto lanes, auto pairs) {
    norm_rope_kernel<T, decltype(lanes)::value, decltype(pairs)::value, kAppend>
        <<<(unsigned)blocks, 32 * kWarps, 0, stream>>>(a, plan);
  };
  const auto by_pairs = [&](auto lanes) {
    if (a.rope.interleaved) go(lanes, std::integral_constant<Pairs, kNeighbours>());
    else if (R % (2 * E) == 0) go(lanes, std::integral_constant<Pairs, kHalves>());
    else go(lanes, std::integral_constant<Pairs, kCrossed>());
  };
  constexpr int kLeast = 16 / (2 * E);  // of a head of 16 elements
  switch (a.d.D / 16) {
    case 1: by_pairs(std::integral_constant<int, kLeast>()); break;
    case 2: by_pairs(std::integral_constant<int, 2 * kLeast>()); break;
    case 3: by_pairs(std::integral_constant<int, 3 * kLeast>()); break;
    case 4: by_pairs(std::integral_constant<int, 4 * kLeast>()); break;
    case 5: by_pairs(std::integral_constant<int, 5 * kLeast>()); break;
    case 6: by_pairs(std::integral_constant<int, 6 * kLeast>()); break;
    case 7: by_pairs(std::integral_constant<int, 7 * kLeast>()); break;
    default: by_pairs(std::integral_constant<int, 8 * kLeast>()); break;
  }
  return cudaGetLastError();
}

}  // namespace
}  // namespace gdn
