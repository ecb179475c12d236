// norm_rope.cu -- heads normalised and rotated, and rows that join the cache on the way.
//
// For a head's row x of D elements at position p, y = x * w * r with r = 1 / sqrt(sum x^2 * a +
// eps) (a = 1 / D or 1), then pair i of the first R elements is turned by p f_i.  f_i comes as
// turns a position in units of 2^-64: the product with the position, mod 2^64, is the angle's
// fraction of a turn, exact to p 2^-65 for every p, and one multiplication where a reduction of
// p f_i in floating point would need more bits than fp32 has (p = 10^6 leaves 2^-4 of a radian).
//
// Everything is read once and written once, so the call is bound by DRAM, or by latency where
// there are few rows.  A warp takes some heads of one row: a head's elements lie over a few lanes
// (8 for 128 of bf16), two 16-byte vectors a lane, and lane c of every head holds the same
// elements, so that the cosines and sines of a row are made once for all heads that a warp takes.
#include <algorithm>
#include <type_traits>

#include "common.cuh"
#include "kernels.h"

namespace gdn {
namespace {

constexpr int kWarps = 4, kBatch = 2;

// How the pairs of a rotation lie in a lane's two vectors of E elements, number va and vb of the
// head's D / E:
//   kNeighbours  elements 2 i and 2 i + 1 are in the same vector
//   kHalves      R a multiple of 2 E (0 included): vb = va + R / 2 E holds va's partners
//   kCrossed     elements i and i + R / 2 for any other R: through shared memory
enum Pairs { kNeighbours, kHalves, kCrossed };

// cos and sin of the angle at position p of a pair of this frequency, times the scale
__device__ __forceinline__ float2 turn(long long p, uint64_t freq, float scale) {
  const uint64_t phase = (uint64_t)p * freq + (1ull << 31);
  float s, c;
  sincospif((float)(int32_t)(phase >> 32) * 4.656612873077392578125e-10f, &s, &c);  // 2^-31
  return {c * scale, s * scale};
}

template <typename T>
struct Vec;
template <>
struct Vec<float> {
  static constexpr int kSize = 4;
  static __device__ __forceinline__ void open(const uint4& v, float* x) {
    x[0] = __uint_as_float(v.x), x[1] = __uint_as_float(v.y);
    x[2] = __uint_as_float(v.z), x[3] = __uint_as_float(v.w);
  }
  static __device__ __forceinline__ uint4 close(const float* x) {
    return {__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]),
            __float_as_uint(x[3])};
  }
};
template <>
struct Vec<__nv_bfloat16> {
  static constexpr int kSize = 8;
  static __device__ __forceinline__ void open(const uint4& v, float* x) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
  static __device__ __forceinline__ uint4 close(const float* x) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 p = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
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

template <typename T, Pairs kPairs, bool kAppend>
__global__ void __launch_bounds__(32 * kWarps)
norm_rope_kernel(const RopeArgs a, int lanes, int splits, int per) {
  constexpr int E = Vec<T>::kSize;
  constexpr int kTurns = kPairs == kCrossed ? 2 * E : E;  // a lane's
  __shared__ float staged[kPairs == kCrossed ? kWarps : 1][kPairs == kCrossed ? 64 * E : 1];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int Hq = a.d.Hq, Hkv = a.d.Hkv, D = a.d.D, R = a.rope.rotary_dim;
  if (kAppend) {
    const int b = blockIdx.x * (32 * kWarps) + threadIdx.x;
    if (b < a.d.B) {
      const int first = a.cu[b], stop = a.cu[b + 1], ctx = a.context_len[b];
      const bool ok = in_range(a.d, first, stop, ctx);
      if (a.new_len) a.new_len[b] = ok ? (int)((unsigned)ctx + (unsigned)(stop - first)) : ctx;
      if (!ok && a.dev_status) atomicMax(a.dev_status + b, GDN_TREE_STATUS_BAD_LAYOUT);
    }
  }
  const int unit = blockIdx.x * kWarps + warp, t = unit / splits;
  if (t >= a.d.T) return;
  // heads: a warp takes 32 / lanes at a time, q's, then k's, then v's
  const int each = 32 / lanes, g = lane / lanes, c = lane & (lanes - 1);
  const int H = Hq + (kAppend ? 2 : 1) * Hkv;
  const int h0 = (unit - t * splits) * per * each + g;
  const int h1 = min(H, (unit - t * splits + 1) * per * each);
  const int nv = D / (2 * E), nr = R / (2 * E);
  const bool has = c < nv;
  const int va = kPairs == kHalves && c >= nr ? c + nr : c;
  const int vb = kPairs != kHalves ? c + nv : c < nr ? c + nr : va + nv - nr;

  const T* const q = static_cast<const T*>(a.q) + t * a.s.q.row;
  const T* const k = static_cast<const T*>(a.k) + t * a.s.k.row;
  const T* const v = static_cast<const T*>(a.v) + (kAppend ? t * a.s.v.row : 0);
  const auto fetch = [&](int h, uint4* x) {
    if (!has || h >= h1) return;
    const T* p = h < Hq ? q + h * a.s.q.head
                 : !kAppend || h < Hq + Hkv ? k + (h - Hq) * a.s.k.head
                                            : v + (h - Hq - Hkv) * a.s.v.head;
    x[0] = __ldcs(reinterpret_cast<const uint4*>(p) + va);
    x[1] = __ldcs(reinterpret_cast<const uint4*>(p) + vb);
  };
  uint4 next[kBatch][2];
#pragma unroll
  for (int i = 0; i < kBatch; ++i) fetch(h0 + i * each, next[i]);

  // the row's position, and its place in the cache (-1: none)
  long long p = 0, place = -1;
  if (kAppend) {
    int ctx;
    const int b = sequence_of(a.cu, a.context_len, a.d.B, t, lane, &ctx);
    if (b < 0 || b >= a.d.B) return;
    const int first = a.cu[b], stop = a.cu[b + 1];
    if (!in_range(a.d, first, stop, ctx) || t < first || t >= stop) return;
    const long long at = (long long)ctx + (t - first);
    p = a.d.prefix_len + at;
    if (h1 > Hq) {
      if (at < (long long)a.d.table_width * a.d.page_size) {
        // (at fits 32 bits here)
        const unsigned entry = (unsigned)at / (unsigned)a.d.page_size;
        const int page = a.page_table[(size_t)b * a.d.table_width + entry];
        if (page >= 0 && page < a.d.n_pages)
          place = (long long)page * a.d.page_size + ((unsigned)at - entry * a.d.page_size);
      }
      if (place < 0 && a.dev_status && lane == 0)
        atomicMax(a.dev_status + b, GDN_TREE_STATUS_BAD_LAYOUT);
    }
  } else if (R > 0) {
    p = a.positions[t];
  }

  // the row's cosines and sines, of the pairs of this lane
  float co[kTurns], si[kTurns];
#pragma unroll
  for (int i = 0; i < kTurns; ++i) {
    co[i] = 1.f, si[i] = 0.f;
    int pair;
    bool turned;
    if (kPairs == kHalves) {
      pair = E * c + i, turned = c < nr;
    } else if (kPairs == kNeighbours) {
      pair = (E / 2) * (i < E / 2 ? va : vb) + (i & (E / 2 - 1)), turned = pair < R / 2;
    } else {
      const int e = E * (i < E ? va : vb) + (i & (E - 1));
      pair = e < R / 2 ? e : e - R / 2, turned = e < R;
    }
    if (turned && has) {
      const float2 cs = turn(p, a.freq[pair], a.rope.scale);
      co[i] = cs.x, si[i] = cs.y;
    }
  }

  const float share = a.rope.norm == GDN_TREE_NORM_RMS ? 1.f / D : 1.f;
  for (int h = h0; h - g < h1; h += kBatch * each) {
    uint4 raw[kBatch][2];
#pragma unroll
    for (int i = 0; i < kBatch; ++i) raw[i][0] = next[i][0], raw[i][1] = next[i][1];
#pragma unroll
    for (int i = 0; i < kBatch; ++i) fetch(h + (kBatch + i) * each, next[i]);
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int hi = h + i * each;
      if (hi - g >= h1) break;  // (the warp's)
      const bool mine = has && hi < h1, value = kAppend && hi >= Hq + Hkv;
      float x[2 * E];
      if (mine) {
        Vec<T>::open(raw[i][0], x);
        Vec<T>::open(raw[i][1], x + E);
      } else {
#pragma unroll
        for (int e = 0; e < 2 * E; ++e) x[e] = 0.f;
      }
      if (a.rope.norm != GDN_TREE_NORM_NONE) {
        float square = 0.f;
#pragma unroll
        for (int e = 0; e < 2 * E; ++e) square += x[e] * x[e];
        for (int o = lanes / 2; o > 0; o >>= 1) square += __shfl_xor_sync(0xffffffffu, square, o);
        if (mine && !value) {
          const float r = __frsqrt_rn(square * share + a.rope.eps);
          const float* const w = hi < Hq ? a.q_weight : a.k_weight;
          if (w) {
#pragma unroll
            for (int e = 0; e < 2 * E; e += 4) {
              const float4 f = __ldg(reinterpret_cast<const float4*>(w + E * (e < E ? va : vb) +
                                                                     (e & (E - 1))));
              x[e] *= r * f.x, x[e + 1] *= r * f.y, x[e + 2] *= r * f.z, x[e + 3] *= r * f.w;
            }
          } else {
#pragma unroll
            for (int e = 0; e < 2 * E; ++e) x[e] *= r;
          }
        }
      }
      if (kPairs == kHalves) {
        if (c < nr && !value) {
#pragma unroll
          for (int e = 0; e < E; ++e) {
            const float u = x[e], w = x[E + e];
            x[e] = u * co[e] - w * si[e];
            x[E + e] = w * co[e] + u * si[e];
          }
        }
      } else if (kPairs == kNeighbours) {
#pragma unroll
        for (int e = 0; e < E; ++e) {
          // (what is not rotated is left alone, not turned by 0: its pair may not be finite)
          const bool turned = (E / 2) * (e < E / 2 ? va : vb) + (e & (E / 2 - 1)) < R / 2;
          const float u = x[2 * e], w = x[2 * e + 1];
          if (turned && !value) {
            x[2 * e] = u * co[e] - w * si[e];
            x[2 * e + 1] = w * co[e] + u * si[e];
          }
        }
      } else {
        float* const row = staged[warp] + g * D;
        __syncwarp();
        if (has) {
#pragma unroll
          for (int e = 0; e < 2 * E; e += 4)
            *reinterpret_cast<float4*>(row + E * (e < E ? va : vb) + (e & (E - 1))) =
                float4{x[e], x[e + 1], x[e + 2], x[e + 3]};
        }
        __syncwarp();
        if (has && !value) {
#pragma unroll
          for (int e = 0; e < 2 * E; ++e) {
            const int n = E * (e < E ? va : vb) + (e & (E - 1));
            if (n < R) {
              const float u = row[n < R / 2 ? n + R / 2 : n - R / 2];
              x[e] = n < R / 2 ? x[e] * co[e] - u * si[e] : x[e] * co[e] + u * si[e];
            }
          }
        }
      }
      if (!mine) continue;
      const uint4 ya = Vec<T>::close(x), yb = Vec<T>::close(x + E);
      const auto put = [&](T* row) {
        reinterpret_cast<uint4*>(row)[va] = ya;
        reinterpret_cast<uint4*>(row)[vb] = yb;
      };
      if (hi < Hq) {
        put(static_cast<T*>(a.q_out) + t * a.s.q_out.row + hi * a.s.q_out.head);
      } else if (!kAppend) {
        put(static_cast<T*>(a.k_out) + t * a.s.k_out.row +
            (hi - Hq) * a.s.k_out.head);
      } else {
        const int n = hi - Hq - (value ? Hkv : 0);
        if (place >= 0)
          put(static_cast<T*>(value ? a.v_cache : a.k_cache) + (place * Hkv + n) * D);
        T* const out = static_cast<T*>(value ? a.v_out : a.k_out);
        const gdn_tree_strides s = value ? a.s.v_out : a.s.k_out;
        if (out) put(out + t * s.row + n * s.head);
      }
    }
  }
}

template <bool kAppend>
cudaError_t launch(const RopeArgs& a, cudaStream_t stream) {
  const bool bf16 = a.d.dtype == GDN_TREE_BF16;
  const int H = a.d.Hq + (kAppend ? 2 : 1) * a.d.Hkv, E = bf16 ? 8 : 4, R = a.rope.rotary_dim;
  int lanes = 1;
  while (lanes * 2 * E < a.d.D) lanes *= 2;
  const int each = 32 / lanes, passes = (H + each - 1) / each;
  const int sms = sm_count();
  int splits = 1;
  if (a.d.T > 0 && (long long)a.d.T < 16ll * sms) splits = std::min(passes, 16 * sms / a.d.T + 1);
  const int per = (passes + splits - 1) / splits;
  splits = (passes + per - 1) / per;
  long long blocks = ((long long)a.d.T * splits + kWarps - 1) / kWarps;
  if (kAppend) blocks = std::max(blocks, ((long long)a.d.B + 32 * kWarps - 1) / (32 * kWarps));
  if (blocks == 0) return cudaSuccess;
  const auto go = [&](auto type, auto pairs) {
    norm_rope_kernel<decltype(type), decltype(pairs)::value, kAppend>
        <<<(unsigned)blocks, 32 * kWarps, 0, stream>>>(a, lanes, splits, per);
  };
  const auto by_pairs = [&](auto type) {
    if (a.rope.interleaved) go(type, std::integral_constant<Pairs, kNeighbours>());
    else if (R % (2 * E) == 0) go(type, std::integral_constant<Pairs, kHalves>());
    else go(type, std::integral_constant<Pairs, kCrossed>());
  };
  if (bf16) by_pairs(__nv_bfloat16());
  else by_pairs(float());
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_norm_rope(const RopeArgs& a, cudaStream_t stream) {
  return launch<false>(a, stream);
}

cudaError_t launch_cache_append_rope(const RopeArgs& a, cudaStream_t stream) {
  return launch<true>(a, stream);
}

}  // namespace gdn
