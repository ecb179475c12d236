// norm_rope.cu -- heads normalised and rotated, and rows that join the cache on the way.
//
// For a head's row x of D elements at position p, y = x * w * r with r = 1 / sqrt(sum x^2 * a +
// eps) (a = 1 / D or 1), then pair i of the first R elements is turned by p f_i.  f_i comes as
// turns a position in units of 2^-64: the product with the position, mod 2^64, is the angle's
// fraction of a turn, exact to p 2^-65 for every p, and one multiplication where a reduction of
// p f_i in floating point would need more bits than fp32 has (p = 10^6 leaves 2^-4 of a radian).
//
// A warp takes one head of one row.
#include <type_traits>

#include "common.cuh"
#include "kernels.h"

namespace gdn {
namespace {

constexpr int kWarps = 4;

// cos and sin of the angle at position p of a pair of this frequency, times the scale
__device__ __forceinline__ float2 turn(long long p, uint64_t freq, float scale) {
  const uint64_t phase = (uint64_t)p * freq + (1ull << 31);
  float s, c;
  sincospif((float)(int32_t)(phase >> 32) * 4.656612873077392578125e-10f, &s, &c);  // 2^-31
  return {c * scale, s * scale};
}

// Which sequence row t belongs to: the last b with cu[b] <= t.  (-1: none.  Whatever cu holds,
// the result is within [-1, B].)
__device__ __forceinline__ int sequence_of(const int32_t* cu, int B, int t) {
  int lo = -1, hi = B + 1;
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (cu[mid] <= t) lo = mid;
    else hi = mid;
  }
  return lo;
}

// rows, context and their place are in range
__device__ __forceinline__ bool valid_sequence(const RopeArgs& a, int b) {
  const int first = a.cu[b], stop = a.cu[b + 1], ctx = a.context_len[b];
  return first >= 0 && stop >= first && stop <= a.d.T && stop - first <= a.d.N && ctx >= 0 &&
         ctx <= (long long)a.d.table_width * a.d.page_size;
}

template <typename T, bool kAppend>
__global__ void __launch_bounds__(32 * kWarps)
norm_rope_kernel(const RopeArgs a) {
  __shared__ float staged[kWarps][kMaxD];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (kAppend) {
    const int b = blockIdx.x * blockDim.x + threadIdx.x;
    if (b < a.d.B) {
      const int ctx = a.context_len[b];
      const bool ok = valid_sequence(a, b);
      if (a.new_len) a.new_len[b] = ok ? (int)((unsigned)ctx + (a.cu[b + 1] - a.cu[b])) : ctx;
      if (!ok && a.dev_status) atomicMax(a.dev_status + b, GDN_TREE_STATUS_BAD_LAYOUT);
    }
  }
  const int H = a.d.Hq + (kAppend ? 2 : 1) * a.d.Hkv, D = a.d.D, R = a.rope.rotary_dim;
  const long long unit = (long long)blockIdx.x * kWarps + warp;
  const long long t = unit / H;
  if (t >= a.d.T) return;
  int h = (int)(unit - t * H);
  long long p = 0;
  T* row = nullptr;  // in the cache
  if (kAppend) {
    const int b = sequence_of(a.cu, a.d.B, (int)t);
    if (b < 0 || b >= a.d.B || !valid_sequence(a, b) || t >= a.cu[b + 1]) return;
    const long long at = (long long)a.context_len[b] + (t - a.cu[b]);
    p = a.d.prefix_len + at;
    if (h >= a.d.Hq) {
      int page = -1;
      if (at < (long long)a.d.table_width * a.d.page_size)
        page = a.page_table[(size_t)b * a.d.table_width + at / a.d.page_size];
      if (page >= 0 && page < a.d.n_pages) {
        const bool is_k = h < a.d.Hq + a.d.Hkv;
        row = static_cast<T*>(is_k ? a.k_cache : a.v_cache) +
              (((size_t)page * a.d.page_size + at % a.d.page_size) * a.d.Hkv +
               (h - a.d.Hq - (is_k ? 0 : a.d.Hkv))) * D;
      } else if (a.dev_status && lane == 0) {
        atomicMax(a.dev_status + b, GDN_TREE_STATUS_BAD_LAYOUT);
      }
    }
  } else if (R > 0) {
    p = a.positions[t];
  }
  const void* from = a.x.q;
  void* to = a.x.q_out;
  gdn_tree_strides si = a.x.q_strides, so = a.x.q_out_strides;
  const float* w = a.q_weight;
  bool plain = false;
  if (h >= a.d.Hq + a.d.Hkv) {
    h -= a.d.Hq + a.d.Hkv;
    from = a.x.v, to = a.x.v_out, si = a.x.v_strides, so = a.x.v_out_strides, w = nullptr;
    plain = true;
  } else if (h >= a.d.Hq) {
    h -= a.d.Hq;
    from = a.x.k, to = a.x.k_out, si = a.x.k_strides, so = a.x.k_out_strides, w = a.k_weight;
  }
  const T* x = static_cast<const T*>(from) + t * si.row + h * si.head;
  T* y = to ? static_cast<T*>(to) + t * so.row + h * so.head : nullptr;
  float v[kMaxD / 32], square = 0.f;
#pragma unroll
  for (int i = 0; i < kMaxD / 32; ++i) {
    const int e = lane + 32 * i;
    v[i] = e < D ? to_f32(x[e]) : 0.f;
    square += v[i] * v[i];
  }
  if (!plain && a.rope.norm != GDN_TREE_NORM_NONE) {
    square = warp_sum(square);
    const float r = __frsqrt_rn(square * (a.rope.norm == GDN_TREE_NORM_RMS ? 1.f / D : 1.f) +
                                a.rope.eps);
#pragma unroll
    for (int i = 0; i < kMaxD / 32; ++i) {
      const int e = lane + 32 * i;
      if (e < D) v[i] *= w ? r * w[e] : r;
    }
  }
  if (!plain && R > 0) {
#pragma unroll
    for (int i = 0; i < kMaxD / 32; ++i) staged[warp][lane + 32 * i] = v[i];
    __syncwarp();
#pragma unroll
    for (int i = 0; i < kMaxD / 32; ++i) {
      const int e = lane + 32 * i;
      if (e >= R) continue;
      const bool second = a.rope.interleaved ? e & 1 : e >= R / 2;
      const int pair = a.rope.interleaved ? e >> 1 : second ? e - R / 2 : e;
      const int other = a.rope.interleaved ? e ^ 1 : second ? pair : e + R / 2;
      const float2 cs = turn(p, a.freq[pair], a.rope.scale);
      const float z = staged[warp][other];
      v[i] = second ? v[i] * cs.x + z * cs.y : v[i] * cs.x - z * cs.y;
    }
  }
#pragma unroll
  for (int i = 0; i < kMaxD / 32; ++i) {
    const int e = lane + 32 * i;
    if (e >= D) continue;
    if (row) row[e] = from_f32<T>(v[i]);
    if (y) y[e] = from_f32<T>(v[i]);
  }
}

template <bool kAppend>
cudaError_t launch(const RopeArgs& a, cudaStream_t stream) {
  const long long H = a.d.Hq + (kAppend ? 2ll : 1ll) * a.d.Hkv;
  long long blocks = (a.d.T * H + kWarps - 1) / kWarps;
  if (kAppend) blocks = blocks > (a.d.B + 32 * kWarps - 1) / (32 * kWarps)
                            ? blocks : (a.d.B + 32 * kWarps - 1) / (32 * kWarps);
  if (blocks == 0) return cudaSuccess;
  if (blocks > 0x7fffffffll) return cudaErrorInvalidConfiguration;
  if (a.d.dtype == GDN_TREE_BF16)
    norm_rope_kernel<__nv_bfloat16, kAppend><<<(unsigned)blocks, 32 * kWarps, 0, stream>>>(a);
  else
    norm_rope_kernel<float, kAppend><<<(unsigned)blocks, 32 * kWarps, 0, stream>>>(a);
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
