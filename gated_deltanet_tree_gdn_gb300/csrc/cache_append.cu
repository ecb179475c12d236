// cache_append.cu -- rows of k and v (an accepted path's, or all of a sequence's) into
// the pages of a paged cache.
//
// A row is Hkv * D contiguous elements in the packed arrays and in a page alike, so the
// call is a copy of rows between two address maps: bound by DRAM (each row read and
// written once), or by latency where a path of a few rows is all there is.  A CTA takes
// kThreads / lanes rows of one sequence, as many lanes a row (a power of two, a warp at most)
// as it has 16-byte pieces, k and v together.  16 prompts of 17 to 4096 rows of 8 heads of 128
// bf16 take 32 us (5.8 TB/s read and written); 32 paths of up to 24 rows 3 us.
#include <algorithm>

#include "common.cuh"
#include "kernels.h"

namespace gdn {
namespace {

constexpr int kThreads = 256;

__global__ void __launch_bounds__(kThreads)
cache_append_kernel(const uint4* __restrict__ k, const uint4* __restrict__ v,
                    const int32_t* __restrict__ path, const int32_t* __restrict__ path_len,
                    int Lmax, const int32_t* __restrict__ cu, uint4* k_cache, uint4* v_cache,
                    const int32_t* __restrict__ table, const int32_t* __restrict__ context_len,
                    int32_t* new_len, gdn_tree_attend_dims d, int vecs, int lanes,
                    int groups, int32_t* dev_status) {
  const int b = blockIdx.x / groups, j0 = (blockIdx.x % groups) * (kThreads / lanes);
  const int lane = threadIdx.x & (lanes - 1), j = j0 + threadIdx.x / lanes;
  const int first = cu[b], stop = cu[b + 1], ctx = context_len[b];
  const int rows = stop - first;
  const int len = path_len ? path_len[b] : rows;
  const long long cap = (long long)d.table_width * d.page_size;
  int bad = GDN_TREE_STATUS_OK;
  // (stop < first, not rows < 0: of two numbers far apart the difference may wrap)
  if (first < 0 || stop < first || stop > d.T || rows > d.N || ctx < 0 || ctx > cap)
    bad = GDN_TREE_STATUS_BAD_LAYOUT;
  else if (path_len && (len < 0 || len > Lmax))
    bad = GDN_TREE_STATUS_BAD_PATH;
  if (j0 == 0 && threadIdx.x == 0) {
    if (new_len) new_len[b] = bad ? ctx : ctx + len;
    if (bad && dev_status) atomicMax(dev_status + b, bad);
  }
  if (bad || j >= len) return;
  const int node = path ? path[(size_t)b * Lmax + j] : j;
  const long long at = (long long)ctx + j;
  int page = -1;
  if (node < 0 || node >= rows) bad = GDN_TREE_STATUS_BAD_PATH;
  else if (at >= cap) bad = GDN_TREE_STATUS_BAD_LAYOUT;
  else {
    page = table[(size_t)b * d.table_width + at / d.page_size];
    if (page < 0 || page >= d.n_pages) bad = GDN_TREE_STATUS_BAD_LAYOUT;
  }
  if (bad) {
    if (dev_status && lane == 0) atomicMax(dev_status + b, bad);
    return;
  }
  const size_t src = (size_t)(first + node) * vecs;
  const size_t dst = ((size_t)page * d.page_size + (size_t)(at % d.page_size)) * vecs;
  // eight loads of a lane in flight (a row of 8 heads of 128 bf16, k and v, is one round)
  for (int i0 = lane; i0 < vecs; i0 += 4 * lanes) {
    uint4 x[4], y[4];
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (i0 + lanes * e < vecs) {
        x[e] = __ldcs(k + src + i0 + lanes * e);
        y[e] = __ldcs(v + src + i0 + lanes * e);
      }
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (i0 + lanes * e < vecs) {
        k_cache[dst + i0 + lanes * e] = x[e];
        v_cache[dst + i0 + lanes * e] = y[e];
      }
  }
}

}  // namespace

cudaError_t launch_cache_append(const AppendArgs& a, cudaStream_t stream) {
  const gdn_tree_attend_dims& d = a.d;
  const int vecs = d.Hkv * d.D * (d.dtype == GDN_TREE_BF16 ? 2 : 4) / 16;
  // (the first row past the last page is reported for all of them: what lies behind it is not
  // looked at, however long the paths may be)
  const long long room = (long long)d.table_width * d.page_size + 1;
  const long long most = std::min<long long>(a.path ? a.Lmax : d.N, room);
  int lanes = 1;
  while (lanes < 32 && lanes < vecs) lanes *= 2;
  const int groups = most > 0 ? (int)((most * lanes + kThreads - 1) / kThreads) : 1;
  const long long blocks = (long long)d.B * groups;
  if (blocks > 0x7fffffffll) return cudaErrorInvalidConfiguration;
  cache_append_kernel<<<(unsigned)blocks, kThreads, 0, stream>>>(
      static_cast<const uint4*>(a.k), static_cast<const uint4*>(a.v), a.path, a.path_len, a.Lmax,
      a.cu, static_cast<uint4*>(a.k_cache), static_cast<uint4*>(a.v_cache), a.page_table,
      a.context_len, a.new_len, d, vecs, lanes, groups, a.dev_status);
  return cudaGetLastError();
}

}  // namespace gdn
