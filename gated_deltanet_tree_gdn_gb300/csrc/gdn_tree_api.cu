// gdn_tree_api.cu -- the extern "C" entry points of libgdntree.
//
// Every shape, dtype, pointer and alignment check happens here, on the host,
// before anything is enqueued; the kernels only check what depends on device
// data (tree and path validity) and report it through dev_status.
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>
#include <stdio.h>
#include <stdlib.h>
#include <string.h>

#include "../../include/gdn_tree.h"
#include "chain_unit.cuh"
#include "kernels.h"

namespace {

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

// [a0, a0 + bytes) and [a1, a1 + bytes) overlap without being the same range
bool partial_overlap(const void* p0, const void* p1, size_t bytes) {
  const char* a0 = reinterpret_cast<const char*>(p0);
  const char* a1 = reinterpret_cast<const char*>(p1);
  return a0 != a1 && a0 < a1 + bytes && a1 < a0 + bytes;
}

// [a0, a0 + b0) and [a1, a1 + b1) overlap at all
bool any_overlap(const void* p0, size_t b0, const void* p1, size_t b1) {
  const char* a0 = reinterpret_cast<const char*>(p0);
  const char* a1 = reinterpret_cast<const char*>(p1);
  return b0 && b1 && a0 < a1 + b1 && a1 < a0 + b0;
}

// packed-layout arguments: offsets and slots (device pointers), row count, slots
int check_packed(const int32_t* cu, int32_t T, const int32_t* slot, int32_t n_slots, int B,
                 gdn::SeqLayout* lay) {
  if (T < 0 || n_slots < 0) return GDN_TREE_EINVAL;
  if (cu == nullptr || !aligned4(cu)) return GDN_TREE_EINVAL;
  if (slot != nullptr && !aligned4(slot)) return GDN_TREE_EINVAL;
  if (slot == nullptr && n_slots < B) return GDN_TREE_EINVAL;
  lay->cu = cu;
  lay->slot = slot;
  lay->T = T;
  lay->n_slots = n_slots;
  return GDN_TREE_OK;
}

bool supported_head_dim(int d) { return d >= 16 && d <= gdn::kMaxDHost && d % 16 == 0; }

int check_dims(const gdn_tree_dims& d) {
  if (d.B < 0 || d.N < 0 || d.Hqk <= 0 || d.Hv <= 0 || d.dk <= 0 || d.dv <= 0)
    return GDN_TREE_EINVAL;
  if (d.Hv % d.Hqk != 0) return GDN_TREE_EINVAL;
  if (d.dtype != GDN_TREE_BF16 && d.dtype != GDN_TREE_F32) return GDN_TREE_EUNSUPPORTED;
  if (d.N > gdn::kMaxNLongHost) return GDN_TREE_EUNSUPPORTED;
  if (!supported_head_dim(d.dk) || !supported_head_dim(d.dv)) return GDN_TREE_EUNSUPPORTED;
  // every flat index must fit comfortably in the kernels' size_t arithmetic and
  // the grid's y dimension
  if (d.B > 65535) return GDN_TREE_EUNSUPPORTED;
  return GDN_TREE_OK;
}

// the dims of a rule over sequences of any length (prefill, decoding step)
int check_rule_dims(gdn_tree_dims d) {
  if (d.N < 0) return GDN_TREE_EINVAL;
  d.N = 1;  // the tree calls' limit on N does not apply
  return check_dims(d);
}

// N, the most rows of a sequence, is a promise of any size: no more than all T rows count, and
// what is worked out from it then fits its types and no unit lies past the rows
int bounded_rows(int N, int T) { return N < T ? N : T; }

int check_attend_dims(const gdn_tree_attend_dims& d) {
  if (d.B < 0 || d.T < 0 || d.N < 0 || d.Hq <= 0 || d.Hkv <= 0 || d.D <= 0 || d.page_size < 1 ||
      d.n_pages < 0 || d.table_width < 0 || d.prefix_len < 0)
    return GDN_TREE_EINVAL;
  if (d.Hq % d.Hkv != 0) return GDN_TREE_EINVAL;
  if (d.dtype != GDN_TREE_BF16 && d.dtype != GDN_TREE_F32) return GDN_TREE_EUNSUPPORTED;
  if (!supported_head_dim(d.D) || d.B > 65535) return GDN_TREE_EUNSUPPORTED;
  // positions within a sequence, rows of the cache and of a key head's query block are
  // 32-bit numbers (element offsets are not)
  if ((long long)d.n_pages * d.page_size > 0x7fffffffll ||
      (long long)d.table_width * d.page_size > 0x7fffffffll - 4096 ||
      d.prefix_len > 0x7fffffff - 4096 || (long long)d.T * d.Hq > 0x7fffffffll - 4096 ||
      (long long)d.Hkv * d.D > 0x7fffffffll / 8)
    return GDN_TREE_EUNSUPPORTED;
  return GDN_TREE_OK;
}

// T rows of H heads of `width` bytes, `row` and `head` bytes apart
struct HeadRows {
  const char* p;
  long long row, head, T, H, width;

  bool any() const { return p != nullptr && T > 0 && H > 0; }
  long long span() const { return (H - 1) * head + width; }  // of a row
  bool same(const HeadRows& o) const {
    return p == o.p && row == o.row && head == o.head && T == o.T && H == o.H;
  }
  size_t extent() const { return any() ? (size_t)((T - 1) * row + span()) : 0; }
  // no two heads of it share a byte
  bool apart() const {
    return T * H <= 1 || (head >= width && (T == 1 || row >= span())) || (H == 1 && row >= width) ||
           (row >= width && head >= (T - 1) * row + width);
  }
};

// two arrays of heads share no byte (as far as their extents, or equal strides, tell)
bool disjoint(const HeadRows& a, const HeadRows& b) {
  if (!a.any() || !b.any() || !any_overlap(a.p, a.extent(), b.p, b.extent())) return true;
  const auto beside = [](long long off, long long period, long long wa, long long wb) {
    off = ((off % period) + period) % period;
    return off >= wa && off + wb <= period;
  };
  const long long off = b.p - a.p;
  // columns of the same rows
  const bool rows = a.T > 1 && b.T > 1;
  if (rows && a.row == b.row && a.span() <= a.row && b.span() <= a.row &&
      beside(off, a.row, a.span(), b.span()))
    return true;
  // columns of the same heads (of one row, or of rows of whole heads)
  return a.H > 1 && b.H > 1 && a.head == b.head && a.head > 0 &&
         (a.T == 1 || a.row % a.head == 0) && (b.T == 1 || b.row % a.head == 0) &&
         beside(off, a.head, a.width, b.width);
}

// fills `out` from a pointer and strides in elements; strides of no array, or that step over a
// single row or head, do not count.  Misaligned or negative ones, or strides out of range, are
// refused.
int check_heads(const void* p, gdn_tree_strides* s, int T, int H, int D, int dtype,
                HeadRows* out) {
  const long long es = dtype == GDN_TREE_BF16 ? 2 : 4;
  if (T <= 1 || p == nullptr) s->row = 0;
  if (H <= 1 || p == nullptr) s->head = 0;
  if (!aligned16(p) || s->row < 0 || s->head < 0 || s->row % (16 / es) || s->head % (16 / es))
    return GDN_TREE_EINVAL;
  // (offsets, in bytes, stay within 63 bits)
  if (s->row > (1ll << 60) / (T > 0 ? T : 1) / es || s->head > (1ll << 60) / (H > 0 ? H : 1) / es)
    return GDN_TREE_EUNSUPPORTED;
  *out = HeadRows{static_cast<const char*>(p), s->row * es, s->head * es, T, H, D * es};
  return GDN_TREE_OK;
}

int check_rope(const gdn_tree_attend_dims& d, const gdn_tree_rope& r, const uint64_t* freq,
               const float* q_weight, const float* k_weight) {
  if (d.T < 0) return GDN_TREE_EINVAL;
  if (d.dtype != GDN_TREE_BF16 && d.dtype != GDN_TREE_F32) return GDN_TREE_EUNSUPPORTED;
  if (!supported_head_dim(d.D)) return GDN_TREE_EUNSUPPORTED;
  if (d.T > 0x7fffffff - 4096) return GDN_TREE_EUNSUPPORTED;  // (a unit's number fits 32 bits)
  if (r.rotary_dim < 0 || r.rotary_dim > d.D || r.rotary_dim % 2 || r.interleaved < 0 ||
      r.interleaved > 1 || r.norm < GDN_TREE_NORM_NONE || r.norm > GDN_TREE_NORM_UNIT)
    return GDN_TREE_EINVAL;
  if (r.norm != GDN_TREE_NORM_NONE && !(r.eps >= 0.f && r.eps <= 3e38f)) return GDN_TREE_EINVAL;
  if (r.norm == GDN_TREE_NORM_NONE && (q_weight || k_weight)) return GDN_TREE_EINVAL;
  if (r.rotary_dim > 0 && freq == nullptr) return GDN_TREE_EINVAL;
  if ((reinterpret_cast<uintptr_t>(freq) & 7u) || !aligned16(q_weight) || !aligned16(k_weight))
    return GDN_TREE_EINVAL;
  return GDN_TREE_OK;
}

struct Range {
  const void* p;
  size_t bytes;
};

// outputs out[i] of inputs in[i] (in place, or apart from every array of the call)
int check_apart(const HeadRows* in, const HeadRows* out, int n, const Range* others, int m) {
  for (int i = 0; i < n; ++i) {
    if (!out[i].any()) continue;
    if (!out[i].apart()) return GDN_TREE_EINVAL;
    for (int j = 0; j < n; ++j) {
      if (!(i == j && out[i].same(in[j])) && !disjoint(out[i], in[j])) return GDN_TREE_EINVAL;
      if (i < j && !disjoint(out[i], out[j])) return GDN_TREE_EINVAL;
    }
    for (int j = 0; j < m; ++j)
      if (others[j].p && any_overlap(out[i].p, out[i].extent(), others[j].p, others[j].bytes))
        return GDN_TREE_EINVAL;
  }
  return GDN_TREE_OK;
}

// heads of a row of the calls in front of the attention (a warp's share of them is counted in
// 32 bits, and no model has more)
constexpr int kMostHeads = 1 << 20;

// Per-sequence status words start at GDN_TREE_STATUS_OK; the kernels raise
// them with atomicMax, so that no unit's report can be lost to another's.
cudaError_t clear_status(int32_t* st, int B, cudaStream_t stream) {
  return st ? cudaMemsetAsync(st, 0, (size_t)B * sizeof(int32_t), stream) : cudaSuccess;
}

}  // namespace

namespace gdn {

WaitHooks wait_hooks() {
  WaitHooks h;
  if (const char* e = getenv("GDN_TREE_TEST_WAIT_LIMIT_NS")) {
    const unsigned long long v = strtoull(e, nullptr, 10);
    if (v > 0 && v < h.limit_ns) h.limit_ns = v;
  }
  if (const char* e = getenv("GDN_TREE_TEST_WITHHOLD_COPY")) h.withhold_copy_seq = atoi(e);
  if (const char* e = getenv("GDN_TREE_TEST_WITHHOLD_NODE")) {
    int u = -1, n = -1;
    if (sscanf(e, "%d:%d", &u, &n) == 2) {
      h.withhold_unit = u;
      h.withhold_node = n;
    }
  }
  return h;
}

// GDN_TREE_KERNEL=generic forces the general CUDA-core kernel, =mid the
// 256-node bf16 one, =long the chunked pass (its tensor-core form where it takes
// the shape) and =long_cuda the chunked pass on CUDA cores (used by the tests to
// cover every kernel on the same shapes); the default picks the tensor-core
// kernel whenever it takes the shape, then the 256-node bf16 kernel, the general
// on-chip kernel up to kMaxNHost nodes and the chunked pass beyond.
static bool kernel_forced(const char* name) {
  const char* e = getenv("GDN_TREE_KERNEL");
  return e && strcmp(e, name) == 0;
}
static bool long_forced() { return kernel_forced("long") || kernel_forced("long_cuda"); }
static bool force_generic() {
  return kernel_forced("generic") || long_forced() || kernel_forced("mid");
}

// the tensor-core kernel takes the shape (packed rows: at least one row, for its
// tensor maps)
static bool tc_takes(const VerifyArgs& a) {
  return !force_generic() && verify_tc_supported(a.d) && (!a.lay.packed() || a.lay.T > 0);
}

// past 128 nodes (bf16, d = 128) the units whose tree is one chain take the
// chunkwise path inside the 256-node kernel or the chunk pass
bool verify_chain_path_fits(const gdn_tree_dims& d) {
  return d.dtype == GDN_TREE_BF16 && d.dk == 128 && d.dv == 128 && d.N >= 1 &&
         d.N <= kMaxNLongHost && chain::smem_bytes(d.N) <= 227 * 1024;
}

cudaError_t launch_verify(const VerifyArgs& a, cudaStream_t stream) {
  if (tc_takes(a)) return launch_verify_tc(a, stream);
  VerifyArgs t = a;
  const bool forced = getenv("GDN_TREE_KERNEL") && *getenv("GDN_TREE_KERNEL") &&
                      !kernel_forced("auto");
  const bool mid = !kernel_forced("generic") && !long_forced() && verify_mid_supported(a.d);
  const bool long_tc = (a.d.N > kMaxNHost || long_forced()) && !kernel_forced("long_cuda") &&
                       !kernel_forced("generic") && verify_long_tc_supported(a.d);
  t.chains = !forced && verify_chain_path_fits(a.d);
  if (mid) return launch_verify_mid(t, stream);
  if (long_tc) return launch_verify_long_tc(t, stream);
  if (a.d.N > kMaxNHost || long_forced()) return launch_verify_long(a, stream);
  return launch_verify_generic(a, stream);
}

// paths of more than 32 entries take the tensor-core commit (the rank-L update is
// then real work: a chain's 256-entry path is ~1 M FMAs a 32-row block); shorter
// ones the CUDA-core kernel, whose warps hide the gathers' latency better
cudaError_t launch_commit(const CommitArgs& a, cudaStream_t stream) {
  if (!kernel_forced("generic") && a.Lmax > 32 && commit_tc_supported(a.d, a.Lmax))
    return launch_commit_tc(a, stream);
  return launch_commit_warp(a, stream);
}

cudaError_t launch_commit_verify(const CommitVerifyArgs& a, cudaStream_t stream) {
  if (tc_takes(a.verify) && commit_verify_tc_supported(a.verify.d, a.prev_N, a.Lmax))
    return launch_commit_verify_tc(a, stream);
  // two launches on the same stream: commit S_prev -> S1, then verify from S1
  gdn_tree_dims dp = a.verify.d;
  dp.N = a.prev_N;
  SeqLayout cl = a.prev_lay;  // the previous tree's rows, the verification's state slots
  cl.slot = a.verify.lay.slot;
  cl.n_slots = a.verify.lay.n_slots;
  const CommitArgs c{a.prev_path, a.prev_path_len, a.prev_parent, a.prev_U, a.prev_k,
                     a.prev_log_alpha, a.S_prev, a.S1, dp, a.Lmax, a.commit_status, cl};
  cudaError_t err = launch_commit(c, stream);
  if (err != cudaSuccess) return err;
  VerifyArgs v = a.verify;
  v.S0 = a.S1;
  return launch_verify(v, stream);
}

}  // namespace gdn

extern "C" {

int gdn_tree_verify(const void* q, const void* k, const void* v, const float* log_alpha,
                    const float* beta, const int32_t* parent, const float* S0, void* o,
                    float* U, gdn_tree_dims dims, int32_t* dev_status, void* stream) {
  const int rc = check_dims(dims);
  if (rc != GDN_TREE_OK) return rc;
  if (dims.B == 0 || dims.N == 0) return GDN_TREE_OK;  // nothing to do
  const void* ptrs[] = {q, k, v, log_alpha, beta, parent, S0, o, U};
  for (const void* p : ptrs)
    if (p == nullptr || !aligned16(p)) return GDN_TREE_EINVAL;
  if (dev_status && (reinterpret_cast<uintptr_t>(dev_status) & 3u)) return GDN_TREE_EINVAL;
  gdn::VerifyArgs a{q, k, v, log_alpha, beta, parent, S0, o, U, dims, dev_status};
  if (clear_status(dev_status, dims.B, static_cast<cudaStream_t>(stream)) != cudaSuccess)
    return GDN_TREE_ECUDA;
  const cudaError_t err = gdn::launch_verify(a, static_cast<cudaStream_t>(stream));
  return err == cudaSuccess ? GDN_TREE_OK : GDN_TREE_ECUDA;
}

int gdn_tree_verify_recurrent(const void* q, const void* k, const void* v,
                              const float* log_alpha, const float* beta,
                              const int32_t* parent, const float* S0, void* o, float* U,
                              gdn_tree_dims dims, int32_t* dev_status, void* stream) {
  const int rc = check_dims(dims);
  if (rc != GDN_TREE_OK) return rc;
  if (dims.N > gdn::kMaxNHost) return GDN_TREE_EUNSUPPORTED;  // the path table is on chip
  if (dims.B == 0 || dims.N == 0) return GDN_TREE_OK;  // nothing to do
  const void* ptrs[] = {q, k, v, log_alpha, beta, parent, S0, o, U};
  for (const void* p : ptrs)
    if (p == nullptr || !aligned16(p)) return GDN_TREE_EINVAL;
  if (dev_status && (reinterpret_cast<uintptr_t>(dev_status) & 3u)) return GDN_TREE_EINVAL;
  if (dims.Hv > 65535) return GDN_TREE_EUNSUPPORTED;  // the grid's y dimension
  gdn::VerifyArgs a{q, k, v, log_alpha, beta, parent, S0, o, U, dims, dev_status};
  if (clear_status(dev_status, dims.B, static_cast<cudaStream_t>(stream)) != cudaSuccess)
    return GDN_TREE_ECUDA;
  const cudaError_t err = gdn::launch_verify_recurrent(a, static_cast<cudaStream_t>(stream));
  return err == cudaSuccess ? GDN_TREE_OK : GDN_TREE_ECUDA;
}

int gdn_tree_commit(const int32_t* path, const int32_t* path_len, const int32_t* parent,
                    const float* U, const void* k, const float* log_alpha, const float* S0,
                    float* S1, gdn_tree_dims dims, int32_t Lmax, int32_t* dev_status,
                    void* stream) {
  const int rc = check_dims(dims);
  if (rc != GDN_TREE_OK) return rc;
  if (Lmax < 0) return GDN_TREE_EINVAL;
  if (dims.B == 0) return GDN_TREE_OK;
  if (Lmax > gdn::kMaxNLongHost) return GDN_TREE_EUNSUPPORTED;
  const void* ptrs[] = {path_len, U, k, log_alpha, S0, S1};
  for (const void* p : ptrs)
    if (p == nullptr || !aligned16(p)) return GDN_TREE_EINVAL;
  if (Lmax > 0 && (path == nullptr || (reinterpret_cast<uintptr_t>(path) & 3u)))
    return GDN_TREE_EINVAL;
  if (parent && (reinterpret_cast<uintptr_t>(parent) & 3u)) return GDN_TREE_EINVAL;
  if (dev_status && (reinterpret_cast<uintptr_t>(dev_status) & 3u)) return GDN_TREE_EINVAL;
  // S1 may be S0 exactly; a partial overlap would race between CTAs
  const size_t bytes = (size_t)dims.B * dims.Hv * dims.dk * dims.dv * sizeof(float);
  const char* a0 = reinterpret_cast<const char*>(S0);
  const char* a1 = reinterpret_cast<const char*>(S1);
  if (a0 != a1 && a0 < a1 + bytes && a1 < a0 + bytes) return GDN_TREE_EINVAL;
  gdn::CommitArgs a{path, path_len, parent, U, k, log_alpha, S0, S1, dims, Lmax, dev_status};
  if (clear_status(dev_status, dims.B, static_cast<cudaStream_t>(stream)) != cudaSuccess)
    return GDN_TREE_ECUDA;
  const cudaError_t err = gdn::launch_commit(a, static_cast<cudaStream_t>(stream));
  return err == cudaSuccess ? GDN_TREE_OK : GDN_TREE_ECUDA;
}

int gdn_tree_commit_verify(const int32_t* prev_path, const int32_t* prev_path_len,
                           const int32_t* prev_parent, const float* prev_U, const void* prev_k,
                           const float* prev_log_alpha, int32_t prev_N, int32_t Lmax,
                           const float* S_prev, float* S1, const void* q, const void* k,
                           const void* v, const float* log_alpha, const float* beta,
                           const int32_t* parent, void* o, float* U, gdn_tree_dims dims,
                           int32_t* commit_status, int32_t* verify_status, void* stream) {
  int rc = check_dims(dims);
  if (rc != GDN_TREE_OK) return rc;
  gdn_tree_dims dp = dims;
  dp.N = prev_N;
  if (prev_N < 0 || Lmax < 0) return GDN_TREE_EINVAL;
  rc = check_dims(dp);
  if (rc != GDN_TREE_OK) return rc;
  if (Lmax > gdn::kMaxNLongHost) return GDN_TREE_EUNSUPPORTED;
  if (dims.B == 0) return GDN_TREE_OK;
  if (prev_N == 0 || dims.N == 0) return GDN_TREE_EUNSUPPORTED;
  const void* ptrs[] = {prev_path_len, prev_U, prev_k, prev_log_alpha, S_prev, S1,
                        q, k, v, log_alpha, beta, parent, o, U};
  for (const void* p : ptrs)
    if (p == nullptr || !aligned16(p)) return GDN_TREE_EINVAL;
  if (Lmax > 0 && (prev_path == nullptr || (reinterpret_cast<uintptr_t>(prev_path) & 3u)))
    return GDN_TREE_EINVAL;
  const void* small[] = {prev_parent, commit_status, verify_status};
  for (const void* p : small)
    if (p && (reinterpret_cast<uintptr_t>(p) & 3u)) return GDN_TREE_EINVAL;
  const size_t sbytes = (size_t)dims.B * dims.Hv * dims.dk * dims.dv * sizeof(float);
  const char* a0 = reinterpret_cast<const char*>(S_prev);
  const char* a1 = reinterpret_cast<const char*>(S1);
  if (a0 != a1 && a0 < a1 + sbytes && a1 < a0 + sbytes) return GDN_TREE_EINVAL;
  // U may be prev_U itself only when both trees have the same node count: then
  // each (b, h) slice sits at the same place in both and is read before it is
  // written.  Any other overlap would let one unit's U rows land on another
  // unit's previous rows before those are read.
  const size_t ubytes = (size_t)dims.B * dims.Hv * dims.N * dims.dv * sizeof(float);
  const size_t pubytes = (size_t)dims.B * dims.Hv * prev_N * dims.dv * sizeof(float);
  if (!(U == prev_U && prev_N == dims.N) && any_overlap(U, ubytes, prev_U, pubytes))
    return GDN_TREE_EINVAL;
  gdn::CommitVerifyArgs a{prev_path, prev_path_len, prev_parent, prev_U, prev_k, prev_log_alpha,
                          prev_N, Lmax, S_prev, S1, commit_status,
                          gdn::VerifyArgs{q, k, v, log_alpha, beta, parent, S1, o, U, dims,
                                          verify_status}};
  if (clear_status(commit_status, dims.B, static_cast<cudaStream_t>(stream)) != cudaSuccess ||
      clear_status(verify_status, dims.B, static_cast<cudaStream_t>(stream)) != cudaSuccess)
    return GDN_TREE_ECUDA;
  const cudaError_t err = gdn::launch_commit_verify(a, static_cast<cudaStream_t>(stream));
  return err == cudaSuccess ? GDN_TREE_OK : GDN_TREE_ECUDA;
}

int gdn_tree_verify_packed(const void* q, const void* k, const void* v, const float* log_alpha,
                           const float* beta, const int32_t* parent, const int32_t* cu_nodes,
                           int32_t T, const float* state_pool, const int32_t* state_slot,
                           int32_t n_slots, void* o, float* U, gdn_tree_dims dims,
                           int32_t* dev_status, void* stream) {
  int rc = check_dims(dims);
  if (rc != GDN_TREE_OK) return rc;
  gdn::SeqLayout lay;
  rc = check_packed(cu_nodes, T, state_slot, n_slots, dims.B, &lay);
  if (rc != GDN_TREE_OK) return rc;
  if (dims.B == 0 || dims.N == 0) return GDN_TREE_OK;  // nothing to do
  const void* ptrs[] = {q, k, v, log_alpha, beta, parent, state_pool, o, U};
  for (const void* p : ptrs)
    if (p == nullptr || !aligned16(p)) return GDN_TREE_EINVAL;
  if (dev_status && !aligned4(dev_status)) return GDN_TREE_EINVAL;
  gdn::VerifyArgs a{q, k, v, log_alpha, beta, parent, state_pool, o, U, dims, dev_status, lay};
  if (clear_status(dev_status, dims.B, static_cast<cudaStream_t>(stream)) != cudaSuccess)
    return GDN_TREE_ECUDA;
  const cudaError_t err = gdn::launch_verify(a, static_cast<cudaStream_t>(stream));
  return err == cudaSuccess ? GDN_TREE_OK : GDN_TREE_ECUDA;
}

int gdn_tree_commit_packed(const int32_t* path, const int32_t* path_len, const int32_t* parent,
                           const int32_t* cu_nodes, int32_t T, const float* U, const void* k,
                           const float* log_alpha, const float* pool_in, float* pool_out,
                           const int32_t* state_slot, int32_t n_slots, gdn_tree_dims dims,
                           int32_t Lmax, int32_t* dev_status, void* stream) {
  int rc = check_dims(dims);
  if (rc != GDN_TREE_OK) return rc;
  gdn::SeqLayout lay;
  rc = check_packed(cu_nodes, T, state_slot, n_slots, dims.B, &lay);
  if (rc != GDN_TREE_OK) return rc;
  if (Lmax < 0) return GDN_TREE_EINVAL;
  if (dims.B == 0) return GDN_TREE_OK;
  if (Lmax > gdn::kMaxNLongHost) return GDN_TREE_EUNSUPPORTED;
  const void* ptrs[] = {path_len, pool_in, pool_out};
  for (const void* p : ptrs)
    if (p == nullptr || !aligned16(p)) return GDN_TREE_EINVAL;
  if (T > 0) {
    const void* rows[] = {U, k, log_alpha};
    for (const void* p : rows)
      if (p == nullptr || !aligned16(p)) return GDN_TREE_EINVAL;
  }
  if (Lmax > 0 && (path == nullptr || !aligned4(path))) return GDN_TREE_EINVAL;
  if (parent && !aligned4(parent)) return GDN_TREE_EINVAL;
  if (dev_status && !aligned4(dev_status)) return GDN_TREE_EINVAL;
  const int slots = state_slot ? n_slots : dims.B;
  if (partial_overlap(pool_in, pool_out, (size_t)slots * dims.Hv * dims.dk * dims.dv * 4))
    return GDN_TREE_EINVAL;
  gdn::CommitArgs a{path, path_len, parent, U, k, log_alpha, pool_in, pool_out,
                    dims, Lmax, dev_status, lay};
  if (clear_status(dev_status, dims.B, static_cast<cudaStream_t>(stream)) != cudaSuccess)
    return GDN_TREE_ECUDA;
  const cudaError_t err = gdn::launch_commit(a, static_cast<cudaStream_t>(stream));
  return err == cudaSuccess ? GDN_TREE_OK : GDN_TREE_ECUDA;
}

int gdn_tree_commit_verify_packed(const int32_t* prev_path, const int32_t* prev_path_len,
                                  const int32_t* prev_parent, const int32_t* prev_cu_nodes,
                                  int32_t prev_T, const float* prev_U, const void* prev_k,
                                  const float* prev_log_alpha, int32_t prev_N, int32_t Lmax,
                                  const float* pool_in, float* pool_out,
                                  const int32_t* state_slot, int32_t n_slots, const void* q,
                                  const void* k, const void* v, const float* log_alpha,
                                  const float* beta, const int32_t* parent,
                                  const int32_t* cu_nodes, int32_t T, void* o, float* U,
                                  gdn_tree_dims dims, int32_t* commit_status,
                                  int32_t* verify_status, void* stream) {
  int rc = check_dims(dims);
  if (rc != GDN_TREE_OK) return rc;
  gdn_tree_dims dp = dims;
  dp.N = prev_N;
  if (prev_N < 0 || Lmax < 0) return GDN_TREE_EINVAL;
  rc = check_dims(dp);
  if (rc != GDN_TREE_OK) return rc;
  gdn::SeqLayout lay, prev_lay;
  rc = check_packed(cu_nodes, T, state_slot, n_slots, dims.B, &lay);
  if (rc != GDN_TREE_OK) return rc;
  rc = check_packed(prev_cu_nodes, prev_T, state_slot, n_slots, dims.B, &prev_lay);
  if (rc != GDN_TREE_OK) return rc;
  if (Lmax > gdn::kMaxNLongHost) return GDN_TREE_EUNSUPPORTED;
  if (dims.B == 0) return GDN_TREE_OK;
  if (prev_N == 0 || dims.N == 0) return GDN_TREE_EUNSUPPORTED;
  const void* ptrs[] = {prev_path_len, prev_U, prev_k, prev_log_alpha, pool_in, pool_out,
                        q, k, v, log_alpha, beta, parent, o, U};
  for (const void* p : ptrs)
    if (p == nullptr || !aligned16(p)) return GDN_TREE_EINVAL;
  if (Lmax > 0 && (prev_path == nullptr || !aligned4(prev_path))) return GDN_TREE_EINVAL;
  const void* small[] = {prev_parent, commit_status, verify_status};
  for (const void* p : small)
    if (p && !aligned4(p)) return GDN_TREE_EINVAL;
  const int slots = state_slot ? n_slots : dims.B;
  if (partial_overlap(pool_in, pool_out, (size_t)slots * dims.Hv * dims.dk * dims.dv * 4))
    return GDN_TREE_EINVAL;
  // the next tree's U must not overlap the previous one's (their row ranges differ)
  if (any_overlap(U, (size_t)dims.Hv * T * dims.dv * 4, prev_U,
                  (size_t)dims.Hv * prev_T * dims.dv * 4))
    return GDN_TREE_EINVAL;
  gdn::CommitVerifyArgs a{prev_path, prev_path_len, prev_parent, prev_U, prev_k, prev_log_alpha,
                          prev_N, Lmax, pool_in, pool_out, commit_status,
                          gdn::VerifyArgs{q, k, v, log_alpha, beta, parent, pool_out, o, U, dims,
                                          verify_status, lay},
                          prev_lay};
  if (clear_status(commit_status, dims.B, static_cast<cudaStream_t>(stream)) != cudaSuccess ||
      clear_status(verify_status, dims.B, static_cast<cudaStream_t>(stream)) != cudaSuccess)
    return GDN_TREE_ECUDA;
  const cudaError_t err = gdn::launch_commit_verify(a, static_cast<cudaStream_t>(stream));
  return err == cudaSuccess ? GDN_TREE_OK : GDN_TREE_ECUDA;
}

int gdn_tree_build_topw(const float* cand_logp, int32_t B, int32_t N, int32_t c, int32_t w,
                        int32_t max_depth, int32_t* parent, int32_t* cand_index, float* score,
                        int32_t* n_built, void* stream) {
  if (B < 0 || N < 1 || c < 1 || w < 1 || max_depth < 1) return GDN_TREE_EINVAL;
  if (N > gdn::kMaxNHost || c > 32 || w > N) return GDN_TREE_EUNSUPPORTED;
  if (B == 0) return GDN_TREE_OK;
  if (cand_logp == nullptr || parent == nullptr || !aligned4(cand_logp) || !aligned4(parent))
    return GDN_TREE_EINVAL;
  const void* opt[] = {cand_index, score, n_built};
  for (const void* p : opt)
    if (p && !aligned4(p)) return GDN_TREE_EINVAL;
  const cudaError_t err = gdn::launch_tree_topw(cand_logp, B, N, c, w, max_depth, parent,
                                                cand_index, score, n_built,
                                                static_cast<cudaStream_t>(stream));
  return err == cudaSuccess ? GDN_TREE_OK : GDN_TREE_ECUDA;
}

static int rule_call(const void* q, const void* k, const void* v, const float* log_alpha,
                     const float* beta, const float* pool_in, float* pool_out, void* o,
                     const gdn_tree_dims& dims, const gdn::SeqLayout& lay, int32_t T,
                     int32_t* dev_status, bool step, void* workspace, size_t workspace_bytes,
                     void* stream) {
  const void* ptrs[] = {pool_in, pool_out};
  for (const void* p : ptrs)
    if (p == nullptr || !aligned16(p)) return GDN_TREE_EINVAL;
  const void* rows[] = {q, k, v, log_alpha, beta, o};
  for (const void* p : rows)
    if ((p == nullptr && T > 0) || !aligned16(p)) return GDN_TREE_EINVAL;
  if (dev_status && !aligned4(dev_status)) return GDN_TREE_EINVAL;
  const int slots = lay.slot ? lay.n_slots : dims.B;
  if (partial_overlap(pool_in, pool_out, (size_t)slots * dims.Hv * dims.dk * dims.dv * 4))
    return GDN_TREE_EINVAL;
  const size_t want = step ? 0 : gdn::prefill_workspace_bytes(dims, T);
  if (want > 0 && (workspace == nullptr || !aligned16(workspace) || workspace_bytes < want))
    return GDN_TREE_EINVAL;
  const gdn::RuleArgs a{q, k, v, log_alpha, beta, pool_in, pool_out, o, dims, dev_status, lay};
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (clear_status(dev_status, dims.B, st) != cudaSuccess) return GDN_TREE_ECUDA;
  const cudaError_t err = step ? gdn::launch_decode_step(a, st) : gdn::launch_prefill(a, workspace, st);
  return err == cudaSuccess ? GDN_TREE_OK : GDN_TREE_ECUDA;
}

int gdn_tree_prefill(const void* q, const void* k, const void* v, const float* log_alpha,
                     const float* beta, const int32_t* cu_tokens, int32_t T,
                     const float* pool_in, float* pool_out, const int32_t* state_slot,
                     int32_t n_slots, void* o, gdn_tree_dims dims, int32_t* dev_status,
                     void* workspace, size_t workspace_bytes, void* stream) {
  int rc = check_rule_dims(dims);
  if (rc != GDN_TREE_OK) return rc;
  gdn::SeqLayout lay;
  rc = check_packed(cu_tokens, T, state_slot, n_slots, dims.B, &lay);
  if (rc != GDN_TREE_OK) return rc;
  if (dims.B == 0) return GDN_TREE_OK;  // nothing to do
  dims.N = bounded_rows(dims.N, T);
  return rule_call(q, k, v, log_alpha, beta, pool_in, pool_out, o, dims, lay, T, dev_status,
                   false, workspace, workspace_bytes, stream);
}

size_t gdn_tree_prefill_workspace(gdn_tree_dims dims, int32_t T) {
  if (check_rule_dims(dims) != GDN_TREE_OK || dims.B == 0 || T <= 0) return 0;
  dims.N = bounded_rows(dims.N, T);
  return gdn::prefill_workspace_bytes(dims, T);
}

int gdn_tree_decode_step(const void* q, const void* k, const void* v, const float* log_alpha,
                         const float* beta, const float* pool_in, float* pool_out,
                         const int32_t* state_slot, int32_t n_slots, void* o,
                         gdn_tree_dims dims, int32_t* dev_status, void* stream) {
  dims.N = 1;
  const int rc = check_rule_dims(dims);
  if (rc != GDN_TREE_OK) return rc;
  if (n_slots < 0 || (state_slot == nullptr && n_slots < dims.B)) return GDN_TREE_EINVAL;
  if (state_slot != nullptr && !aligned4(state_slot)) return GDN_TREE_EINVAL;
  if (dims.B == 0) return GDN_TREE_OK;  // nothing to do
  gdn::SeqLayout lay;
  lay.slot = state_slot;
  lay.n_slots = n_slots;
  return rule_call(q, k, v, log_alpha, beta, pool_in, pool_out, o, dims, lay, dims.B, dev_status,
                   true, nullptr, 0, stream);
}

size_t gdn_tree_attend_workspace(gdn_tree_attend_dims dims) {
  if (check_attend_dims(dims) != GDN_TREE_OK || dims.B == 0 || dims.T == 0) return 0;
  dims.N = bounded_rows(dims.N, dims.T);
  return gdn::attend_workspace_bytes(dims);
}

int gdn_tree_attend(const void* q, const void* k, const void* v, const int32_t* parent,
                    const int32_t* cu_nodes, const void* k_cache, const void* v_cache,
                    const int32_t* page_table, const int32_t* context_len,
                    const int32_t* prefix_pages, float scale, void* o, float* lse,
                    gdn_tree_attend_dims dims, int32_t* dev_status, void* workspace,
                    size_t workspace_bytes, void* stream) {
  const int rc = check_attend_dims(dims);
  if (rc != GDN_TREE_OK) return rc;
  if (parent && dims.N > gdn::kMaxNLongHost) return GDN_TREE_EUNSUPPORTED;
  if (dims.B == 0) return GDN_TREE_OK;  // nothing to do
  if (dev_status && !aligned4(dev_status)) return GDN_TREE_EINVAL;
  if (dims.T == 0)  // nothing but the statuses
    return clear_status(dev_status, dims.B, static_cast<cudaStream_t>(stream)) == cudaSuccess
               ? GDN_TREE_OK
               : GDN_TREE_ECUDA;
  dims.N = bounded_rows(dims.N, dims.T);
  if ((k == nullptr) != (v == nullptr)) return GDN_TREE_EINVAL;
  const void* need[] = {q, o};
  for (const void* p : need)
    if (p == nullptr || !aligned16(p)) return GDN_TREE_EINVAL;
  // the cache may be absent where no row of it can be seen
  const bool cached = dims.n_pages > 0 && (dims.prefix_len > 0 || dims.table_width > 0);
  const void* cache[] = {k_cache, v_cache};
  for (const void* p : cache)
    if ((cached && p == nullptr) || !aligned16(p)) return GDN_TREE_EINVAL;
  if (!aligned16(k) || !aligned16(v)) return GDN_TREE_EINVAL;
  const void* ints[] = {cu_nodes, context_len};
  for (const void* p : ints)
    if (p == nullptr || !aligned4(p)) return GDN_TREE_EINVAL;
  const void* opt[] = {parent, page_table, prefix_pages, lse};
  for (const void* p : opt)
    if (!aligned4(p)) return GDN_TREE_EINVAL;
  if ((dims.table_width > 0 && page_table == nullptr) ||
      (dims.prefix_len > 0 && prefix_pages == nullptr))
    return GDN_TREE_EINVAL;
  const size_t want = gdn::attend_workspace_bytes(dims);
  if (want > 0 && (workspace == nullptr || !aligned16(workspace) || workspace_bytes < want))
    return GDN_TREE_EINVAL;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (clear_status(dev_status, dims.B, st) != cudaSuccess) return GDN_TREE_ECUDA;
  const gdn::AttendArgs a{q, k, v, parent, cu_nodes, k_cache, v_cache, page_table, context_len,
                          prefix_pages, scale, o, lse, dims, dev_status, workspace};
  const cudaError_t err = gdn::launch_attend(a, st);
  return err == cudaSuccess ? GDN_TREE_OK : GDN_TREE_ECUDA;
}

int gdn_tree_cache_append(const void* k, const void* v, const int32_t* path,
                          const int32_t* path_len, int32_t Lmax, const int32_t* cu_nodes,
                          void* k_cache, void* v_cache, const int32_t* page_table,
                          const int32_t* context_len, int32_t* new_len,
                          gdn_tree_attend_dims dims, int32_t* dev_status, void* stream) {
  dims.Hq = dims.Hkv;
  dims.prefix_len = 0;
  const int rc = check_attend_dims(dims);
  if (rc != GDN_TREE_OK) return rc;
  if ((path_len == nullptr) != (path == nullptr) && !(path_len != nullptr && Lmax == 0))
    return GDN_TREE_EINVAL;
  if (path_len != nullptr && Lmax < 0) return GDN_TREE_EINVAL;
  if (dims.B == 0) return GDN_TREE_OK;
  dims.N = bounded_rows(dims.N, dims.T);
  const bool rows = dims.T > 0 && dims.table_width > 0 && dims.n_pages > 0;
  const void* data[] = {k, v, k_cache, v_cache};
  for (const void* p : data)
    if ((rows && p == nullptr) || !aligned16(p)) return GDN_TREE_EINVAL;
  const void* ints[] = {cu_nodes, context_len};
  for (const void* p : ints)
    if (p == nullptr || !aligned4(p)) return GDN_TREE_EINVAL;
  const void* opt[] = {path, path_len, page_table, new_len, dev_status};
  for (const void* p : opt)
    if (!aligned4(p)) return GDN_TREE_EINVAL;
  if (dims.table_width > 0 && page_table == nullptr) return GDN_TREE_EINVAL;
  if (new_len && any_overlap(new_len, (size_t)dims.B * 4, context_len, (size_t)dims.B * 4))
    return GDN_TREE_EINVAL;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (clear_status(dev_status, dims.B, st) != cudaSuccess) return GDN_TREE_ECUDA;
  const gdn::AppendArgs a{k, v, path, path_len, Lmax, cu_nodes, k_cache, v_cache, page_table,
                          context_len, new_len, dims, dev_status};
  const cudaError_t err = gdn::launch_cache_append(a, st);
  return err == cudaSuccess ? GDN_TREE_OK : GDN_TREE_ECUDA;
}

int gdn_tree_norm_rope(const void* q, const void* k, const int32_t* positions,
                       const uint64_t* freq, const float* q_weight, const float* k_weight,
                       void* q_out, void* k_out, gdn_tree_head_strides strides,
                       gdn_tree_attend_dims dims, gdn_tree_rope rope, void* stream) {
  if (q == nullptr) dims.Hq = 0, q_weight = nullptr, q_out = nullptr;
  if (k == nullptr) dims.Hkv = 0, k_weight = nullptr, k_out = nullptr;
  int rc = check_rope(dims, rope, freq, q_weight, k_weight);
  if (rc != GDN_TREE_OK) return rc;
  if ((q != nullptr && dims.Hq <= 0) || (k != nullptr && dims.Hkv <= 0)) return GDN_TREE_EINVAL;
  if (dims.Hq + (long long)dims.Hkv > kMostHeads) return GDN_TREE_EUNSUPPORTED;
  if (!aligned4(positions)) return GDN_TREE_EINVAL;
  if (dims.T == 0) return GDN_TREE_OK;
  if (q == nullptr && k == nullptr) return GDN_TREE_EINVAL;
  if ((q == nullptr) != (q_out == nullptr) || (k == nullptr) != (k_out == nullptr) ||
      (rope.rotary_dim > 0 && positions == nullptr))
    return GDN_TREE_EINVAL;
  HeadRows in[2], out[2];
  const int T = dims.T, D = dims.D, dt = dims.dtype;
  if ((rc = check_heads(q, &strides.q, T, dims.Hq, D, dt, &in[0])) != GDN_TREE_OK ||
      (rc = check_heads(k, &strides.k, T, dims.Hkv, D, dt, &in[1])) != GDN_TREE_OK ||
      (rc = check_heads(q_out, &strides.q_out, T, dims.Hq, D, dt, &out[0])) != GDN_TREE_OK ||
      (rc = check_heads(k_out, &strides.k_out, T, dims.Hkv, D, dt, &out[1])) != GDN_TREE_OK)
    return rc;
  const Range others[] = {{positions, rope.rotary_dim ? (size_t)T * 4 : 0},
                          {freq, (size_t)rope.rotary_dim * 4},
                          {q_weight, (size_t)D * 4},
                          {k_weight, (size_t)D * 4}};
  rc = check_apart(in, out, 2, others, 4);
  if (rc != GDN_TREE_OK) return rc;
  gdn::RopeArgs a{};
  a.q = q, a.k = k, a.q_out = q_out, a.k_out = k_out;
  a.s = strides;
  a.positions = positions;
  a.freq = freq;
  a.q_weight = q_weight;
  a.k_weight = k_weight;
  a.d = dims;
  a.rope = rope;
  const cudaError_t err = gdn::launch_norm_rope(a, static_cast<cudaStream_t>(stream));
  return err == cudaSuccess ? GDN_TREE_OK : GDN_TREE_ECUDA;
}

int gdn_tree_cache_append_rope(const void* q, const void* k, const void* v, const uint64_t* freq,
                               const float* q_weight, const float* k_weight,
                               const int32_t* cu_nodes, void* q_out, void* k_out, void* v_out,
                               void* k_cache, void* v_cache, const int32_t* page_table,
                               const int32_t* context_len, int32_t* new_len,
                               gdn_tree_head_strides strides, gdn_tree_attend_dims dims,
                               gdn_tree_rope rope, int32_t* dev_status, void* stream) {
  const int Hq = q ? dims.Hq : 0;
  if (q == nullptr) q_weight = nullptr, q_out = nullptr;
  if (Hq < 0 || (q != nullptr && Hq == 0)) return GDN_TREE_EINVAL;
  dims.Hq = dims.Hkv;  // (no multiple of Hkv is wanted here)
  int rc = check_attend_dims(dims);
  if (rc != GDN_TREE_OK) return rc;
  dims.Hq = Hq;
  rc = check_rope(dims, rope, freq, q_weight, k_weight);
  if (rc != GDN_TREE_OK) return rc;
  if (dims.Hq + 2ll * dims.Hkv > kMostHeads) return GDN_TREE_EUNSUPPORTED;
  if (dims.B == 0) return GDN_TREE_OK;
  dims.N = bounded_rows(dims.N, dims.T);
  const bool rows = dims.T > 0, paged = rows && dims.table_width > 0 && dims.n_pages > 0;
  if (rows && (k == nullptr || v == nullptr)) return GDN_TREE_EINVAL;
  if (rows && (q == nullptr) != (q_out == nullptr)) return GDN_TREE_EINVAL;
  void* const cache[] = {k_cache, v_cache};
  for (const void* p : cache)
    if ((paged && p == nullptr) || !aligned16(p)) return GDN_TREE_EINVAL;
  const void* ints[] = {cu_nodes, context_len};
  for (const void* p : ints)
    if (p == nullptr || !aligned4(p)) return GDN_TREE_EINVAL;
  const void* opt[] = {page_table, new_len, dev_status};
  for (const void* p : opt)
    if (!aligned4(p)) return GDN_TREE_EINVAL;
  if (dims.table_width > 0 && page_table == nullptr) return GDN_TREE_EINVAL;
  HeadRows in[3], out[3];
  const int T = dims.T, Hkv = dims.Hkv, D = dims.D, dt = dims.dtype;
  if ((rc = check_heads(q, &strides.q, T, Hq, D, dt, &in[0])) != GDN_TREE_OK ||
      (rc = check_heads(k, &strides.k, T, Hkv, D, dt, &in[1])) != GDN_TREE_OK ||
      (rc = check_heads(v, &strides.v, T, Hkv, D, dt, &in[2])) != GDN_TREE_OK ||
      (rc = check_heads(q_out, &strides.q_out, T, Hq, D, dt, &out[0])) != GDN_TREE_OK ||
      (rc = check_heads(k_out, &strides.k_out, T, Hkv, D, dt, &out[1])) != GDN_TREE_OK ||
      (rc = check_heads(v_out, &strides.v_out, T, Hkv, D, dt, &out[2])) != GDN_TREE_OK)
    return rc;
  const size_t one = (size_t)Hkv * D * (dt == GDN_TREE_BF16 ? 2 : 4);
  const size_t held = (size_t)dims.n_pages * dims.page_size * one, B4 = (size_t)dims.B * 4;
  const Range others[] = {{freq, (size_t)rope.rotary_dim * 4},
                          {q_weight, (size_t)D * 4},
                          {k_weight, (size_t)D * 4},
                          {cu_nodes, B4 + 4},
                          {context_len, B4},
                          {page_table, B4 * dims.table_width},
                          {dev_status, B4},
                          {new_len, B4},
                          {v_cache, held},
                          {k_cache, held}};
  constexpr int kOthers = sizeof(others) / sizeof(others[0]);
  rc = check_apart(in, out, 3, others, kOthers);
  if (rc != GDN_TREE_OK) return rc;
  // what else is written: the caches, new_len and dev_status
  for (int w = kOthers - 4; w < kOthers; ++w) {
    if (others[w].p == nullptr) continue;
    for (int j = 0; j < w; ++j)
      if (others[j].p && any_overlap(others[w].p, others[w].bytes, others[j].p, others[j].bytes))
        return GDN_TREE_EINVAL;
    for (const HeadRows& i : in)
      if (any_overlap(others[w].p, others[w].bytes, i.p, i.extent())) return GDN_TREE_EINVAL;
  }
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (clear_status(dev_status, dims.B, st) != cudaSuccess) return GDN_TREE_ECUDA;
  const gdn::RopeArgs a{q, k, v, q_out, k_out, v_out, strides, nullptr, freq, q_weight, k_weight, dims, rope, cu_nodes, page_table,
                        context_len, k_cache, v_cache, new_len, dev_status};
  const cudaError_t err = gdn::launch_cache_append_rope(a, st);
  return err == cudaSuccess ? GDN_TREE_OK : GDN_TREE_ECUDA;
}

int gdn_tree_positions(const int32_t* parent, const int32_t* cu_nodes,
                       const int32_t* context_len, int32_t prefix_len, int32_t* positions,
                       int32_t B, int32_t T, int32_t N, int32_t* dev_status, void* stream) {
  if (B < 0 || T < 0 || N < 0 || prefix_len < 0) return GDN_TREE_EINVAL;
  if (B > 65535 || (parent && N > gdn::kMaxNLongHost)) return GDN_TREE_EUNSUPPORTED;
  if (B == 0) return GDN_TREE_OK;
  if (cu_nodes == nullptr || (T > 0 && positions == nullptr)) return GDN_TREE_EINVAL;
  const void* ints[] = {parent, cu_nodes, context_len, positions, dev_status};
  for (const void* p : ints)
    if (!aligned4(p)) return GDN_TREE_EINVAL;
  const size_t T4 = (size_t)T * 4, B4 = (size_t)B * 4;
  const Range others[] = {{parent, T4}, {cu_nodes, B4 + 4}, {context_len, B4}};
  for (const Range& o : others)
    if (o.p && ((positions && any_overlap(positions, T4, o.p, o.bytes)) ||
                (dev_status && any_overlap(dev_status, B4, o.p, o.bytes))))
      return GDN_TREE_EINVAL;
  if (positions && dev_status && any_overlap(positions, T4, dev_status, B4))
    return GDN_TREE_EINVAL;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (clear_status(dev_status, B, st) != cudaSuccess) return GDN_TREE_ECUDA;
  const gdn::PositionArgs a{parent, cu_nodes, context_len, prefix_len, positions, B, T,
                            bounded_rows(N, T), dev_status};
  const cudaError_t err = gdn::launch_tree_positions(a, st);
  return err == cudaSuccess ? GDN_TREE_OK : GDN_TREE_ECUDA;
}

int gdn_tree_rope_frequencies(int32_t rotary_dim, double base, gdn_tree_rope_stretch stretch,
                              uint64_t* freq, float* scale) {
  const int R = rotary_dim;
  const gdn_tree_rope_stretch& s = stretch;
  const bool bands = s.kind == GDN_TREE_STRETCH_YARN || s.kind == GDN_TREE_STRETCH_BANDS;
  if (R < 2 || R % 2 || !(base > 1.0) || !isfinite(base) || freq == nullptr || scale == nullptr)
    return GDN_TREE_EINVAL;
  if (R > gdn::kMaxDHost || s.kind < GDN_TREE_STRETCH_NONE || s.kind > GDN_TREE_STRETCH_BANDS)
    return GDN_TREE_EUNSUPPORTED;
  if (s.kind != GDN_TREE_STRETCH_NONE && !(s.factor >= 1.0 && isfinite(s.factor)))
    return GDN_TREE_EINVAL;
  if (s.kind == GDN_TREE_STRETCH_NTK && R == 2) return GDN_TREE_EINVAL;
  if (bands && !(s.trained_len > 0.0 && isfinite(s.trained_len) && s.slow > 0.0 &&
                 s.fast > s.slow && isfinite(s.fast)))
    return GDN_TREE_EINVAL;
  const double kTurn = 6.283185307179586476925;  // 2 pi
  if (s.kind == GDN_TREE_STRETCH_NTK) base *= pow(s.factor, (double)R / (R - 2));
  // the number of the pair that turns `turns` times within the trained length
  const auto pair_of = [&](double turns) {
    return R * log(s.trained_len / (kTurn * turns)) / (2.0 * log(base));
  };
  double lo = 0.0, hi = 0.0;
  if (s.kind == GDN_TREE_STRETCH_YARN) {
    lo = fmax(floor(pair_of(s.fast)), 0.0);
    hi = fmin(ceil(pair_of(s.slow)), R - 1.0);
  }
  for (int i = 0; i < R / 2; ++i) {
    double f = pow(base, -2.0 * i / R);
    double slow = s.kind == GDN_TREE_STRETCH_LINEAR ? 1.0 : 0.0;  // how much of it is slowed down
    if (s.kind == GDN_TREE_STRETCH_YARN)
      slow = hi > lo ? fmin(fmax((i - lo) / (hi - lo), 0.0), 1.0) : i >= hi;  // (else all of a kind)
    if (s.kind == GDN_TREE_STRETCH_BANDS)
      slow = 1.0 - fmin(fmax((s.trained_len * f / kTurn - s.slow) / (s.fast - s.slow), 0.0), 1.0);
    if (slow > 0.0) f = f * (1.0 - slow) + f / s.factor * slow;
    // (below 2^63: f is at most 1, a sixth of a turn)
    freq[i] = (uint64_t)llround(ldexp(f / kTurn, 64));
  }
  *scale = s.kind == GDN_TREE_STRETCH_YARN ? (float)(0.1 * log(s.factor) + 1.0) : 1.f;
  return GDN_TREE_OK;
}

const char* gdn_tree_strerror(int code) {
  switch (code) {
    case GDN_TREE_OK: return "ok";
    case GDN_TREE_EINVAL: return "invalid argument (NULL or misaligned pointer, bad dims)";
    case GDN_TREE_EUNSUPPORTED: return "unsupported shape or dtype";
    case GDN_TREE_ECUDA: return "CUDA launch failed";
    case GDN_TREE_STATUS_BAD_TREE: return "device status: parent[] is not topologically ordered";
    case GDN_TREE_STATUS_BAD_PATH: return "device status: accepted path is invalid";
    case GDN_TREE_STATUS_TIMEOUT: return "device status: an on-device wait timed out";
    case GDN_TREE_STATUS_BAD_LAYOUT:
      return "device status: the sequence's packed row range or state slot is out of range";
    default: return "unknown code";
  }
}

int gdn_tree_version(void) { return 100; }

}  // extern "C"
