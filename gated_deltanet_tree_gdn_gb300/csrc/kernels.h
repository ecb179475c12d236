// kernels.h -- internal launch interface between the C-ABI layer and the
// kernels of libgdntree (not installed, not part of the ABI).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/gdn_tree.h"

namespace gdn {

constexpr int kMaxNHost = 256;       // largest tree of the on-chip kernels
constexpr int kMaxNLongHost = 1024;  // largest tree of the chunked kernel and commit path
constexpr int kMaxDHost = 128;  // largest dk / dv

// Where the rows and the state of sequence b live.
//  - fixed layout (cu == nullptr): every sequence has dims.N nodes; node rows of
//    q, k, v, o, log_alpha, beta, parent are at b * N + t; U is [B, Hv, N, dv].
//  - packed (ragged) layout: sequence b owns rows cu[b] .. cu[b+1] - 1 of the
//    packed arrays ([T, ...]); dims.N is the largest tree; U is [Hv, T, dv].
//  - the state of sequence b is S[slot[b]] of a state pool (slot == nullptr:
//    S[b]); n_slots bounds the slots.
struct SeqLayout {
  const int32_t* cu = nullptr;
  const int32_t* slot = nullptr;
  int32_t T = 0;
  int32_t n_slots = 0;

  __host__ __device__ bool packed() const { return cu != nullptr; }
#ifdef __CUDACC__
  // first row and node count of sequence b (count < 0: invalid offsets)
  __device__ __forceinline__ int row0(int b, int N) const { return cu ? cu[b] : b * N; }
  __device__ __forceinline__ int count(int b, int N) const {
    if (!cu) return N;
    const int a = cu[b], e = cu[b + 1];
    return (a < 0 || e < a || e > T || e - a > N) ? -1 : e - a;
  }
  // state index of sequence b (-1: out of range)
  __device__ __forceinline__ int state(int b) const {
    if (!slot) return b;
    const int s = slot[b];
    return (s < 0 || s >= n_slots) ? -1 : s;
  }
  // row (in units of dv floats) of node 0 of unit (b, h) in U
  __device__ __forceinline__ size_t urow0(int b, int h, int Hv, int N) const {
    return cu ? (size_t)h * T + cu[b] : ((size_t)b * Hv + h) * N;
  }
#endif
};

struct VerifyArgs {
  const void *q, *k, *v;
  const float *log_alpha, *beta;
  const int32_t* parent;
  const float* S0;
  void* o;
  float* U;
  gdn_tree_dims d;
  int32_t* dev_status;
  SeqLayout lay = {};
  // the 256-node kernel and the chunk pass run the units whose tree is one chain in
  // the chunkwise form (bf16, dk = dv = 128)
  bool chains = false;
};

struct CommitArgs {
  const int32_t *path, *path_len, *parent;
  const float* U;
  const void* k;
  const float *log_alpha, *S0;
  float* S1;
  gdn_tree_dims d;
  int32_t Lmax;
  int32_t* dev_status;
  SeqLayout lay = {};
};

// delayed commitment of the previous tree's accepted path fused with the
// verification of the next tree (the next tree is verified from S1)
struct CommitVerifyArgs {
  const int32_t *prev_path, *prev_path_len, *prev_parent;
  const float* prev_U;
  const void* prev_k;
  const float* prev_log_alpha;
  int32_t prev_N, Lmax;
  const float* S_prev;
  float* S1;
  int32_t* commit_status;
  VerifyArgs verify;  // verify.S0 is ignored (the state is S1)
  SeqLayout prev_lay = {};  // the previous tree's rows (state slots: verify.lay's)
};

// Bound of the on-device waits, and test-only controls that make one run out.
// Normal calls use the defaults (2 s, nothing withheld); a test sets them
// through the environment (read at every launch by wait_hooks()):
//   GDN_TREE_TEST_WAIT_LIMIT_NS=<ns>       the bound of every wait
//   GDN_TREE_TEST_WITHHOLD_NODE=<unit>:<node>  the tensor-core, 256-node and
//       tensor-core chunk-pass verifications of unit (b * Hv + h) never arrive on
//       that node's solve barrier, so the waits of its descendants (in its chunk,
//       for the chunk pass) run out (thread arrivals only: no copy or MMA is left
//       in flight); in the attention on the tensor cores, warp <node> of the units
//       (b * Hkv + key head; 0 for b in the shared prefix's) never says that Q and the
//       tree are in place; in the prefill in chunks, warp <node> of the chains of
//       (b * Hv + h) that its part of the first state is
//   GDN_TREE_TEST_WITHHOLD_COPY=<b>        the tensor-core commit of sequence b
//       expects its state copy but never issues it, so the wait for it runs out; the
//       prefill's first kernel does so with the keys and queries of b's chunks
struct WaitHooks {
  uint64_t limit_ns = 2000000000ull;
  int withhold_unit = -1, withhold_node = -1;
  int withhold_copy_seq = -1;
};
WaitHooks wait_hooks();

// picks the kernel for the shape and dtype
cudaError_t launch_verify(const VerifyArgs& a, cudaStream_t stream);

size_t verify_generic_smem_bytes(int N, int dk, int dv);
cudaError_t launch_verify_generic(const VerifyArgs& a, cudaStream_t stream);

// trees longer than kMaxNHost: the two-level chunk pass
size_t verify_long_smem_bytes(int N, int dk, int dv);
cudaError_t launch_verify_long(const VerifyArgs& a, cudaStream_t stream);

// the chunkwise path for units whose tree is one chain fits beside the tree kernels
bool verify_chain_path_fits(const gdn_tree_dims& d);

// bf16 trees of up to kMaxNLongHost nodes with dk = dv = 128: the chunk pass with
// R and the output seeds on the tensor cores
bool verify_long_tc_supported(const gdn_tree_dims& d);
cudaError_t launch_verify_long_tc(const VerifyArgs& a, cudaStream_t stream);

// bf16 trees of up to 256 nodes with dk = dv = 128 (R and the seeds on the tensor
// cores, the solve on CUDA cores, on chip)
bool verify_mid_supported(const gdn_tree_dims& d);
cudaError_t launch_verify_mid(const VerifyArgs& a, cudaStream_t stream);

// 128-byte-swizzled TMA maps of fp32 states [n_states, 128, 128] as four boxes of
// 32 columns x 128 rows each (false when the driver's encoder is unavailable)
bool encode_state_map(CUtensorMap* map, const float* base, long long n_states);

// 128-byte-swizzled TMA map of bf16 rows [rows, heads, width] (width a multiple of 64):
// boxes of 64 columns x one head x box_rows rows
bool encode_head_rows_map(CUtensorMap* map, const void* base, long long rows, int heads, int width,
                          int box_rows);
// the same with boxes of box_heads heads of each of box_rows rows, in that order
bool encode_q_map(CUtensorMap* map, const void* base, long long rows, int heads, int width,
                  int box_heads, int box_rows);

bool verify_tc_supported(const gdn_tree_dims& d);
cudaError_t launch_verify_tc(const VerifyArgs& a, cudaStream_t stream);

// the commit: on the tensor cores (bf16 k, dk = dv = 128) unless the CUDA-core
// kernels are forced, else one warp per 32-row block on CUDA cores
cudaError_t launch_commit(const CommitArgs& a, cudaStream_t stream);
cudaError_t launch_commit_warp(const CommitArgs& a, cudaStream_t stream);
bool commit_tc_supported(const gdn_tree_dims& d, int32_t Lmax);
cudaError_t launch_commit_tc(const CommitArgs& a, cudaStream_t stream);

// streaming multiprocessors of the current device (cached per device; 0: no device)
int sm_count();

// top-w best-first draft-tree construction
size_t tree_topw_smem_bytes(int N, int c);
cudaError_t launch_tree_topw(const float* cand_logp, int B, int N, int c, int w, int max_depth,
                             int32_t* parent, int32_t* cand_index, float* score, int32_t* n_built,
                             cudaStream_t stream);

// single-branch recurrent verification (the measurement baseline)
cudaError_t launch_verify_recurrent(const VerifyArgs& a, cudaStream_t stream);

// the gated delta rule over whole sequences (lay.cu set) or one token of each (lay.cu
// null): rows q .. o as in the packed layout, states pool_in -> pool_out
struct RuleArgs {
  const void *q, *k, *v;
  const float *log_alpha, *beta;
  const float* pool_in;
  float* pool_out;
  void* o;
  gdn_tree_dims d;
  int32_t* dev_status;
  SeqLayout lay = {};
};
size_t prefill_workspace_bytes(const gdn_tree_dims& d, int32_t T);
cudaError_t launch_prefill(const RuleArgs& a, void* workspace, cudaStream_t stream);
// the chunked form on the tensor cores (bf16, dk = dv = 128)
bool prefill_tc_supported(const gdn_tree_dims& d);
size_t prefill_tc_workspace_bytes(const gdn_tree_dims& d, int32_t T);
cudaError_t launch_prefill_tc(const RuleArgs& a, void* workspace, cudaStream_t stream);
cudaError_t launch_decode_step(const RuleArgs& a, cudaStream_t stream);

// attention over a paged cache with a shared prefix
struct AttendArgs {
  const void *q, *k, *v;
  const int32_t *parent, *cu;
  const void *k_cache, *v_cache;
  const int32_t *page_table, *context_len, *prefix_pages;
  float scale;
  void* o;
  float* lse;
  gdn_tree_attend_dims d;
  int32_t* dev_status;
  void* workspace;
};
size_t attend_workspace_bytes(const gdn_tree_attend_dims& d);
cudaError_t launch_attend(const AttendArgs& a, cudaStream_t stream);
// sequences of at most kAttendFewRows query rows a key head (others are left alone); parts
// of the rows' keys that other units took ([parts][T * Hq][D], [parts][T * Hq]) are added
constexpr int kAttendFewRows = 16;
constexpr int kAttendMaxParts = 64;  // of the shared prefix
int attend_few_cluster(const gdn_tree_attend_dims& d, int prefix_len, float* us);
cudaError_t launch_attend_few(const AttendArgs& a, int prefix_len, const float* part_o,
                              const float* part_lse, int parts, cudaStream_t stream);
cudaError_t launch_attend_f32(const AttendArgs& a, cudaStream_t stream);

// rows of accepted paths (or all rows) into the pages of a cache
struct AppendArgs {
  const void *k, *v;
  const int32_t *path, *path_len;
  int32_t Lmax;
  const int32_t* cu;
  void *k_cache, *v_cache;
  const int32_t *page_table, *context_len;
  int32_t* new_len;
  gdn_tree_attend_dims d;
  int32_t* dev_status;
};
cudaError_t launch_cache_append(const AppendArgs& a, cudaStream_t stream);

bool commit_verify_tc_supported(const gdn_tree_dims& d, int prev_N, int Lmax);
cudaError_t launch_commit_verify_tc(const CommitVerifyArgs& a, cudaStream_t stream);
cudaError_t launch_commit_verify(const CommitVerifyArgs& a, cudaStream_t stream);

}  // namespace gdn
