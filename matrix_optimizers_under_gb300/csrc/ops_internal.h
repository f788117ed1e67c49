// Launch descriptors and host helpers of the operators next to the owner step:
// gradient norm and clipping, id sort, embedding lookup and gradient, products
// grouped by expert, log-probabilities of tokens, norms around a block, AdamW over
// many tensors.
#pragma once

#include <algorithm>
#include <cstddef>
#include <cstdint>

#include <cuda_runtime.h>

#include "mfsdp.h"

namespace mfsdp {
namespace ops {

// ------------------------------------------------------------- host helpers
inline bool aligned(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

inline bool ranges_overlap(const void* p, size_t pb, const void* q, size_t qb) {
  if (pb == 0 || qb == 0) return false;
  const uintptr_t a = reinterpret_cast<uintptr_t>(p), b = reinterpret_cast<uintptr_t>(q);
  return a < b + qb && b < a + pb;
}

inline bool known_dtype(int32_t dt) { return dt == MFSDP_DTYPE_F32 || dt == MFSDP_DTYPE_BF16; }
inline size_t dtype_size(int32_t dt) { return dt == MFSDP_DTYPE_BF16 ? 2 : 4; }
inline size_t round_up(size_t x, size_t a) { return (x + a - 1) / a * a; }
inline int cuda_status(cudaError_t e) { return e == cudaSuccess ? MFSDP_OK : MFSDP_ERR_CUDA; }

// Launch that may overlap the kernel before it in the stream from where that
// one allows it (ptx::launch_dependents), or in plain order.  The kernel calls
// ptx::wait_dependencies() before it reads that one's results.
template <typename... P, typename... A>
cudaError_t launch_overlapped(void (*kernel)(P...), dim3 grid, dim3 block, size_t smem, cudaStream_t s, bool overlap,
                              A&&... args) {
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cfg.attrs = &attr;
  cfg.numAttrs = overlap ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<A&&>(args)...);
}

constexpr int kMaxDevices = 64;

// SM count of the current device, looked up once per device (0: no device).
int sm_count();

// SMs of a GB300.  Sizes that a workspace's length follows from use it, since that length is asked
// for where there may be no device; on another count the results stay right and the CTAs
// meant to run at once may not.
constexpr int kSms = 152;

// ------------------------------------------------- gradient norm and clipping
// One tensor of a gradient set and the chunks it is cut into.
struct ClipTensor {
  const void* src;
  void* dst;
  int64_t numel;
  int32_t chunk0;        // its first chunk of the launch
  int16_t src_bf16, dst_bf16;
};
constexpr int kClipChunkBytes = 32768;  // source bytes of one chunk
constexpr int kClipTable = 512;         // tensors per launch
constexpr int kClipShort = 16;          // tensors of a short table (a launch copies its table)
struct ClipHead {
  int32_t n;
  int32_t chunks;        // chunks of this launch
  int32_t first_partial; // this launch's first slot in `partials`
  int32_t n_partials;    // slots of the whole set
  double* partials;      // one sum of squares per CTA of the norm launches
  float* out;            // {norm, coefficient}
  double max_norm, eps;
};
template <int kN>
struct ClipBatch : ClipHead {
  ClipTensor t[kN];
};
static_assert(sizeof(ClipBatch<kClipTable>) < 32000, "kernel parameter limit");
cudaError_t launch_clip_norm(const ClipBatch<kClipTable>& b, int blocks, cudaStream_t s);
cudaError_t launch_clip_finish(const ClipHead& b, cudaStream_t s);
cudaError_t launch_clip_scale(const ClipBatch<kClipTable>& b, int blocks, bool overlap, cudaStream_t s);

// ------------------------------------------------------------------- id sort
struct SortArgs {
  const void* ids;
  int32_t ids64;
  int64_t n;
  int64_t n_keys;        // valid ids are 0 .. n_keys-1; any other sorts as n_keys
  int32_t* keys_out;     // sorted keys [n]
  int32_t* order_out;    // the position each came from [n]
  void* scratch;         // sort_scratch_bytes(n, n_keys)
  int32_t* zero;         // a word the sort sets to 0 (may be null)
};
size_t sort_scratch_bytes(int64_t n, int64_t n_keys);
constexpr int kSortSms = 8;            // SMs that a sort of few ids takes
cudaError_t launch_sort(const SortArgs& a, cudaStream_t s);
cudaError_t launch_key_starts(const int32_t* keys, int64_t n, int64_t n_keys, int32_t* starts, cudaStream_t s);

// ----------------------------------------------------------------- embedding
struct LookupArgs {
  const void* w;
  const void* ids;
  void* out;
  int64_t vocab, dim, w_ld, n, out_ld;
  int32_t w_bf16, out_bf16, ids64;
  float scale;
};
cudaError_t launch_lookup(const LookupArgs& a, cudaStream_t s);

struct EmbedGradArgs {
  const void* dout;
  void* grad;
  const void* ids;
  const int32_t* keys;   // sorted
  const int32_t* order;
  float* partials;       // embed_grad_partial_bytes(n, vocab, dim)
  int32_t* header;       // the status word, zeroed before
  int64_t n, vocab, dim, dout_ld, grad_ld;
  int32_t dout_bf16, grad_bf16, accumulate, ids64;
  float scale;
};
size_t embed_grad_partial_bytes(int64_t n, int64_t vocab, int64_t dim);
// Whether the gradient takes the ids sorted (few it takes as they are).
bool embed_grad_sorts(const EmbedGradArgs& a);
cudaError_t launch_embed_grad(const EmbedGradArgs& a, cudaStream_t s);

// --------------------------------------------- products grouped by expert
enum ExpertMode : int32_t {
  kExpertForward = 0,     // Y = X W^T
  kExpertInputGrad = 1,   // dX = dY W
  kExpertWeightGrad = 2,  // dW = dY^T X
};
struct ExpertArgs {
  int32_t mode;
  int32_t n_experts;
  int64_t n_rows, rows, cols;
  const void* a;          // forward: X; input gradient: dY; weight gradient: dY
  const void* b;          // forward, input gradient: W; weight gradient: X
  void* out;
  const int32_t* starts;
  int64_t a_ld, b_ld;     // leading dimensions (b_ld: of W, its columns)
  int64_t b_stride;       // forward, input gradient: elements between experts' matrices
  int64_t out_ld, out_stride;
  int32_t out_bf16, accumulate;
  int32_t out_vec;        // the output's rows start on 16-byte boundaries
  int32_t* status;        // first wait that gave up (0: none)
  uint8_t* packs;         // workspace for operands whose rows are not 16-byte aligned
  uint64_t wait_limit_ns;
  int32_t prepared;       // kernels of this call that prepare operands run right before
  int32_t only_ends;      // and what they prepare is the groups' padded ends
  int32_t chunk;          // weight gradient: tokens of a chunk of a split contraction (0: whole groups)
  int32_t slots;          // and chunks that there can be in all
};
// Bytes of a copy of n rows of `width` bf16 elements, each padded to 16 bytes.
inline size_t packed_bytes(int64_t n, int64_t width) {
  return round_up((size_t)n * (size_t)((width + 7) / 8 * 8) * 2, 256);
}
// Workspace of a weight gradient whose contraction is split (0: it is not).
size_t expert_split_bytes(int64_t n_experts, int64_t n_rows, int64_t rows, int64_t cols);
cudaError_t launch_expert(const ExpertArgs& a, cudaStream_t s);

// ------------------------------------------------- AdamW over many tensors
struct AdamwTensor {
  void* p;
  const void* g;
  void* m;
  void* v;
  float* m_scale;
  float* v_scale;
  void* copy;
  int64_t numel;
  int32_t chunk0;        // its first chunk of the launch
  float decay;           // 1 - lr wd
  float step_size;       // lr / (1 - beta1^step)
  int32_t form;          // 1: p bf16, 2: g bf16, 4: state in 8 bits, 8: all on 4 elements' boundaries
};
constexpr int kAdamwChunk = 2048;      // elements of a chunk
constexpr int kAdamwTable = 384;       // tensors per launch
constexpr int kAdamwShort = 16;        // tensors of a short table
struct AdamwHead {
  int32_t n;
  int32_t chunks;
  float beta1, omb1, beta2, omb2, inv_sqrt_bc2, eps;
  const float* norm;     // {norm, clipping coefficient}, or null
};
template <int kN>
struct AdamwBatch : AdamwHead {
  AdamwTensor t[kN];
};
static_assert(sizeof(AdamwBatch<kAdamwTable>) < 32000, "kernel parameter limit");
cudaError_t launch_adamw_set(const AdamwBatch<kAdamwTable>& b, int sms, cudaStream_t s);

// --------------------------------------- log-probabilities of given tokens
struct LogprobArgs {
  const void* x;
  const void* targets;   // may be null, like each output
  float* logprob;
  float* lse;
  float* entropy;
  int32_t* top_ids;
  float* top_logprob;
  int64_t n, vocab, x_ld;
  int32_t x_bf16, ids64, top_k;
  float scale;
  float k2;              // the scale in powers of two: scale * log2(e)
};
cudaError_t launch_logprob(const LogprobArgs& a, int sms, cudaStream_t s);

struct LogprobGradArgs {
  const void* x;
  const void* targets;
  const float* lse;
  const float* entropy;
  const float* dlogprob;
  const float* dentropy;
  void* dx;
  int64_t n, vocab, x_ld, dx_ld;
  int32_t x_bf16, ids64;
  float scale;
};
cudaError_t launch_logprob_grad(const LogprobGradArgs& a, int sms, cudaStream_t s);

// ------------------------------------------------- the norms around a block
// Bytes from a row to the one after it, and to the next that the same threads take (set by the launch).
struct RowStep {
  int64_t row, next;
};
struct NormArgs {
  const void* residual;
  const void* branch;    // null: no block before
  const void* w_post;    // vectors: null is ones (weights, gate) or zeros (biases)
  const void* b_post;
  const void* gate;
  const void* w_pre;
  const void* b_pre;
  void* out;
  void* normed;
  float4* stats;
  int64_t n;
  RowStep residual_step, branch_step, out_step, normed_step;
  int64_t gate_rows;
  int32_t dim, post, pre;
  int32_t r_bf16, b_bf16, w_bf16;
  int32_t vec;           // every row and vector consists of 16-byte vectors
  float eps, inv_dim, residual_scale, branch_scale;
};
cudaError_t launch_norm(NormArgs a, cudaStream_t s);

struct NormGradArgs {
  NormArgs f;            // the forward call's, without its outputs
  const float4* stats;
  const void* d_out;
  const void* d_normed;
  void* d_residual;
  void* d_branch;
  RowStep d_out_step, d_normed_step, d_residual_step, d_branch_step;
  float* d_w_post;       // any may be null
  float* d_b_post;
  float* d_gate;
  float* d_w_pre;
  float* d_b_pre;
  int32_t accumulate;
  int32_t* status;       // workspace: first wait that gave up (0: none)
  float* parts;          // kNormParts x dim sums of each CTA
  float* gate_parts;     // after them, set by the launch: two rows of a gate of each run of rows, where a run's end cuts a group
};
constexpr int kNormParts = 5;
size_t norm_grad_part_bytes(int64_t dim, int64_t n);
cudaError_t launch_norm_grad(NormGradArgs g, cudaStream_t s);

}  // namespace ops
}  // namespace mfsdp
