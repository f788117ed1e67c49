// Host side of the tokens' log-probabilities, the norms around a block and AdamW over many
// tensors: argument checks, the workspace layout and launches.
#include <cmath>
#include <vector>

#include "mfsdp.h"
#include "ops_host.h"
#include "ops_internal.h"

namespace mfsdp {
namespace ops {
namespace {

// What takes x to powers of two of exp(scale * x): from the scale as fp32 has it.
float log2_scale(double scale) { return (float)((double)(float)scale * 1.4426950408889634); }

// ------------------------------------------------- AdamW over many tensors
int64_t adamw_chunks(int64_t numel) { return (numel + kAdamwChunk - 1) / kAdamwChunk; }
int64_t adamw_scales(int64_t numel) { return (numel + MFSDP_STATE_BLOCK - 1) / MFSDP_STATE_BLOCK; }

int check_adamw(const mfsdp_adamw_tensor* t, int32_t n, double lr, double bc1) {
  for (int i = 0; i < n; ++i) {
    if (!known_dtype(t[i].p_dtype) || !known_dtype(t[i].g_dtype)) return MFSDP_ERR_UNSUPPORTED_DTYPE;
    if (t[i].state != MFSDP_STATE_F32 && t[i].state != MFSDP_STATE_E4M3) return MFSDP_ERR_INVALID_ARG;
    const double rate = lr * t[i].lr_scale;
    if (t[i].numel < 0 || !scale_ok(t[i].lr_scale) || !scale_ok(t[i].wd) || !scale_ok(rate / bc1) ||
        !scale_ok(1.0 - rate * t[i].wd))
      return MFSDP_ERR_INVALID_ARG;
    if (t[i].numel > (int64_t)1 << 40) return MFSDP_ERR_UNSUPPORTED_SHAPE;
    if (t[i].numel == 0) continue;
    const bool eight = t[i].state == MFSDP_STATE_E4M3;
    if (!t[i].p || !t[i].g || !t[i].m || !t[i].v || (eight && (!t[i].m_scale || !t[i].v_scale)))
      return MFSDP_ERR_INVALID_ARG;
    if (!aligned(t[i].p, dtype_size(t[i].p_dtype)) || !aligned(t[i].g, dtype_size(t[i].g_dtype)) ||
        !aligned(t[i].m, eight ? 1 : 4) || !aligned(t[i].v, eight ? 1 : 4) || !aligned(t[i].copy, 2) ||
        (eight && (!aligned(t[i].m_scale, 4) || !aligned(t[i].v_scale, 4))))
      return MFSDP_ERR_MISALIGNED;
  }
  return MFSDP_OK;
}

struct Range {
  uintptr_t lo, hi;
};
bool by_lo(const Range& a, const Range& b) { return a.lo < b.lo; }

// What the step writes is apart from each other and from what it only reads.  A
// set's tensors mostly lie in order in one buffer a role, so each role is sorted
// by itself, most often at no cost, and the roles are merged.
int check_adamw_overlap(const mfsdp_adamw_tensor* t, int32_t n, const float* norm) try {
  constexpr int kWritten = 6;
  std::vector<Range> written, role, read;
  written.reserve((size_t)n * kWritten);
  const auto push = [](std::vector<Range>& to, const void* p, size_t bytes) {
    const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
    if (p && bytes) to.push_back({lo, lo + bytes});
  };
  const auto sort = [](std::vector<Range>& r) {
    if (!std::is_sorted(r.begin(), r.end(), by_lo)) std::sort(r.begin(), r.end(), by_lo);
  };
  for (int k = 0; k < kWritten; ++k) {
    role.clear();
    for (int i = 0; i < n; ++i) {
      const size_t numel = (size_t)t[i].numel, scales = (size_t)adamw_scales(t[i].numel) * 4;
      const bool eight = t[i].state == MFSDP_STATE_E4M3;
      if (k == 0) push(role, t[i].p, numel * dtype_size(t[i].p_dtype));
      if (k == 1) push(role, t[i].m, numel * (eight ? 1 : 4));
      if (k == 2) push(role, t[i].v, numel * (eight ? 1 : 4));
      if (k == 3) push(role, t[i].copy, numel * 2);
      if (k == 4 && eight) push(role, t[i].m_scale, scales);
      if (k == 5 && eight) push(role, t[i].v_scale, scales);
    }
    sort(role);
    const size_t before = written.size();
    written.insert(written.end(), role.begin(), role.end());
    std::inplace_merge(written.begin(), written.begin() + before, written.end(), by_lo);
  }
  for (size_t i = 1; i < written.size(); ++i)
    if (written[i - 1].hi > written[i].lo) return MFSDP_ERR_OVERLAP;
  for (int i = 0; i < n; ++i) push(read, t[i].g, (size_t)t[i].numel * dtype_size(t[i].g_dtype));
  push(read, norm, norm ? 8 : 0);
  sort(read);
  // The written ranges are apart, so their ends ascend too: the first that ends past a read
  // range's start is the only one that may begin before its end without others doing so.
  size_t j = 0;
  for (const Range& r : read) {
    while (j < written.size() && written[j].hi <= r.lo) ++j;
    if (j < written.size() && written[j].lo < r.hi) return MFSDP_ERR_OVERLAP;
  }
  return MFSDP_OK;
} catch (...) {                                           // no host memory for the tables: nothing leaves a C entry
  return MFSDP_ERR_CUDA;
}

bool on_four(const mfsdp_adamw_tensor& t) {
  const size_t state = t.state == MFSDP_STATE_E4M3 ? 4 : 16;
  return aligned(t.p, 4 * dtype_size(t.p_dtype)) && aligned(t.g, 4 * dtype_size(t.g_dtype)) && aligned(t.m, state) &&
         aligned(t.v, state) && aligned(t.copy, 8);
}

// --------------------------------------- log-probabilities of given tokens
// What both calls check of the logits and targets.
int check_logits(const void* x, int32_t dtype, int64_t n, int64_t vocab, int64_t ld, const void* targets,
                 int32_t id_type, double scale) {
  if (!known_dtype(dtype) || !known_id_type(id_type)) return MFSDP_ERR_UNSUPPORTED_DTYPE;
  if (n < 0 || vocab < 1) return MFSDP_ERR_INVALID_ARG;
  if (!(scale >= 0x1p-20 && scale <= 0x1p20)) return MFSDP_ERR_INVALID_ARG;   // 2^100 of it is in fp32, and far from 0
  if (n > INT32_MAX || vocab >= INT32_MAX || !rows_fit(n, ld, vocab)) return MFSDP_ERR_UNSUPPORTED_SHAPE;
  if (n == 0) return MFSDP_OK;
  if (!x) return MFSDP_ERR_INVALID_ARG;
  if (!aligned(x, dtype_size(dtype)) || !aligned(targets, id_size(id_type))) return MFSDP_ERR_MISALIGNED;
  return MFSDP_OK;
}

// ------------------------------------------------- the norms around a block
bool known_norm(int32_t k) { return k == MFSDP_NORM_NONE || k == MFSDP_NORM_RMS || k == MFSDP_NORM_LAYER; }

int check_norm_spec(const mfsdp_block_norm_spec* s, int64_t n) {
  if (!s || n < 0) return MFSDP_ERR_INVALID_ARG;
  if (!known_dtype(s->residual_dtype) || !known_dtype(s->branch_dtype) || !known_dtype(s->weight_dtype))
    return MFSDP_ERR_UNSUPPORTED_DTYPE;
  if (s->dim < 1 || !known_norm(s->post_norm) || !known_norm(s->pre_norm) || !(s->eps >= 0.0) || !scale_ok(s->eps) ||
      !scale_ok(s->residual_scale) || !scale_ok(s->branch_scale) || (s->gate && s->gate_rows < 1))
    return MFSDP_ERR_INVALID_ARG;
  // (the kernels count rows in int32, some turns past the last one)
  if (s->dim > MFSDP_MAX_NORM_DIM || n > (int64_t)1 << 30) return MFSDP_ERR_UNSUPPORTED_SHAPE;
  const size_t w = dtype_size(s->weight_dtype);
  if (!aligned(s->post_weight, w) || !aligned(s->post_bias, w) || !aligned(s->gate, w) || !aligned(s->pre_weight, w) ||
      !aligned(s->pre_bias, w))
    return MFSDP_ERR_MISALIGNED;
  return MFSDP_OK;
}

// A tensor of rows of a call.
struct Rows {
  const void* p;
  int64_t ld;
  int32_t dtype;
};

// Rows whose leading dimensions and alignment fit (absent ones do).
int check_rows(const Rows* r, int count, int64_t n, int64_t dim) {
  for (int i = 0; i < count; ++i)
    if (r[i].p && !rows_fit(n, r[i].ld, dim)) return MFSDP_ERR_UNSUPPORTED_SHAPE;
  for (int i = 0; i < count; ++i)
    if (!aligned(r[i].p, dtype_size(r[i].dtype))) return MFSDP_ERR_MISALIGNED;
  return MFSDP_OK;
}

Buf rows_buf(const Rows& r, int64_t n, int64_t dim) {
  return {r.p, r.p ? extent(n, r.ld, dim, dtype_size(r.dtype)) : 0};
}
int64_t step_of(const Rows& r) { return r.p ? r.ld * (int64_t)dtype_size(r.dtype) : 0; }
bool same_rows(const Rows& a, const Rows& b) { return a.p == b.p && a.ld == b.ld && a.dtype == b.dtype; }

int64_t gate_count(const mfsdp_block_norm_spec* s, int64_t n) {
  const int64_t rows = std::min(s->gate_rows, std::max<int64_t>(n, 1));
  return s->gate ? (n + rows - 1) / rows : 0;
}

// The vectors as buffers that are only read.
void vector_bufs(const mfsdp_block_norm_spec* s, int64_t n, Buf (&b)[5]) {
  const size_t one = (size_t)s->dim * dtype_size(s->weight_dtype);
  b[0] = {s->post_weight, s->post_weight ? one : 0};
  b[1] = {s->post_bias, s->post_bias ? one : 0};
  b[2] = {s->gate, one * (size_t)gate_count(s, n)};
  b[3] = {s->pre_weight, s->pre_weight ? one : 0};
  b[4] = {s->pre_bias, s->pre_bias ? one : 0};
}

void fill_norm(NormArgs& a, const mfsdp_block_norm_spec* s, int64_t n, const Rows& residual, const Rows& branch) {
  a.residual = residual.p;
  a.residual_step.row = step_of(residual);
  a.branch = branch.p;
  a.branch_step.row = step_of(branch);
  a.post = branch.p ? s->post_norm : MFSDP_NORM_NONE;
  a.pre = s->pre_norm;
  const bool post = a.post != MFSDP_NORM_NONE, pre = a.pre != MFSDP_NORM_NONE;
  a.w_post = post ? s->post_weight : nullptr;
  a.b_post = post ? s->post_bias : nullptr;
  a.gate = branch.p ? s->gate : nullptr;
  a.gate_rows = a.gate ? std::min(s->gate_rows, std::max<int64_t>(n, 1)) : std::max<int64_t>(n, 1);
  a.w_pre = pre ? s->pre_weight : nullptr;
  a.b_pre = pre ? s->pre_bias : nullptr;
  a.n = n;
  a.dim = (int32_t)s->dim;
  a.r_bf16 = s->residual_dtype == MFSDP_DTYPE_BF16;
  a.b_bf16 = s->branch_dtype == MFSDP_DTYPE_BF16;
  a.w_bf16 = s->weight_dtype == MFSDP_DTYPE_BF16;
  a.eps = (float)s->eps;
  a.inv_dim = (float)(1.0 / (double)s->dim);
  a.residual_scale = (float)s->residual_scale;
  a.branch_scale = (float)s->branch_scale;
}

// Whether rows and vectors all consist of 16-byte vectors.
bool norm_vectors(const mfsdp_block_norm_spec* s, const Rows* r, int count, int64_t n) {
  bool ok = s->dim % 8 == 0 && aligned(s->post_weight, 16) && aligned(s->post_bias, 16) && aligned(s->gate, 16) &&
            aligned(s->pre_weight, 16) && aligned(s->pre_bias, 16);
  for (int i = 0; i < count; ++i)
    ok = ok && (!r[i].p || (aligned(r[i].p, 16) && (n <= 1 || r[i].ld * (int64_t)dtype_size(r[i].dtype) % 16 == 0)));
  return ok;
}

}  // namespace
}  // namespace ops
}  // namespace mfsdp

using namespace mfsdp;
using namespace mfsdp::ops;

extern "C" int mfsdp_adamw_set_step(const mfsdp_adamw_tensor* tensors, int32_t n, double lr, double beta1, double beta2,
                                    double eps, int64_t step, const float* norm, void* stream) {
  if (n < 0 || (n > 0 && !tensors) || step < 1) return MFSDP_ERR_INVALID_ARG;
  if (!(beta1 >= 0.0 && beta1 < 1.0) || !(beta2 >= 0.0 && beta2 < 1.0) || !scale_ok(lr) ||
      !(eps == 0.0 || (eps >= 0x1p-126 && eps <= 0x1p120)))            // its reciprocal is a normal number
    return MFSDP_ERR_INVALID_ARG;
  const double bc1 = 1.0 - std::pow(beta1, (double)step), bc2 = 1.0 - std::pow(beta2, (double)step);
  int st = check_adamw(tensors, n, lr, bc1);
  if (st != MFSDP_OK) return st;
  if (!aligned(norm, 4)) return MFSDP_ERR_MISALIGNED;
  int64_t total = 0;
  for (int i = 0; i < n; ++i) total += adamw_chunks(tensors[i].numel);
  if (total == 0) return MFSDP_OK;
  if (total > (int64_t)1 << 30) return MFSDP_ERR_UNSUPPORTED_SHAPE;
  st = check_adamw_overlap(tensors, n, norm);
  if (st != MFSDP_OK) return st;
  const int sms = sm_count();
  if (sms <= 0) return MFSDP_ERR_CUDA;
  const OpRange range("mfsdp adamw set");
  AdamwBatch<kAdamwTable> b;
  b.beta1 = (float)beta1;
  b.omb1 = (float)(1.0 - beta1);
  b.beta2 = (float)beta2;
  b.omb2 = (float)(1.0 - beta2);
  b.inv_sqrt_bc2 = (float)(1.0 / std::sqrt(bc2));
  b.eps = (float)eps;
  b.norm = norm;
  for (int i = 0; i < n;) {
    b.n = b.chunks = 0;
    for (; i < n && b.n < kAdamwTable; ++i) {
      const mfsdp_adamw_tensor& t = tensors[i];
      if (t.numel == 0) continue;
      AdamwTensor& a = b.t[b.n++];
      const double rate = lr * t.lr_scale;
      a.p = t.p;
      a.g = t.g;
      a.m = t.m;
      a.v = t.v;
      a.m_scale = t.m_scale;
      a.v_scale = t.v_scale;
      a.copy = t.copy;
      a.numel = t.numel;
      a.chunk0 = b.chunks;
      a.decay = (float)(1.0 - rate * t.wd);
      a.step_size = (float)(rate / bc1);
      a.form = (t.p_dtype == MFSDP_DTYPE_BF16 ? 1 : 0) | (t.g_dtype == MFSDP_DTYPE_BF16 ? 2 : 0) |
               (t.state == MFSDP_STATE_E4M3 ? 4 : 0) | (on_four(t) ? 8 : 0);
      b.chunks += (int32_t)adamw_chunks(t.numel);
    }
    if (b.chunks == 0) continue;
    const cudaError_t e = launch_adamw_set(b, sms, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_status(e);
  }
  return MFSDP_OK;
}

extern "C" int mfsdp_token_logprob(const void* logits, int32_t logits_dtype, int64_t n, int64_t vocab, int64_t logits_ld,
                                   const void* targets, int32_t id_type, double scale, float* logprob, float* lse,
                                   float* entropy, int32_t top_k, int32_t* top_ids, float* top_logprob, void* stream) {
  int st = check_logits(logits, logits_dtype, n, vocab, logits_ld, targets, id_type, scale);
  if (st != MFSDP_OK) return st;
  if (top_k < 0 || top_k > MFSDP_MAX_TOP || top_k > vocab) return MFSDP_ERR_INVALID_ARG;
  if (n == 0) return MFSDP_OK;
  if ((logprob && !targets) || (top_k == 0 && (top_ids || top_logprob)) || (top_k > 0 && !top_ids && !top_logprob) ||
      (!logprob && !lse && !entropy && top_k == 0))
    return MFSDP_ERR_INVALID_ARG;
  if (!aligned(logprob, 4) || !aligned(lse, 4) || !aligned(entropy, 4) || !aligned(top_ids, 4) ||
      !aligned(top_logprob, 4))
    return MFSDP_ERR_MISALIGNED;
  const size_t rows = (size_t)n * 4, tops = rows * (size_t)top_k;
  const Buf bufs[7] = {{logprob, logprob ? rows : 0}, {lse, lse ? rows : 0}, {entropy, entropy ? rows : 0},
                       {top_ids, top_ids ? tops : 0}, {top_logprob, top_logprob ? tops : 0},
                       {logits, extent(n, logits_ld, vocab, dtype_size(logits_dtype))},
                       {targets, targets ? (size_t)n * id_size(id_type) : 0}};
  if (any_overlap(bufs, 7, 5)) return MFSDP_ERR_OVERLAP;
  const int sms = sm_count();
  if (sms <= 0) return MFSDP_ERR_CUDA;
  LogprobArgs a{};
  a.x = logits;
  a.targets = targets;
  a.logprob = logprob;
  a.lse = lse;
  a.entropy = entropy;
  a.top_ids = top_ids;
  a.top_logprob = top_logprob;
  a.n = n;
  a.vocab = vocab;
  a.x_ld = logits_ld;
  a.x_bf16 = logits_dtype == MFSDP_DTYPE_BF16;
  a.ids64 = id_type == MFSDP_ID_I64;
  a.top_k = top_k;
  a.scale = (float)scale;
  a.k2 = log2_scale(scale);
  const OpRange range("mfsdp token logprob");
  return cuda_status(launch_logprob(a, sms, static_cast<cudaStream_t>(stream)));
}

extern "C" int mfsdp_token_logprob_grad(const void* logits, int32_t logits_dtype, int64_t n, int64_t vocab,
                                        int64_t logits_ld, const void* targets, int32_t id_type, double scale,
                                        const float* lse, const float* entropy, const float* dlogprob,
                                        const float* dentropy, void* dlogits, int64_t dlogits_ld, void* stream) {
  int st = check_logits(logits, logits_dtype, n, vocab, logits_ld, targets, id_type, scale);
  if (st != MFSDP_OK) return st;
  if (!rows_fit(n, dlogits_ld, vocab)) return MFSDP_ERR_UNSUPPORTED_SHAPE;
  if (n == 0) return MFSDP_OK;
  if (!lse || !dlogits || (!dlogprob && !dentropy) || (dlogprob && !targets) || (dentropy && !entropy))
    return MFSDP_ERR_INVALID_ARG;
  if (!aligned(dlogits, dtype_size(logits_dtype)) || !aligned(lse, 4) || !aligned(entropy, 4) ||
      !aligned(dlogprob, 4) || !aligned(dentropy, 4))
    return MFSDP_ERR_MISALIGNED;
  const bool in_place = dlogits == logits && dlogits_ld == logits_ld;
  const size_t rows = (size_t)n * 4, es = dtype_size(logits_dtype);
  const Buf bufs[7] = {{dlogits, extent(n, dlogits_ld, vocab, es)},
                       {logits, in_place ? 0 : extent(n, logits_ld, vocab, es)},
                       {targets, targets ? (size_t)n * id_size(id_type) : 0}, {lse, rows},
                       {entropy, entropy ? rows : 0}, {dlogprob, dlogprob ? rows : 0}, {dentropy, dentropy ? rows : 0}};
  if (any_overlap(bufs, 7, 1)) return MFSDP_ERR_OVERLAP;
  const int sms = sm_count();
  if (sms <= 0) return MFSDP_ERR_CUDA;
  LogprobGradArgs a{};
  a.x = logits;
  a.targets = targets;
  a.lse = lse;
  a.entropy = entropy;
  a.dlogprob = dlogprob;
  a.dentropy = dentropy;
  a.dx = dlogits;
  a.n = n;
  a.vocab = vocab;
  a.x_ld = logits_ld;
  a.dx_ld = dlogits_ld;
  a.x_bf16 = logits_dtype == MFSDP_DTYPE_BF16;
  a.ids64 = id_type == MFSDP_ID_I64;
  a.scale = (float)scale;
  const OpRange range("mfsdp token logprob gradient");
  return cuda_status(launch_logprob_grad(a, sms, static_cast<cudaStream_t>(stream)));
}

// ------------------------------------------------- the norms around a block
extern "C" int mfsdp_block_norm(const mfsdp_block_norm_spec* spec, int64_t n, const void* residual, int64_t residual_ld,
                                const void* branch, int64_t branch_ld, void* out, int64_t out_ld, void* normed,
                                int64_t normed_ld, float* stats, void* stream) {
  int st = check_norm_spec(spec, n);
  if (st != MFSDP_OK) return st;
  const Rows r[4] = {{out, out_ld, spec->residual_dtype}, {normed, normed_ld, spec->branch_dtype},
                     {residual, residual_ld, spec->residual_dtype}, {branch, branch_ld, spec->branch_dtype}};
  st = check_rows(r, 4, n, spec->dim);
  if (st != MFSDP_OK) return st;
  if (n == 0) return MFSDP_OK;
  if (!residual || (!out && !normed && !stats) || (out && !branch) || (normed && spec->pre_norm == MFSDP_NORM_NONE))
    return MFSDP_ERR_INVALID_ARG;
  if (!aligned(stats, 16)) return MFSDP_ERR_MISALIGNED;
  // in place: out over residual, normed over branch
  Buf bufs[10] = {rows_buf(r[0], n, spec->dim), rows_buf(r[1], n, spec->dim), {stats, stats ? (size_t)n * 16 : 0},
                  rows_buf(r[2], n, spec->dim), rows_buf(r[3], n, spec->dim)};
  Buf vecs[5];
  vector_bufs(spec, n, vecs);
  std::copy(vecs, vecs + 5, bufs + 5);
  if (same_rows(r[0], r[2])) bufs[3].bytes = 0;
  if (same_rows(r[1], r[3])) bufs[4].bytes = 0;
  if (any_overlap(bufs, 10, 3)) return MFSDP_ERR_OVERLAP;
  NormArgs a{};
  fill_norm(a, spec, n, r[2], r[3]);
  a.out = out;
  a.out_step.row = step_of(r[0]);
  a.normed = normed;
  a.normed_step.row = step_of(r[1]);
  a.stats = reinterpret_cast<float4*>(stats);
  a.vec = norm_vectors(spec, r, 4, n);
  const OpRange range("mfsdp block norm");
  return cuda_status(launch_norm(a, static_cast<cudaStream_t>(stream)));
}

extern "C" size_t mfsdp_block_norm_grad_workspace_bytes(const mfsdp_block_norm_spec* spec, int64_t n) {
  return check_norm_spec(spec, n) == MFSDP_OK ? 256 + round_up(norm_grad_part_bytes(spec->dim, n), 256) : 0;
}

extern "C" int mfsdp_block_norm_grad(const mfsdp_block_norm_spec* spec, int64_t n, const void* residual,
                                     int64_t residual_ld, const void* branch, int64_t branch_ld, const float* stats,
                                     const void* d_out, int64_t d_out_ld, const void* d_normed, int64_t d_normed_ld,
                                     void* d_residual, int64_t d_residual_ld, void* d_branch, int64_t d_branch_ld,
                                     const mfsdp_block_norm_grads* grads, void* workspace, size_t workspace_bytes,
                                     void* stream) {
  int st = check_norm_spec(spec, n);
  if (st != MFSDP_OK) return st;
  const mfsdp_block_norm_grads none = {};
  const mfsdp_block_norm_grads& gv = grads ? *grads : none;
  if (gv.accumulate != 0 && gv.accumulate != 1) return MFSDP_ERR_INVALID_ARG;
  const Rows r[6] = {{d_residual, d_residual_ld, spec->residual_dtype}, {d_branch, d_branch_ld, spec->branch_dtype},
                     {d_out, d_out_ld, spec->residual_dtype}, {d_normed, d_normed_ld, spec->branch_dtype},
                     {residual, residual_ld, spec->residual_dtype}, {branch, branch_ld, spec->branch_dtype}};
  st = check_rows(r, 6, n, spec->dim);
  if (st != MFSDP_OK) return st;
  float* const d[5] = {gv.d_post_weight, gv.d_post_bias, gv.d_gate, gv.d_pre_weight, gv.d_pre_bias};
  const bool gate_sums = d[2] && n > 0;                       // without rows a gate has none either
  const bool sums = d[0] || d[1] || gate_sums || d[3] || d[4];
  if (n > 0 && (!residual || !stats || (!d_out && !d_normed) || (!d_residual && !d_branch && !sums)))
    return MFSDP_ERR_INVALID_ARG;
  // a gradient is of what the forward call had
  if ((n > 0 && !branch && (d_branch || d[0] || d[1] || d[2])) || (d[2] && !spec->gate) ||
      (spec->post_norm == MFSDP_NORM_NONE && (d[0] || d[1])) ||
      (spec->pre_norm == MFSDP_NORM_NONE && (d_normed || d[3] || d[4])) || ((d[3] || d[4]) && n > 0 && !d_normed))
    return MFSDP_ERR_INVALID_ARG;
  if (n == 0 && (!sums || gv.accumulate)) return MFSDP_OK;
  for (float* p : d)
    if (!aligned(p, 16)) return MFSDP_ERR_MISALIGNED;
  if (!aligned(stats, 16)) return MFSDP_ERR_MISALIGNED;
  const size_t need = mfsdp_block_norm_grad_workspace_bytes(spec, n);
  st = check_workspace(workspace, workspace_bytes, need);
  if (st != MFSDP_OK) return st;
  const size_t one = (size_t)spec->dim * 4;
  Buf bufs[18] = {rows_buf(r[0], n, spec->dim), rows_buf(r[1], n, spec->dim), {d[0], d[0] ? one : 0},
                  {d[1], d[1] ? one : 0}, {d[2], d[2] ? one * (size_t)gate_count(spec, n) : 0}, {d[3], d[3] ? one : 0},
                  {d[4], d[4] ? one : 0}, {workspace, need}, rows_buf(r[2], n, spec->dim),
                  rows_buf(r[3], n, spec->dim), rows_buf(r[4], n, spec->dim), rows_buf(r[5], n, spec->dim),
                  {stats, (size_t)n * 16}};
  Buf vecs[5];
  vector_bufs(spec, n, vecs);
  std::copy(vecs, vecs + 5, bufs + 13);
  if (same_rows(r[0], r[2])) bufs[8].bytes = 0;              // in place
  if (same_rows(r[1], r[3])) bufs[9].bytes = 0;
  if (any_overlap(bufs, 18, 8)) return MFSDP_ERR_OVERLAP;
  NormGradArgs g{};
  fill_norm(g.f, spec, n, r[4], r[5]);
  g.f.vec = norm_vectors(spec, r, 6, n);
  g.stats = reinterpret_cast<const float4*>(stats);
  g.d_out = d_out;
  g.d_out_step.row = step_of(r[2]);
  g.d_normed = d_normed;
  g.d_normed_step.row = step_of(r[3]);
  g.d_residual = d_residual;
  g.d_residual_step.row = step_of(r[0]);
  g.d_branch = d_branch;
  g.d_branch_step.row = step_of(r[1]);
  g.d_w_post = d[0];
  g.d_b_post = d[1];
  g.d_gate = gate_sums ? d[2] : nullptr;
  g.d_w_pre = d[3];
  g.d_b_pre = d[4];
  g.accumulate = gv.accumulate;
  g.status = static_cast<int32_t*>(workspace);
  g.parts = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + 256);
  const OpRange range("mfsdp block norm gradient");
  return cuda_status(launch_norm_grad(g, static_cast<cudaStream_t>(stream)));
}
