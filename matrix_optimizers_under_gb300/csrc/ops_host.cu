// Host side of the operators next to the owner step: argument checks, the
// workspace layouts and the launches of the gradient norm and clipping, the id
// sort, the embedding lookup and gradient, and the products grouped by expert.
#include <climits>
#include <cmath>
#include <cstring>
#include <mutex>
#include <new>
#include <vector>

#include <nvtx3/nvToolsExt.h>

#include "mfsdp.h"
#include "ops_internal.h"

namespace mfsdp {
namespace ops {

int sm_count() {
  static std::mutex mu;
  static int sms[kMaxDevices] = {};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return 0;
  std::lock_guard<std::mutex> lock(mu);
  if (sms[dev] == 0 && cudaDeviceGetAttribute(&sms[dev], cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    sms[dev] = 0;
  return sms[dev];
}

namespace {

// NVTX range around the queuing of one operator.
struct OpRange {
  explicit OpRange(const char* name) { nvtxRangePushA(name); }
  ~OpRange() { nvtxRangePop(); }
  OpRange(const OpRange&) = delete;
  OpRange& operator=(const OpRange&) = delete;
};

// Bytes from the first to the last element of `n` rows of `width` elements.
// The callers bound n * ld below 2^60 first.
size_t extent(int64_t n, int64_t ld, int64_t width, size_t elem) {
  return n <= 0 || width <= 0 ? 0 : (size_t)((n - 1) * ld + width) * elem;
}

// n rows of `width` elements, ld apart: inside the index range of the kernels.
bool rows_fit(int64_t n, int64_t ld, int64_t width) {
  return ld >= width && ld <= (int64_t)1 << 40 && n <= (int64_t)INT32_MAX && (n <= 1 || ld <= ((int64_t)1 << 60) / n);
}

// ------------------------------------------------- gradient norm and clipping
constexpr int64_t kMaxChunks = (int64_t)1 << 30;
constexpr int kMaxClipBlocks = 2048;     // CTAs (and partial sums) of one launch

// Chunks of a tensor: its 16-byte vectors from the first boundary on, 32 KB a
// chunk (the elements before and after them go with the first and last one).
int64_t chunks_of(const mfsdp_grad_tensor& t) {
  if (t.numel == 0) return 0;
  const size_t es = dtype_size(t.src_dtype);
  const int64_t head = (int64_t)(((16 - (reinterpret_cast<uintptr_t>(t.src) & 15)) & 15) / es);
  const int64_t vecs = t.numel <= head ? 0 : (t.numel - head) / (int64_t)(16 / es);
  return std::max<int64_t>(1, (vecs + kClipChunkBytes / 16 - 1) / (kClipChunkBytes / 16));
}

// The checks shared by the norm and the clipping; `clip`: the destinations too.
int check_clip(const mfsdp_grad_tensor* t, int32_t n, double max_norm, double eps, bool clip) {
  if (n < 0 || (n > 0 && !t)) return MFSDP_ERR_INVALID_ARG;
  if (std::isnan(max_norm) || max_norm < 0.0 || !std::isfinite(eps) || eps < 0.0) return MFSDP_ERR_INVALID_ARG;
  int64_t chunks = 0;
  for (int i = 0; i < n; ++i) {
    if (!known_dtype(t[i].src_dtype) || (clip && !known_dtype(t[i].dst_dtype))) return MFSDP_ERR_UNSUPPORTED_DTYPE;
    if (t[i].numel < 0 || t[i].numel > (int64_t)1 << 48) return MFSDP_ERR_INVALID_ARG;
    if (t[i].numel == 0) continue;
    if (!t[i].src || (clip && !t[i].dst)) return MFSDP_ERR_INVALID_ARG;
    if (!aligned(t[i].src, dtype_size(t[i].src_dtype)) || (clip && !aligned(t[i].dst, dtype_size(t[i].dst_dtype))))
      return MFSDP_ERR_MISALIGNED;
    chunks += chunks_of(t[i]);
    if (chunks > kMaxChunks) return MFSDP_ERR_UNSUPPORTED_SHAPE;
  }
  return MFSDP_OK;
}

struct Interval {
  uintptr_t lo, hi;
  int32_t tensor;
};

bool by_lo(const Interval& a, const Interval& b) { return a.lo < b.lo; }

// Destinations must be apart from each other, from the other tensors' sources,
// and from their own source unless they are it (in place, one dtype).
int check_clip_overlap(const mfsdp_grad_tensor* t, int32_t n, const void* out, const void* ws, size_t ws_bytes) try {
  std::vector<Interval> src, dst;
  src.reserve(n);
  dst.reserve(n);
  for (int i = 0; i < n; ++i) {
    if (t[i].numel == 0) continue;
    const size_t sb = (size_t)t[i].numel * dtype_size(t[i].src_dtype);
    const size_t db = (size_t)t[i].numel * dtype_size(t[i].dst_dtype);
    if (ranges_overlap(t[i].dst, db, out, 8) || ranges_overlap(t[i].dst, db, ws, ws_bytes)) return MFSDP_ERR_OVERLAP;
    const uintptr_t s = reinterpret_cast<uintptr_t>(t[i].src), d = reinterpret_cast<uintptr_t>(t[i].dst);
    src.push_back({s, s + sb, i});
    dst.push_back({d, d + db, i});
  }
  if (!std::is_sorted(src.begin(), src.end(), by_lo)) std::sort(src.begin(), src.end(), by_lo);
  if (!std::is_sorted(dst.begin(), dst.end(), by_lo)) std::sort(dst.begin(), dst.end(), by_lo);
  for (size_t i = 1; i < dst.size(); ++i)
    if (dst[i - 1].hi > dst[i].lo) return MFSDP_ERR_OVERLAP;
  // The sources may overlap each other, so a source that reaches far past the
  // next one's start hides none of them: every destination is held against the
  // sources that start before its end, from the first whose running end
  // passes its start.
  std::vector<uintptr_t> reach(src.size());
  uintptr_t far = 0;
  for (size_t i = 0; i < src.size(); ++i) reach[i] = far = std::max(far, src[i].hi);
  size_t j = 0;
  for (const Interval& d : dst) {
    while (j < src.size() && reach[j] <= d.lo) ++j;
    for (size_t k = j; k < src.size() && src[k].lo < d.hi; ++k) {
      if (src[k].hi <= d.lo) continue;
      const mfsdp_grad_tensor& g = t[d.tensor];
      if (src[k].tensor != d.tensor || g.src != g.dst || g.src_dtype != g.dst_dtype) return MFSDP_ERR_OVERLAP;
    }
  }
  return MFSDP_OK;
} catch (...) {                                           // no host memory for the tables: nothing leaves a C entry
  return MFSDP_ERR_CUDA;
}

int clip_blocks(int64_t chunks, int sms) {
  return (int)std::min<int64_t>(chunks, std::min(8 * sms, kMaxClipBlocks));
}

int run_clip(const mfsdp_grad_tensor* t, int32_t n, double max_norm, double eps, float* out, void* ws,
             size_t ws_bytes, cudaStream_t stream, bool clip) {
  int st = check_clip(t, n, max_norm, eps, clip);
  if (st != MFSDP_OK) return st;
  if (!out || !ws) return MFSDP_ERR_INVALID_ARG;
  if (!aligned(out, 8) || !aligned(ws, 256)) return MFSDP_ERR_MISALIGNED;
  const size_t need = mfsdp_grad_clip_workspace_bytes(n);
  if (ws_bytes < need) return MFSDP_ERR_WORKSPACE_TOO_SMALL;
  if (ranges_overlap(out, 8, ws, need)) return MFSDP_ERR_OVERLAP;
  for (int i = 0; i < n; ++i) {
    const size_t sb = (size_t)t[i].numel * dtype_size(t[i].src_dtype);
    if (ranges_overlap(t[i].src, sb, out, 8) || ranges_overlap(t[i].src, sb, ws, need)) return MFSDP_ERR_OVERLAP;
  }
  if (clip) {
    st = check_clip_overlap(t, n, out, ws, need);
    if (st != MFSDP_OK) return st;
  }
  const int sms = sm_count();
  if (sms <= 0) return MFSDP_ERR_CUDA;
  const OpRange range(clip ? "mfsdp grad clip" : "mfsdp grad norm");
  // Launches of at most kClipTable tensors: all sums first, then the scaling,
  // whose launches add up all partial sums.
  cudaStream_t s = stream;
  const auto fill = [&](ClipBatch<kClipTable>& b, int& i) {
    b.n = 0;
    int64_t chunks = 0;
    for (; i < n && b.n < kClipTable; ++i) {
      if (t[i].numel == 0) continue;
      ClipTensor& c = b.t[b.n++];
      c.src = t[i].src;
      c.dst = clip ? t[i].dst : nullptr;
      c.numel = t[i].numel;
      c.chunk0 = (int32_t)chunks;
      c.src_bf16 = t[i].src_dtype == MFSDP_DTYPE_BF16;
      c.dst_bf16 = t[i].dst_dtype == MFSDP_DTYPE_BF16;
      chunks += chunks_of(t[i]);
    }
    b.chunks = (int32_t)chunks;
  };
  ClipBatch<kClipTable> b;
  b.partials = static_cast<double*>(ws);
  b.out = out;
  b.max_norm = max_norm;
  b.eps = eps;
  b.first_partial = b.n_partials = 0;
  cudaError_t e = cudaSuccess;
  int launches = 0;
  for (int i = 0; i < n || launches == 0; ++launches) {
    fill(b, i);
    if (b.chunks == 0) continue;
    const int blocks = clip_blocks(b.chunks, sms);
    e = launch_clip_norm(b, blocks, s);
    if (e != cudaSuccess) return cuda_status(e);
    b.first_partial += blocks;
  }
  b.n_partials = b.first_partial;
  if (!clip || b.n_partials == 0) return cuda_status(launch_clip_finish(b, s));
  b.first_partial = 0;
  bool first = true;
  for (int i = 0; i < n;) {
    if (launches > 1) fill(b, i);
    else i = n;                                                  // still filled
    if (b.chunks == 0) continue;
    const int blocks = clip_blocks(b.chunks, sms);
    e = launch_clip_scale(b, blocks, first, s);
    if (e != cudaSuccess) return cuda_status(e);
    first = false;
    b.first_partial += blocks;
  }
  return MFSDP_OK;
}

// ------------------------------------------------------------ sort, embedding
bool known_id_type(int32_t t) { return t == MFSDP_ID_I32 || t == MFSDP_ID_I64; }
size_t id_size(int32_t t) { return t == MFSDP_ID_I64 ? 8 : 4; }

int check_ids(const void* ids, int32_t id_type, int64_t n, int64_t n_keys) {
  if (!known_id_type(id_type)) return MFSDP_ERR_UNSUPPORTED_DTYPE;
  if (n < 0 || n_keys < 1) return MFSDP_ERR_INVALID_ARG;
  if (n > INT32_MAX || n_keys >= INT32_MAX) return MFSDP_ERR_UNSUPPORTED_SHAPE;
  if (n > 0 && !ids) return MFSDP_ERR_INVALID_ARG;
  if (n > 0 && !aligned(ids, id_size(id_type))) return MFSDP_ERR_MISALIGNED;
  return MFSDP_OK;
}

// Workspace of the embedding gradient: sorted keys, their positions, the
// sort's scratch, the partial rows.
struct EmbedLayout {
  size_t keys, order, sort, partials, bytes;
};
EmbedLayout embed_layout(int64_t n, int64_t vocab, int64_t dim) {
  EmbedLayout l;
  size_t off = 256;                                         // the status word
  l.keys = off; off += round_up((size_t)n * 4, 256);
  l.order = off; off += round_up((size_t)n * 4, 256);
  l.sort = off; off += round_up(sort_scratch_bytes(n, vocab), 256);
  l.partials = off; off += round_up(embed_grad_partial_bytes(n, vocab, dim), 256);
  l.bytes = off;
  return l;
}

// The kernels take the scale in fp32: finite there too.
bool scale_ok(double scale) { return std::isfinite((float)scale); }

bool embed_shape_ok(int64_t n, int64_t vocab, int64_t dim) {
  return n >= 0 && n <= INT32_MAX && vocab >= 1 && vocab < INT32_MAX && dim >= 1 && dim <= (1 << 24);
}

// ------------------------------------------------------ products by expert
int check_expert_shape(int32_t n_experts, int64_t n_rows, int64_t rows, int64_t cols) {
  if (n_experts < 1 || n_rows < 0 || rows < 1 || cols < 1) return MFSDP_ERR_INVALID_ARG;
  if (n_experts > MFSDP_MAX_EXPERTS || n_rows > (1 << 30) || rows > (1 << 24) || cols > (1 << 24))
    return MFSDP_ERR_UNSUPPORTED_SHAPE;
  // the kernels count 256 x 256 tiles in int32, in each of the three products
  const int64_t tr = (rows + 255) / 256, tc = (cols + 255) / 256, tn = n_rows / 256 + n_experts;
  if (std::max(n_experts * tr * tc, std::max(tr, tc) * tn) > (1 << 30)) return MFSDP_ERR_UNSUPPORTED_SHAPE;
  return MFSDP_OK;
}

// Elements between the first and the end of the last of n matrices; 0 if the
// count leaves the index range.
int64_t stack_extent(int32_t n, int64_t stride, int64_t rows, int64_t cols) {
  if (n > 1 && (stride < rows * cols || stride > ((int64_t)1 << 56) / n)) return 0;
  return (n > 1 ? (n - 1) * stride : 0) + rows * cols;
}

int check_workspace(const void* ws, size_t ws_bytes, size_t need) {
  if (!ws) return MFSDP_ERR_INVALID_ARG;
  if (!aligned(ws, 256)) return MFSDP_ERR_MISALIGNED;
  if (ws_bytes < need) return MFSDP_ERR_WORKSPACE_TOO_SMALL;
  return MFSDP_OK;
}

struct Buf {
  const void* p;
  size_t bytes;
};

// The first `writes` buffers are written: apart from each other and the rest.
bool any_overlap(const Buf* b, int n, int writes) {
  for (int i = 0; i < writes; ++i)
    for (int j = i + 1; j < n; ++j)
      if (ranges_overlap(b[i].p, b[i].bytes, b[j].p, b[j].bytes)) return true;
  return false;
}

}  // namespace
}  // namespace ops
}  // namespace mfsdp

using namespace mfsdp;
using namespace mfsdp::ops;

// ---------------------------------------------------- gradient norm, clipping
extern "C" size_t mfsdp_grad_clip_workspace_bytes(int32_t n) {
  if (n < 0) return 0;
  const size_t launches = std::max<size_t>(1, ((size_t)n + kClipTable - 1) / kClipTable);
  return launches * kMaxClipBlocks * sizeof(double);
}

extern "C" int mfsdp_grad_norm(const mfsdp_grad_tensor* tensors, int32_t n, double max_norm, double eps, float* out,
                               void* workspace, size_t workspace_bytes, void* stream) {
  return run_clip(tensors, n, max_norm, eps, out, workspace, workspace_bytes, static_cast<cudaStream_t>(stream),
                  false);
}

extern "C" int mfsdp_grad_clip(const mfsdp_grad_tensor* tensors, int32_t n, double max_norm, double eps, float* out,
                               void* workspace, size_t workspace_bytes, void* stream) {
  return run_clip(tensors, n, max_norm, eps, out, workspace, workspace_bytes, static_cast<cudaStream_t>(stream),
                  true);
}

// ------------------------------------------------------------------------ sort
extern "C" size_t mfsdp_sort_ids_workspace_bytes(int64_t n, int64_t n_keys) {
  if (n < 0 || n > INT32_MAX || n_keys < 1 || n_keys >= INT32_MAX) return 0;
  return round_up((size_t)n * 4, 256) + std::max<size_t>(256, sort_scratch_bytes(n, n_keys));
}

extern "C" int mfsdp_sort_ids(const void* ids, int32_t id_type, int64_t n, int64_t n_keys, int32_t* order,
                              int32_t* starts, void* workspace, size_t workspace_bytes, void* stream_ptr) {
  int st = check_ids(ids, id_type, n, n_keys);
  if (st != MFSDP_OK) return st;
  if ((n > 0 && !order) || !starts) return MFSDP_ERR_INVALID_ARG;
  if (!aligned(order, 4) || !aligned(starts, 4)) return MFSDP_ERR_MISALIGNED;
  const size_t need = mfsdp_sort_ids_workspace_bytes(n, n_keys);
  st = check_workspace(workspace, workspace_bytes, need);
  if (st != MFSDP_OK) return st;
  const Buf bufs[4] = {{order, (size_t)n * 4}, {starts, (size_t)(n_keys + 1) * 4}, {workspace, need},
                       {ids, (size_t)n * id_size(id_type)}};
  if (any_overlap(bufs, 4, 3)) return MFSDP_ERR_OVERLAP;
  const OpRange range("mfsdp sort ids");
  cudaStream_t stream = static_cast<cudaStream_t>(stream_ptr);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  SortArgs a{};
  a.ids = ids;
  a.ids64 = id_type == MFSDP_ID_I64;
  a.n = n;
  a.n_keys = n_keys;
  a.keys_out = reinterpret_cast<int32_t*>(ws);
  a.order_out = order;
  a.scratch = ws + round_up((size_t)n * 4, 256);
  cudaError_t e = launch_sort(a, stream);
  if (e == cudaSuccess) e = launch_key_starts(a.keys_out, n, n_keys, starts, stream);
  return cuda_status(e);
}

// ------------------------------------------------------------------- embedding
extern "C" int mfsdp_embedding_lookup(const void* weight, int32_t weight_dtype, int64_t vocab, int64_t dim,
                                      int64_t weight_ld, const void* ids, int32_t id_type, int64_t n, double scale,
                                      void* out, int32_t out_dtype, int64_t out_ld, void* stream) {
  if (!known_dtype(weight_dtype) || !known_dtype(out_dtype)) return MFSDP_ERR_UNSUPPORTED_DTYPE;
  int st = check_ids(ids, id_type, n, vocab);
  if (st != MFSDP_OK) return st;
  if (dim < 1 || !scale_ok(scale)) return MFSDP_ERR_INVALID_ARG;
  if (!embed_shape_ok(n, vocab, dim) || !rows_fit(vocab, weight_ld, dim) || !rows_fit(n, out_ld, dim))
    return MFSDP_ERR_UNSUPPORTED_SHAPE;
  if (n == 0) return MFSDP_OK;
  if (!weight || !out) return MFSDP_ERR_INVALID_ARG;
  if (!aligned(weight, 16) || !aligned(out, 16)) return MFSDP_ERR_MISALIGNED;
  const Buf bufs[3] = {{out, extent(n, out_ld, dim, dtype_size(out_dtype))},
                       {weight, extent(vocab, weight_ld, dim, dtype_size(weight_dtype))},
                       {ids, (size_t)n * id_size(id_type)}};
  if (any_overlap(bufs, 3, 1)) return MFSDP_ERR_OVERLAP;
  LookupArgs a{};
  a.w = weight;
  a.ids = ids;
  a.out = out;
  a.vocab = vocab;
  a.dim = dim;
  a.w_ld = weight_ld;
  a.n = n;
  a.out_ld = out_ld;
  a.w_bf16 = weight_dtype == MFSDP_DTYPE_BF16;
  a.out_bf16 = out_dtype == MFSDP_DTYPE_BF16;
  a.ids64 = id_type == MFSDP_ID_I64;
  a.scale = (float)scale;
  const OpRange range("mfsdp embedding lookup");
  return cuda_status(launch_lookup(a, static_cast<cudaStream_t>(stream)));
}

extern "C" size_t mfsdp_embedding_grad_workspace_bytes(int64_t n, int64_t vocab, int64_t dim) {
  return embed_shape_ok(n, vocab, dim) ? embed_layout(n, vocab, dim).bytes : 0;
}

extern "C" int mfsdp_embedding_grad(const void* dout, int32_t dout_dtype, int64_t dout_ld, const void* ids,
                                    int32_t id_type, int64_t n, double scale, void* grad, int32_t grad_dtype,
                                    int64_t vocab, int64_t dim, int64_t grad_ld, int32_t accumulate, void* workspace,
                                    size_t workspace_bytes, void* stream_ptr) {
  if (!known_dtype(dout_dtype) || !known_dtype(grad_dtype)) return MFSDP_ERR_UNSUPPORTED_DTYPE;
  int st = check_ids(ids, id_type, n, vocab);
  if (st != MFSDP_OK) return st;
  if (dim < 1 || !scale_ok(scale) || (accumulate != 0 && accumulate != 1)) return MFSDP_ERR_INVALID_ARG;
  if (!embed_shape_ok(n, vocab, dim) || !rows_fit(vocab, grad_ld, dim) || !rows_fit(n, dout_ld, dim))
    return MFSDP_ERR_UNSUPPORTED_SHAPE;
  if (!grad || (n > 0 && !dout)) return MFSDP_ERR_INVALID_ARG;
  if (!aligned(grad, 16) || (n > 0 && !aligned(dout, 16))) return MFSDP_ERR_MISALIGNED;
  const EmbedLayout l = embed_layout(n, vocab, dim);
  st = check_workspace(workspace, workspace_bytes, l.bytes);
  if (st != MFSDP_OK) return st;
  const Buf bufs[4] = {{grad, extent(vocab, grad_ld, dim, dtype_size(grad_dtype))}, {workspace, l.bytes},
                       {dout, extent(n, dout_ld, dim, dtype_size(dout_dtype))}, {ids, (size_t)n * id_size(id_type)}};
  if (any_overlap(bufs, 4, 2)) return MFSDP_ERR_OVERLAP;
  if (n == 0 && accumulate) return MFSDP_OK;
  cudaStream_t stream = static_cast<cudaStream_t>(stream_ptr);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  SortArgs s{};
  s.ids = ids;
  s.ids64 = id_type == MFSDP_ID_I64;
  s.n = n;
  s.n_keys = vocab;
  s.keys_out = reinterpret_cast<int32_t*>(ws + l.keys);
  s.order_out = reinterpret_cast<int32_t*>(ws + l.order);
  s.scratch = ws + l.sort;
  EmbedGradArgs a{};
  a.dout = dout;
  a.grad = grad;
  a.ids = ids;
  a.ids64 = s.ids64;
  a.keys = s.keys_out;
  a.order = s.order_out;
  a.partials = reinterpret_cast<float*>(ws + l.partials);
  a.n = n;
  a.vocab = vocab;
  a.dim = dim;
  a.dout_ld = dout_ld;
  a.grad_ld = grad_ld;
  a.dout_bf16 = dout_dtype == MFSDP_DTYPE_BF16;
  a.grad_bf16 = grad_dtype == MFSDP_DTYPE_BF16;
  a.accumulate = accumulate;
  a.scale = (float)scale;
  a.header = s.zero = reinterpret_cast<int32_t*>(ws);
  const OpRange range("mfsdp embedding gradient");
  cudaError_t e = embed_grad_sorts(a) ? launch_sort(s, stream) : cudaSuccess;
  if (e == cudaSuccess) e = launch_embed_grad(a, stream);
  return cuda_status(e);
}

// ------------------------------------------------------ products by expert
extern "C" size_t mfsdp_expert_workspace_bytes(int32_t n_experts, int64_t n_rows, int64_t rows, int64_t cols,
                                               int64_t w_stride, int64_t rows_ld, int64_t cols_ld) {
  if (check_expert_shape(n_experts, n_rows, rows, cols) != MFSDP_OK ||
      stack_extent(n_experts, w_stride, rows, cols) == 0 || !rows_fit(n_rows, rows_ld, rows) ||
      !rows_fit(n_rows, cols_ld, cols))
    return 0;
  size_t bytes = 256;                                       // the status word
  if (cols % 8 != 0 || (n_experts > 1 && w_stride % 8 != 0)) bytes += packed_bytes(n_experts * rows, cols);
  if (n_rows > 1 && rows_ld % 8 != 0) bytes += packed_bytes(n_rows, rows);
  if (n_rows > 1 && cols_ld % 8 != 0) bytes += packed_bytes(n_rows, cols);
  // weight gradient: the last rows of each group, padded to 16, of both operands
  if (n_rows > 0) bytes += packed_bytes(16 * (int64_t)n_experts, rows) + packed_bytes(16 * (int64_t)n_experts, cols);
  bytes += expert_split_bytes(n_experts, n_rows, rows, cols);
  return bytes;
}

extern "C" int mfsdp_op_device_status(const void* workspace, void* stream, int32_t* detail) {
  return mfsdp_muon_device_status(workspace, stream, detail);
}

extern "C" int mfsdp_expert_matmul(const void* x, int64_t x_ld, const void* w, int64_t w_stride, int32_t in_dtype,
                                   const int32_t* starts, int32_t n_experts, int64_t n_rows, int64_t rows,
                                   int64_t cols, int32_t input_grad, void* y, int32_t y_dtype, int64_t y_ld,
                                   void* workspace, size_t workspace_bytes, void* stream) {
  if (in_dtype != MFSDP_DTYPE_BF16 || !known_dtype(y_dtype)) return MFSDP_ERR_UNSUPPORTED_DTYPE;
  int st = check_expert_shape(n_experts, n_rows, rows, cols);
  if (st != MFSDP_OK) return st;
  if (input_grad != 0 && input_grad != 1) return MFSDP_ERR_INVALID_ARG;
  const int64_t x_width = input_grad ? rows : cols, y_width = input_grad ? cols : rows;
  const int64_t w_elems = stack_extent(n_experts, w_stride, rows, cols);
  if (w_elems == 0 || !rows_fit(n_rows, x_ld, x_width) || !rows_fit(n_rows, y_ld, y_width))
    return MFSDP_ERR_UNSUPPORTED_SHAPE;
  if (n_rows == 0) return MFSDP_OK;
  if (!x || !w || !y || !starts) return MFSDP_ERR_INVALID_ARG;
  if (!aligned(x, 16) || !aligned(w, 16) || !aligned(y, 16) || !aligned(starts, 4)) return MFSDP_ERR_MISALIGNED;
  const size_t need = mfsdp_expert_workspace_bytes(n_experts, n_rows, rows, cols, w_stride, input_grad ? x_ld : y_ld,
                                                   input_grad ? y_ld : x_ld);
  st = check_workspace(workspace, workspace_bytes, need);
  if (st != MFSDP_OK) return st;
  const Buf bufs[5] = {{y, extent(n_rows, y_ld, y_width, dtype_size(y_dtype))}, {workspace, need},
                       {x, extent(n_rows, x_ld, x_width, 2)}, {w, (size_t)w_elems * 2},
                       {starts, (size_t)(n_experts + 1) * 4}};
  if (any_overlap(bufs, 5, 2)) return MFSDP_ERR_OVERLAP;
  ExpertArgs a{};
  a.mode = input_grad ? kExpertInputGrad : kExpertForward;
  a.n_experts = n_experts;
  a.n_rows = n_rows;
  a.rows = rows;
  a.cols = cols;
  a.a = x;
  a.b = w;
  a.out = y;
  a.starts = starts;
  a.a_ld = x_ld;
  a.b_ld = cols;
  a.b_stride = w_stride;
  a.out_ld = y_ld;
  a.out_bf16 = y_dtype == MFSDP_DTYPE_BF16;
  a.status = static_cast<int32_t*>(workspace);
  a.packs = static_cast<uint8_t*>(workspace) + 256;
  const OpRange range(input_grad ? "mfsdp expert input gradient" : "mfsdp expert matmul");
  return cuda_status(launch_expert(a, static_cast<cudaStream_t>(stream)));
}

extern "C" int mfsdp_expert_weight_grad(const void* dy, int64_t dy_ld, const void* x, int64_t x_ld, int32_t in_dtype,
                                        const int32_t* starts, int32_t n_experts, int64_t n_rows, int64_t rows,
                                        int64_t cols, void* dw, int32_t dw_dtype, int64_t dw_stride,
                                        int32_t accumulate, void* workspace, size_t workspace_bytes, void* stream) {
  if (in_dtype != MFSDP_DTYPE_BF16 || !known_dtype(dw_dtype)) return MFSDP_ERR_UNSUPPORTED_DTYPE;
  int st = check_expert_shape(n_experts, n_rows, rows, cols);
  if (st != MFSDP_OK) return st;
  if (accumulate != 0 && accumulate != 1) return MFSDP_ERR_INVALID_ARG;
  const int64_t dw_elems = stack_extent(n_experts, dw_stride, rows, cols);
  if (dw_elems == 0 || !rows_fit(n_rows, dy_ld, rows) || !rows_fit(n_rows, x_ld, cols))
    return MFSDP_ERR_UNSUPPORTED_SHAPE;
  if (n_rows == 0 && accumulate) return MFSDP_OK;
  if (!dw || !starts || (n_rows > 0 && (!dy || !x))) return MFSDP_ERR_INVALID_ARG;
  if (!aligned(dw, 16) || !aligned(starts, 4) || (n_rows > 0 && (!aligned(dy, 16) || !aligned(x, 16))))
    return MFSDP_ERR_MISALIGNED;
  const size_t need =
      mfsdp_expert_workspace_bytes(n_experts, n_rows, rows, cols, rows * cols, dy_ld, x_ld);
  st = check_workspace(workspace, workspace_bytes, need);
  if (st != MFSDP_OK) return st;
  const Buf bufs[5] = {{dw, (size_t)dw_elems * dtype_size(dw_dtype)}, {workspace, need},
                       {dy, extent(n_rows, dy_ld, rows, 2)}, {x, extent(n_rows, x_ld, cols, 2)},
                       {starts, (size_t)(n_experts + 1) * 4}};
  if (any_overlap(bufs, 5, 2)) return MFSDP_ERR_OVERLAP;
  ExpertArgs a{};
  a.mode = kExpertWeightGrad;
  a.n_experts = n_experts;
  a.n_rows = n_rows;
  a.rows = rows;
  a.cols = cols;
  a.a = dy;
  a.b = x;
  a.out = dw;
  a.starts = starts;
  a.a_ld = dy_ld;
  a.b_ld = x_ld;
  a.out_ld = cols;
  a.out_stride = dw_stride;
  a.out_bf16 = dw_dtype == MFSDP_DTYPE_BF16;
  a.accumulate = accumulate;
  a.status = static_cast<int32_t*>(workspace);
  a.packs = static_cast<uint8_t*>(workspace) + 256;
  const OpRange range("mfsdp expert weight gradient");
  return cuda_status(launch_expert(a, static_cast<cudaStream_t>(stream)));
}
