// Embedding lookup with scaling, and its gradient by sorted tokens.
//
//   lookup:    out[t, :]  = scale * W[id_t, :]          (zeros for an id outside [0, vocab))
//   gradient:  dW[v, :] (+)= scale * sum over t with id_t = v of dout[t, :]
//
// The embedding is the largest tensor of the AdamW tail; its gradient is dense
// there (a row no token names is zero, and AdamW still decays its moments), so
// the gradient writes every row of dW once, or with `accumulate` adds to the
// rows that tokens name.
//
// The gradient walks positions sorted by token (stable), so a row's sum runs
// in ascending position in fp32: no atomics, bitwise reproducible.
#include <cuda_bf16.h>

#include "ops_internal.h"

namespace mfsdp {
namespace ops {
namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ float load1(const void* p, int64_t i, int bf16) {
  return bf16 ? __uint_as_float((uint32_t)static_cast<const uint16_t*>(p)[i] << 16) : static_cast<const float*>(p)[i];
}
__device__ __forceinline__ void store1(void* p, int64_t i, int bf16, float v) {
  if (bf16) static_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(v);
  else static_cast<float*>(p)[i] = v;
}

__global__ void __launch_bounds__(kThreads) lookup_kernel(const __grid_constant__ LookupArgs a) {
  for (int64_t t = blockIdx.x; t < a.n; t += gridDim.x) {
    const int64_t id = a.ids64 ? static_cast<const int64_t*>(a.ids)[t] : static_cast<const int32_t*>(a.ids)[t];
    const bool ok = id >= 0 && id < a.vocab;
    for (int64_t c = threadIdx.x; c < a.dim; c += kThreads)
      store1(a.out, t * a.out_ld + c, a.out_bf16, ok ? a.scale * load1(a.w, id * a.w_ld + c, a.w_bf16) : 0.f);
  }
}

// First sorted position whose key is not below v.
__device__ __forceinline__ int64_t lower_bound(const int32_t* keys, int64_t n, int64_t v) {
  int64_t lo = 0, hi = n;
  while (lo < hi) {
    const int64_t mid = (lo + hi) >> 1;
    if (keys[mid] < v) lo = mid + 1; else hi = mid;
  }
  return lo;
}

// One row of dW at a time.
__global__ void __launch_bounds__(kThreads) embed_grad_kernel(const __grid_constant__ EmbedGradArgs a) {
  for (int64_t v = blockIdx.x; v < a.vocab; v += gridDim.x) {
    const int64_t lo = lower_bound(a.keys, a.n, v), hi = lower_bound(a.keys, a.n, v + 1);
    if (lo == hi && a.accumulate) continue;
    for (int64_t c = threadIdx.x; c < a.dim; c += kThreads) {
      float s = 0.f;
      for (int64_t i = lo; i < hi; ++i) s += load1(a.dout, (int64_t)a.order[i] * a.dout_ld + c, a.dout_bf16);
      s *= a.scale;
      if (a.accumulate) s += load1(a.grad, v * a.grad_ld + c, a.grad_bf16);
      store1(a.grad, v * a.grad_ld + c, a.grad_bf16, s);
    }
  }
}

}  // namespace

cudaError_t launch_lookup(const LookupArgs& a, cudaStream_t s) {
  const int64_t blocks = std::min<int64_t>(a.n, (int64_t)sm_count() * 8);
  if (blocks <= 0) return cudaErrorInvalidConfiguration;
  lookup_kernel<<<(unsigned)blocks, kThreads, 0, s>>>(a);
  return cudaGetLastError();
}

size_t embed_grad_partial_bytes(int64_t, int64_t, int64_t) { return 0; }

cudaError_t launch_embed_grad(const EmbedGradArgs& a, cudaStream_t s) {
  const int64_t blocks = std::min<int64_t>(a.vocab, (int64_t)sm_count() * 8);
  if (blocks <= 0) return cudaErrorInvalidConfiguration;
  embed_grad_kernel<<<(unsigned)blocks, kThreads, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace ops
}  // namespace mfsdp
