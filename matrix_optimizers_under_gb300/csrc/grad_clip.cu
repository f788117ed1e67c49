// Global gradient norm over many tensors, and clipping.
//
// Muon's update does not depend on the gradient's scale once the momentum is
// normalised, but the momentum mixes steps of different scale and AdamW's
// moments do too, so training programs clip the gradient by its global norm
// before the step:
//   S = sum over tensors t, elements i of g_ti^2,   norm = sqrt(S)
//   coef = min(1, max_norm / (norm + eps)),         out_ti = round(coef * g_ti)
//
// The norm has to be known before the first output, so this is two passes:
// the first leaves one partial sum per CTA, the second adds all partials (the
// same order in every CTA, so that all use the same coefficient) and scales.
// Every sum has a fixed order: the norm is bitwise reproducible.
//
// Sums: a thread adds the squares of its 64 elements of a chunk in fp32 (eight
// running sums of eight), and everything above that in double, so the norm is
// good to ~1e-7 at any length.  A thread whose fp32 sum left the range where
// that holds (overflow, or a nonzero sum small enough for the squares to lose
// bits below the fp32 range) adds its elements again in double, so
// any finite gradient has a right norm.
#include <cuda_bf16.h>

#include "ops_internal.h"

namespace mfsdp {
namespace ops {
namespace {

constexpr int kThreads = 256;
constexpr int kVec = 8;                                      // elements a thread takes at a time
constexpr int kRounds = kClipChunk / (kThreads * kVec);      // 8

__device__ __forceinline__ int find_tensor(const ClipBatch& p, int chunk) {
  int lo = 0, hi = p.n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (p.t[mid].chunk0 <= chunk) lo = mid; else hi = mid - 1;
  }
  return lo;
}

__device__ __forceinline__ float load1(const void* p, int64_t i, int bf16) {
  return bf16 ? __uint_as_float((uint32_t)static_cast<const uint16_t*>(p)[i] << 16) : static_cast<const float*>(p)[i];
}

__device__ __forceinline__ void store1(void* p, int64_t i, int bf16, float v) {
  if (bf16) static_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(v);
  else static_cast<float*>(p)[i] = v;
}

// 8 consecutive elements with 16-byte loads (the first one 16-byte aligned).
__device__ __forceinline__ void load8(const void* p, int64_t i, int bf16, float (&x)[8]) {
  if (bf16) {
    const uint4 q = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + i);
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      x[2 * k] = __uint_as_float(w[k] << 16);
      x[2 * k + 1] = __uint_as_float(w[k] & 0xFFFF0000u);
    }
  } else {
    const float4* f = reinterpret_cast<const float4*>(static_cast<const float*>(p) + i);
    const float4 a = f[0], b = f[1];
    x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w; x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
  }
}

__device__ __forceinline__ void store8(void* p, int64_t i, int bf16, const float (&x)[8]) {
  if (bf16) {
    __nv_bfloat162 h[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) h[k] = __floats2bfloat162_rn(x[2 * k], x[2 * k + 1]);
    *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p) + i) = *reinterpret_cast<const uint4*>(h);
  } else {
    float4* f = reinterpret_cast<float4*>(static_cast<float*>(p) + i);
    f[0] = make_float4(x[0], x[1], x[2], x[3]);
    f[1] = make_float4(x[4], x[5], x[6], x[7]);
  }
}

// Elements before the tensor's first 16-byte boundary.
__device__ __forceinline__ int head_of(const void* p, int bf16) {
  const int bytes = (int)((16 - (reinterpret_cast<uintptr_t>(p) & 15)) & 15);
  return bf16 ? bytes >> 1 : bytes >> 2;
}

// Chunk c of a tensor of numel elements is [16384 c, 16384 (c + 1)), moved up
// to the boundary: elements [head + 16384 c, ...), the first chunk with the
// head, so that every vector of every chunk is aligned.
struct Span {
  int64_t lo, hi;
};
__device__ __forceinline__ Span chunk_span(const ClipTensor& t, int c, int head) {
  Span s;
  s.lo = head + (int64_t)c * kClipChunk;
  s.hi = s.lo + kClipChunk < t.numel ? s.lo + kClipChunk : t.numel;
  return s;
}

constexpr float kSumMax = 1e37f, kSumMin = 1e-20f;

__device__ __forceinline__ double block_sum(double v, double* warp_sum) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) warp_sum[threadIdx.x >> 5] = v;
  __syncthreads();
  double s = 0.0;
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) s += warp_sum[w];
  return s;
}

__global__ void __launch_bounds__(kThreads) clip_norm_kernel(const __grid_constant__ ClipBatch p) {
  __shared__ double warp_sum[kThreads / 32];
  double total = 0.0;
  for (int ch = blockIdx.x; ch < p.chunks; ch += gridDim.x) {
    const ClipTensor& t = p.t[find_tensor(p, ch)];
    const int c = ch - t.chunk0;
    const int head = head_of(t.src, t.src_bf16);
    const Span sp = chunk_span(t, c, head);
    float acc[kVec] = {};
    bool any = false;
    for (int64_t i = sp.lo + (int64_t)threadIdx.x * kVec; i < sp.hi; i += kThreads * kVec) {
      float x[kVec];
      if (i + kVec <= sp.hi) {
        load8(t.src, i, t.src_bf16, x);
      } else {
#pragma unroll
        for (int k = 0; k < kVec; ++k) x[k] = i + k < sp.hi ? load1(t.src, i + k, t.src_bf16) : 0.f;
      }
#pragma unroll
      for (int k = 0; k < kVec; ++k) {
        acc[k] = fmaf(x[k], x[k], acc[k]);
        any |= x[k] != 0.f;
      }
    }
    const bool extra = c == 0 && (int)threadIdx.x < head && (int)threadIdx.x < t.numel;
    if (extra) {
      const float x = load1(t.src, threadIdx.x, t.src_bf16);
      acc[0] = fmaf(x, x, acc[0]);
      any |= x != 0.f;
    }
    const float s = ((acc[0] + acc[1]) + (acc[2] + acc[3])) + ((acc[4] + acc[5]) + (acc[6] + acc[7]));
    if (any && !(s >= kSumMin && s <= kSumMax)) {
      double d = 0.0;
      for (int64_t i = sp.lo + (int64_t)threadIdx.x * kVec; i < sp.hi; i += kThreads * kVec)
        for (int k = 0; k < kVec; ++k)
          if (i + k < sp.hi) {
            const double x = load1(t.src, i + k, t.src_bf16);
            d += x * x;
          }
      if (extra) {
        const double x = load1(t.src, threadIdx.x, t.src_bf16);
        d += x * x;
      }
      total += d;
    } else {
      total += s;
    }
  }
  const double s = block_sum(total, warp_sum);
  if (threadIdx.x == 0) p.partials[p.first_partial + blockIdx.x] = s;
}

// The norm and the coefficient from all partial sums.
__device__ __forceinline__ float finish_norm(const ClipBatch& p, double* warp_sum, float* norm_out) {
  double v = 0.0;
  for (int i = threadIdx.x; i < p.n_partials; i += kThreads) v += p.partials[i];
  const double norm = sqrt(block_sum(v, warp_sum));
  const double den = norm + p.eps;
  double c = 1.0;                                   // an infinite limit, or nothing to scale
  if (!isinf(p.max_norm) && den != 0.0) c = p.max_norm / den;
  if (c > 1.0) c = 1.0;                             // a NaN stays one
  *norm_out = (float)norm;
  return (float)c;
}

__global__ void __launch_bounds__(kThreads) clip_finish_kernel(const __grid_constant__ ClipBatch p) {
  __shared__ double warp_sum[kThreads / 32];
  float norm;
  const float coef = finish_norm(p, warp_sum, &norm);
  if (threadIdx.x == 0) {
    p.out[0] = norm;
    p.out[1] = coef;
  }
}

__global__ void __launch_bounds__(kThreads) clip_scale_kernel(const __grid_constant__ ClipBatch p) {
  __shared__ double warp_sum[kThreads / 32];
  float norm;
  const float coef = finish_norm(p, warp_sum, &norm);
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    p.out[0] = norm;
    p.out[1] = coef;
  }
  for (int ch = blockIdx.x; ch < p.chunks; ch += gridDim.x) {
    const ClipTensor& t = p.t[find_tensor(p, ch)];
    if (coef == 1.0f && t.src == t.dst) continue;   // in place and not clipped: nothing changes
    const int c = ch - t.chunk0;
    const int head = head_of(t.src, t.src_bf16);
    const Span sp = chunk_span(t, c, head);
    const bool vec = head_of(static_cast<char*>(t.dst) + (int64_t)head * (t.dst_bf16 ? 2 : 4), t.dst_bf16) == 0;
    for (int64_t i = sp.lo + (int64_t)threadIdx.x * kVec; i < sp.hi; i += kThreads * kVec) {
      float x[kVec];
      if (i + kVec <= sp.hi) {
        load8(t.src, i, t.src_bf16, x);
#pragma unroll
        for (int k = 0; k < kVec; ++k) x[k] *= coef;
        if (vec) {
          store8(t.dst, i, t.dst_bf16, x);
        } else {
#pragma unroll
          for (int k = 0; k < kVec; ++k) store1(t.dst, i + k, t.dst_bf16, x[k]);
        }
      } else {
        for (int64_t j = i; j < sp.hi; ++j) store1(t.dst, j, t.dst_bf16, load1(t.src, j, t.src_bf16) * coef);
      }
    }
    if (c == 0 && (int)threadIdx.x < head && (int)threadIdx.x < t.numel)
      store1(t.dst, threadIdx.x, t.dst_bf16, load1(t.src, threadIdx.x, t.src_bf16) * coef);
  }
}

}  // namespace

cudaError_t launch_clip_norm(const ClipBatch& b, int blocks, cudaStream_t s) {
  clip_norm_kernel<<<blocks, kThreads, 0, s>>>(b);
  return cudaGetLastError();
}
cudaError_t launch_clip_finish(const ClipBatch& b, cudaStream_t s) {
  clip_finish_kernel<<<1, kThreads, 0, s>>>(b);
  return cudaGetLastError();
}
cudaError_t launch_clip_scale(const ClipBatch& b, int blocks, cudaStream_t s) {
  clip_scale_kernel<<<blocks, kThreads, 0, s>>>(b);
  return cudaGetLastError();
}

}  // namespace ops
}  // namespace mfsdp
