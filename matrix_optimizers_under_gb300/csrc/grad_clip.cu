// Global gradient norm over many tensors, and clipping.
//
// Muon's update does not depend on the gradient's scale once the momentum is
// normalised, but the momentum mixes steps of different scale and AdamW's
// moments do too, so training programs clip the gradient by its global norm
// before the step:
//   S = sum over tensors t, elements i of g_ti^2,   norm = sqrt(S)
//   coef = min(1, max_norm / (norm + eps)),         out_ti = round(coef * g_ti)
// (an infinite limit clips nothing, not even an infinite norm; a NaN stays one).
//
// The norm has to be known before the first output, so the data is read twice.
// The first launch leaves one partial sum per CTA, the second adds all
// partials (the same order in every CTA, so that all use the same coefficient)
// and scales.  It takes the chunks from the last to the first: what the first
// launch read last is still in L2.  Its first chunk's loads go out before the
// norm is there.  Every sum has a fixed order: the norm is bitwise reproducible.
//
// Double arithmetic is scarce (2 operations a clock and SM): with the sums and the
// root in every thread, the second launch spent 4 us a CTA on them.  One warp
// adds the partials, and one thread works out the coefficient.
//
// 872 M bf16 elements in 28 matrices: 783 us, 240 for the first launch (7.3 TB/s) and 533
// for the second (6.4 TB/s, half of it writes).  135 k fp32 elements: 5.3 us.
//
// Bound by HBM (by launches, for a small set).  A chunk is 32 KB of one tensor,
// eight 16-byte loads a thread, all issued before the first is used; a tensor
// may start at any element, its chunks start at its first 16-byte boundary.
//
// Sums: a thread adds the squares of its eight vectors of a chunk in fp32 (a
// running sum for each place in the vector), and everything above that in
// double, so the norm is good to ~1e-7 at any length.  A thread whose fp32 sum
// left the range where that holds (overflow, or a nonzero sum small enough for
// the squares to lose bits below the fp32 range) adds its elements again in
// double, so any finite gradient has a right norm.
#include <cuda_bf16.h>

#include <cstring>

#include "ops_internal.h"
#include "ops_ptx.cuh"

namespace mfsdp {
namespace ops {
namespace {

constexpr int kThreads = 256;
constexpr int kVecs = kClipChunkBytes / 16 / kThreads;       // 8 vectors of a thread
constexpr float kSumMax = 1e37f, kSumMin = 1e-20f;

template <int kN>
__device__ __forceinline__ int find_tensor(const ClipBatch<kN>& p, int chunk) {
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

// Chunk c of a tensor: its vectors, which start at the tensor's first 16-byte
// boundary (head elements in), and the elements outside any vector, up to 7 before the
// first (with chunk 0) and up to 7 after the last (with the last chunk).
struct Span {
  const uint4* v;      // this thread's first vector; the next ones kThreads apart
  int vecs;            // how many of this thread's kVecs exist
  int64_t first;       // element index of this thread's first vector
  int64_t odd;         // this thread's element outside the vectors, or -1
};
__device__ __forceinline__ Span chunk_span(const ClipTensor& t, int c, int tid) {
  const int per = t.src_bf16 ? 8 : 4, esz = t.src_bf16 ? 2 : 4;
  int64_t head = (int64_t)((16 - (reinterpret_cast<uintptr_t>(t.src) & 15)) & 15) / esz;
  if (head > t.numel) head = t.numel;
  const int64_t all = (t.numel - head) / per;                 // vectors of the tensor
  const int64_t v0 = (int64_t)c * (kClipChunkBytes / 16) + tid;
  const int64_t left = all - v0;
  Span s;
  s.v = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(t.src) + head * esz) + v0;
  s.vecs = left <= 0 ? 0 : (int)min((int64_t)kVecs, (left + kThreads - 1) / kThreads);
  s.first = head + v0 * per;
  s.odd = -1;
  if (c == 0 && tid < head) s.odd = tid;
  const int64_t end = head + all * per;                       // elements from here on are in no vector
  if ((int64_t)(c + 1) * (kClipChunkBytes / 16) >= all && tid >= 8 && end + tid - 8 < t.numel) s.odd = end + tid - 8;
  return s;
}

__device__ __forceinline__ void load_vecs(const Span& s, uint4 (&q)[kVecs]) {
#pragma unroll
  for (int k = 0; k < kVecs; ++k)
    if (k < s.vecs) q[k] = s.v[k * kThreads];
}

__device__ __forceinline__ float lo16(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi16(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// Sum of squares of this thread's elements of a chunk.
__device__ __forceinline__ double chunk_sum(const ClipTensor& t, int c, int tid) {
  const Span s = chunk_span(t, c, tid);
  uint4 q[kVecs];
  load_vecs(s, q);
  float acc[8] = {};
  uint32_t any = 0;
#pragma unroll
  for (int k = 0; k < kVecs; ++k) {
    if (k >= s.vecs) break;
    const uint32_t w[4] = {q[k].x, q[k].y, q[k].z, q[k].w};
    if (t.src_bf16) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        any |= w[j] & 0x7FFF7FFFu;
        acc[2 * j] = fmaf(lo16(w[j]), lo16(w[j]), acc[2 * j]);
        acc[2 * j + 1] = fmaf(hi16(w[j]), hi16(w[j]), acc[2 * j + 1]);
      }
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        any |= w[j] & 0x7FFFFFFFu;
        acc[j] = fmaf(__uint_as_float(w[j]), __uint_as_float(w[j]), acc[j]);
      }
    }
  }
  if (s.odd >= 0) {
    const float x = load1(t.src, s.odd, t.src_bf16);
    any |= x != 0.f;
    acc[7] = fmaf(x, x, acc[7]);
  }
  const float sum = ((acc[0] + acc[1]) + (acc[2] + acc[3])) + ((acc[4] + acc[5]) + (acc[6] + acc[7]));
  if (any == 0 || (sum >= kSumMin && sum <= kSumMax)) return sum;
  double d = 0.0;
  const int per = t.src_bf16 ? 8 : 4;
  for (int k = 0; k < s.vecs; ++k)
    for (int j = 0; j < per; ++j) {
      const double x = load1(t.src, s.first + (int64_t)k * kThreads * per + j, t.src_bf16);
      d += x * x;
    }
  if (s.odd >= 0) {
    const double x = load1(t.src, s.odd, t.src_bf16);
    d += x * x;
  }
  return d;
}

// out = coef * g for this thread's elements of a chunk.
__device__ __forceinline__ void chunk_scale(const ClipTensor& t, const Span& s, const uint4 (&q)[kVecs], int tid,
                                            float coef) {
  const int per = t.src_bf16 ? 8 : 4;
  uint8_t* d = static_cast<uint8_t*>(t.dst) + s.first * (t.dst_bf16 ? 2 : 4);
  const int64_t step = (int64_t)kThreads * per * (t.dst_bf16 ? 2 : 4);
  // a vector's outputs: 16 bytes in the same type, 32 (two stores) or 8 in the other
  const bool whole = (reinterpret_cast<uintptr_t>(d) & (t.dst_bf16 && !t.src_bf16 ? 7 : 15)) == 0;
#pragma unroll
  for (int k = 0; k < kVecs; ++k) {
    if (k >= s.vecs) break;
    const uint32_t w[4] = {q[k].x, q[k].y, q[k].z, q[k].w};
    float x[8];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (t.src_bf16) {
        x[2 * j] = lo16(w[j]) * coef;
        x[2 * j + 1] = hi16(w[j]) * coef;
      } else {
        x[j] = __uint_as_float(w[j]) * coef;
      }
    }
    uint8_t* o = d + k * step;
    if (!whole) {
      const int64_t at = s.first + (int64_t)k * kThreads * per;
      for (int j = 0; j < 8; ++j)
        if (j < per) store1(t.dst, at + j, t.dst_bf16, x[j]);
    } else if (t.dst_bf16) {
      __nv_bfloat162 h[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) h[j] = __floats2bfloat162_rn(x[2 * j], x[2 * j + 1]);
      if (t.src_bf16) __stcs(reinterpret_cast<uint4*>(o), *reinterpret_cast<const uint4*>(h));
      else __stcs(reinterpret_cast<uint2*>(o), *reinterpret_cast<const uint2*>(h));
    } else {
      __stcs(reinterpret_cast<float4*>(o), make_float4(x[0], x[1], x[2], x[3]));
      if (t.src_bf16) __stcs(reinterpret_cast<float4*>(o) + 1, make_float4(x[4], x[5], x[6], x[7]));
    }
  }
  if (s.odd >= 0) store1(t.dst, s.odd, t.dst_bf16, load1(t.src, s.odd, t.src_bf16) * coef);
}

// The coefficient of a sum of squares.
__device__ __forceinline__ float coefficient(const ClipHead& p, double sum, float* norm_out) {
  const double norm = sqrt(sum), den = norm + p.eps;
  double c = 1.0;                                   // an infinite limit, or nothing to scale
  if (isnan(norm)) c = norm;                        // whatever the limit
  else if (!isinf(p.max_norm) && den != 0.0) c = p.max_norm / den;
  if (c > 1.0) c = 1.0;                             // a NaN stays one
  *norm_out = (float)norm;
  return (float)c;
}

__device__ __forceinline__ double warp_add(double v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

template <int kN>
__global__ void __launch_bounds__(kThreads) clip_norm_kernel(const __grid_constant__ ClipBatch<kN> p) {
  __shared__ double warp_sum[kThreads / 32];
  double total = 0.0;
  for (int ch = blockIdx.x; ch < p.chunks; ch += gridDim.x) {
    const ClipTensor& t = p.t[find_tensor(p, ch)];
    total += chunk_sum(t, ch - t.chunk0, threadIdx.x);
  }
  ptx::launch_dependents();
  total = warp_add(total);
  if ((threadIdx.x & 31) == 0) warp_sum[threadIdx.x >> 5] = total;
  __syncthreads();
  if (threadIdx.x == 0) {
    double s = 0.0;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) s += warp_sum[w];
    p.partials[p.first_partial + blockIdx.x] = s;
  }
}

// The norm and the coefficient from all partial sums, added by the first warp.
__device__ __forceinline__ float finish_norm(const ClipHead& p, float* coef, bool write) {
  if (threadIdx.x < 32) {
    double v = 0.0;
#pragma unroll 8
    for (int i = threadIdx.x; i < p.n_partials; i += 32) v += p.partials[i];
    v = warp_add(v);
    if (threadIdx.x == 0) {
      float norm;
      *coef = coefficient(p, v, &norm);
      if (write) {
        p.out[0] = norm;
        p.out[1] = *coef;
      }
    }
  }
  __syncthreads();
  return *coef;
}

__global__ void __launch_bounds__(32) clip_finish_kernel(const __grid_constant__ ClipHead p) {
  __shared__ float shared_coef;
  ptx::wait_dependencies();
  finish_norm(p, &shared_coef, true);
}

template <int kN>
__global__ void __launch_bounds__(kThreads) clip_scale_kernel(const __grid_constant__ ClipBatch<kN> p) {
  __shared__ float shared_coef;
  int ch = p.chunks - 1 - (int)blockIdx.x;
  const ClipTensor* t = &p.t[find_tensor(p, ch)];
  Span sp = chunk_span(*t, ch - t->chunk0, threadIdx.x);
  uint4 q[kVecs];
  load_vecs(sp, q);                                  // the sources: no earlier kernel of this call writes them
  ptx::wait_dependencies();
  const float coef = finish_norm(p, &shared_coef, blockIdx.x == 0 && p.first_partial == 0);
  while (true) {
    if (coef != 1.0f || t->src != t->dst) chunk_scale(*t, sp, q, threadIdx.x, coef);   // else nothing changes
    ch -= gridDim.x;
    if (ch < 0) break;
    t = &p.t[find_tensor(p, ch)];
    if (coef == 1.0f && t->src == t->dst) continue;
    sp = chunk_span(*t, ch - t->chunk0, threadIdx.x);
    load_vecs(sp, q);
  }
}

// The launch's table as its kernel takes it: a launch copies its parameters,
// and 512 tensors are 20 KB.
void shorten(const ClipBatch<kClipTable>& b, ClipBatch<kClipShort>* s) {
  static_cast<ClipHead&>(*s) = b;
  std::memcpy(s->t, b.t, sizeof(ClipTensor) * b.n);
}

}  // namespace

cudaError_t launch_clip_norm(const ClipBatch<kClipTable>& b, int blocks, cudaStream_t s) {
  if (b.n > kClipShort) {
    clip_norm_kernel<<<blocks, kThreads, 0, s>>>(b);
  } else {
    ClipBatch<kClipShort> sb;
    shorten(b, &sb);
    clip_norm_kernel<<<blocks, kThreads, 0, s>>>(sb);
  }
  return cudaGetLastError();
}
cudaError_t launch_clip_finish(const ClipHead& b, cudaStream_t s) {
  return launch_overlapped(clip_finish_kernel, dim3(1), dim3(32), 0, s, true, b);
}
cudaError_t launch_clip_scale(const ClipBatch<kClipTable>& b, int blocks, bool overlap, cudaStream_t s) {
  if (b.n > kClipShort)
    return launch_overlapped(clip_scale_kernel<kClipTable>, dim3((unsigned)blocks), dim3(kThreads), 0, s, overlap, b);
  ClipBatch<kClipShort> sb;
  shorten(b, &sb);
  return launch_overlapped(clip_scale_kernel<kClipShort>, dim3((unsigned)blocks), dim3(kThreads), 0, s, overlap, sb);
}

}  // namespace ops
}  // namespace mfsdp
