// Matrix products grouped by expert: rows [starts[e], starts[e + 1]) of the
// activations meet expert e's matrix W_e (rows x cols).
//   forward:          Y[t, :]  = X[t, :] W_e^T
//   input gradient:   dX[t, :] = dY[t, :] W_e
//   weight gradient:  dW_e (+)= dY_e^T X_e         (zero for an expert without rows)
// bf16 operands, fp32 accumulation.
#include <cuda_bf16.h>

#include "ops_internal.h"

namespace mfsdp {
namespace ops {
namespace {

constexpr int kT = 32;       // output tile edge and K step

__device__ __forceinline__ float bf(const void* p, int64_t i) {
  return __uint_as_float((uint32_t)static_cast<const uint16_t*>(p)[i] << 16);
}
__device__ __forceinline__ int64_t clamp_row(int64_t s, int64_t n) { return s < 0 ? 0 : (s > n ? n : s); }

__device__ __forceinline__ void put(const ExpertArgs& p, int64_t at, float v) {
  if (p.out_bf16) {
    __nv_bfloat16* o = static_cast<__nv_bfloat16*>(p.out) + at;
    *o = __float2bfloat16_rn(p.accumulate ? v + __bfloat162float(*o) : v);
  } else {
    float* o = static_cast<float*>(p.out) + at;
    *o = p.accumulate ? v + *o : v;
  }
}

// One CTA: a 32 x 32 tile of expert blockIdx.z's product; a group with more
// row tiles than the grid has takes several turns.
__global__ void __launch_bounds__(kT * kT) expert_kernel(const __grid_constant__ ExpertArgs p) {
  __shared__ float sa[kT][kT + 1], sb[kT][kT + 1];
  const int tx = threadIdx.x % kT, ty = threadIdx.x / kT;
  const int64_t width = p.mode == kExpertForward ? p.rows : p.cols;       // columns of the output
  for (int e = blockIdx.z; e <= p.n_experts; e += gridDim.z) {
    if (e == p.n_experts && p.mode == kExpertWeightGrad) break;
    const int64_t lo = clamp_row(p.starts[e], p.n_rows);
    const int64_t hi = e == p.n_experts ? p.n_rows : clamp_row(p.starts[e + 1], p.n_rows);
    const int64_t height = p.mode == kExpertWeightGrad ? p.rows : hi - lo;
    const int64_t k_end = p.mode == kExpertForward ? p.cols : (p.mode == kExpertInputGrad ? p.rows : hi - lo);
    for (int64_t r0 = (int64_t)blockIdx.y * kT; r0 < height; r0 += (int64_t)gridDim.y * kT)
      for (int64_t c0 = (int64_t)blockIdx.x * kT; c0 < width; c0 += (int64_t)gridDim.x * kT) {
        const int64_t r = r0 + ty, c = c0 + tx;
        float acc = 0.f;
        if (e < p.n_experts)
          for (int64_t k0 = 0; k0 < k_end; k0 += kT) {
            // sa[i][k] = A(r0 + i, k0 + k), sb[k][j] = B(k0 + k, c0 + j)
            float va = 0.f, vb = 0.f;
            if (p.mode == kExpertWeightGrad) {
              if (r0 + tx < height && k0 + ty < k_end) va = bf(p.a, (lo + k0 + ty) * p.a_ld + r0 + tx);
              if (c < width && k0 + ty < k_end) vb = bf(p.b, (lo + k0 + ty) * p.b_ld + c);
              sa[tx][ty] = va;
              sb[ty][tx] = vb;
            } else {
              if (r < height && k0 + tx < k_end) va = bf(p.a, (lo + r) * p.a_ld + k0 + tx);
              sa[ty][tx] = va;
              if (p.mode == kExpertForward) {
                if (c0 + ty < width && k0 + tx < k_end) vb = bf(p.b, e * p.b_stride + (c0 + ty) * p.b_ld + k0 + tx);
                sb[tx][ty] = vb;
              } else {
                if (c < width && k0 + ty < k_end) vb = bf(p.b, e * p.b_stride + (k0 + ty) * p.b_ld + c);
                sb[ty][tx] = vb;
              }
            }
            __syncthreads();
#pragma unroll
            for (int k = 0; k < kT; ++k) acc = fmaf(sa[ty][k], sb[k][tx], acc);
            __syncthreads();
          }
        if (r < height && c < width) {
          if (p.mode == kExpertWeightGrad) put(p, e * p.out_stride + r * p.out_ld + c, acc);
          else put(p, (lo + r) * p.out_ld + c, acc);
        }
      }
  }
}

}  // namespace

cudaError_t launch_expert(const ExpertArgs& a, cudaStream_t s) {
  const int64_t width = a.mode == kExpertForward ? a.rows : a.cols;
  const int64_t height = a.mode == kExpertWeightGrad ? a.rows : a.n_rows;
  const unsigned z = (unsigned)(a.mode == kExpertWeightGrad ? a.n_experts : a.n_experts + 1);
  const unsigned x = (unsigned)std::min<int64_t>((width + kT - 1) / kT, 64);
  const unsigned y = (unsigned)std::max<int64_t>(1, std::min<int64_t>((height + kT - 1) / kT, 16));
  expert_kernel<<<dim3(x, y, z), kT * kT, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace ops
}  // namespace mfsdp
