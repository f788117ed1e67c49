// Every float from 0 up, infinity and the NaNs with them, through ptx::root, in either half of a pair, against CUDA's
// __fsqrt_rn.  Prints how many differ, and the first.
#include <cstdio>

#include "ops_ptx.cuh"

__device__ bool differ(float got, float v) {
  const float want = __fsqrt_rn(v);
  return want != want ? got == got : __float_as_uint(got) != __float_as_uint(want);
}

__global__ void sweep(unsigned long long* bad, unsigned int* least) {
  const uint32_t all = 1u << 31, step = gridDim.x * blockDim.x;
  for (uint32_t i = blockIdx.x * blockDim.x + threadIdx.x; i < all; i += step) {
    const uint32_t j = (i + 0x12345678u) & (all - 1);          // the other half: another exponent
    const float2 v = make_float2(__uint_as_float(i), __uint_as_float(j)), r = mfsdp::ptx::root(v);
    if (!differ(r.x, v.x) && !differ(r.y, v.y)) continue;
    atomicAdd(bad, 1ull);
    atomicMin(least, i);
  }
}

int main() {
  unsigned long long* bad = nullptr;
  unsigned int* least = nullptr;
  if (cudaMallocManaged(&bad, 8) != cudaSuccess || cudaMallocManaged(&least, 4) != cudaSuccess) return 2;
  *bad = 0;
  *least = 0xFFFFFFFFu;
  sweep<<<1024, 256>>>(bad, least);
  const cudaError_t e = cudaDeviceSynchronize();
  std::printf("%s: %llu differ, first %08x\n", cudaGetErrorString(e), *bad, *least);
  return e != cudaSuccess || *bad != 0;
}
