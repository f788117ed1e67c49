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
// Both are bound by HBM.  A thread takes 8 columns with one 16- or 32-byte access
// a row (layouts whose rows do not start on such a boundary: 8 columns a block
// apart, so a warp's scalar accesses are still contiguous).
//
// Gradient.  Positions come sorted by token (stable).  Text repeats a few tokens
// thousands of times and leaves most of the vocabulary unnamed, so neither a
// row nor a position is a fair share of work; the merge of both is: the list
// in which every row's positions are followed by the row itself has vocab + n
// entries of about one row's traffic each, and every CTA takes an equal run of
// it (a slab), found by a search along its diagonal.  A row that lies in one slab is written there.
// A row cut by slab ends leaves one partial row a slab in the workspace, and a
// second kernel adds them in slab order.  The slabs depend on the sizes alone, so every
// sum has a fixed order: no atomics, bitwise reproducible, in fp32.
#include <cuda_bf16.h>

#include "ops_internal.h"
#include "ops_ptx.cuh"

namespace mfsdp {
namespace ops {
namespace {

constexpr int kCols = 8;                   // columns of a thread
constexpr int kMaxThreads = 256;

__device__ __forceinline__ void unpack8(const uint32_t (&w)[4], float (&x)[8]) {
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    x[2 * k] = __uint_as_float(w[k] << 16);
    x[2 * k + 1] = __uint_as_float(w[k] & 0xFFFF0000u);
  }
}

// The 8 columns of thread `tid` of `threads` in the column block starting at
// c0: [c0 + 8 tid, + 8) with vectors, c0 + tid + k threads without.
template <bool kBf16, bool kVec>
struct Row8 {
  uint32_t w[kBf16 && kVec ? 4 : 8];

  __device__ __forceinline__ void load(const void* base, int64_t at, int tid, int threads, int cols) {
    if constexpr (kVec) {
      if (kCols * tid >= cols) return;
      if constexpr (kBf16) {
        const uint4 q = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(base) + at + kCols * tid);
        w[0] = q.x; w[1] = q.y; w[2] = q.z; w[3] = q.w;
      } else {
        ptx::ld_v8(static_cast<const float*>(base) + at + kCols * tid, w);
      }
    } else {
#pragma unroll
      for (int k = 0; k < kCols; ++k) {
        const int c = tid + k * threads;
        if (c < cols)
          w[k] = kBf16 ? (uint32_t)static_cast<const uint16_t*>(base)[at + c] << 16
                       : static_cast<const uint32_t*>(base)[at + c];
      }
    }
  }
  __device__ __forceinline__ void get(float (&x)[8]) const {
    if constexpr (kBf16 && kVec) {
      unpack8(w, x);
    } else {
#pragma unroll
      for (int k = 0; k < kCols; ++k) x[k] = __uint_as_float(w[k]);
    }
  }
};

template <bool kBf16, bool kVec>
__device__ __forceinline__ void store8(void* base, int64_t at, int tid, int threads, int cols, const float (&x)[8]) {
  if constexpr (kVec) {
    if (kCols * tid >= cols) return;
    if constexpr (kBf16) {
      __nv_bfloat162 h[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) h[k] = __floats2bfloat162_rn(x[2 * k], x[2 * k + 1]);
      *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(base) + at + kCols * tid) =
          *reinterpret_cast<const uint4*>(h);
    } else {
      uint32_t w[8];
#pragma unroll
      for (int k = 0; k < kCols; ++k) w[k] = __float_as_uint(x[k]);
      ptx::st_v8(static_cast<float*>(base) + at + kCols * tid, w);
    }
  } else {
#pragma unroll
    for (int k = 0; k < kCols; ++k) {
      const int c = tid + k * threads;
      if (c < cols) {
        if constexpr (kBf16) static_cast<__nv_bfloat16*>(base)[at + c] = __float2bfloat16_rn(x[k]);
        else static_cast<float*>(base)[at + c] = x[k];
      }
    }
  }
}

// ---------------------------------------------------------------------- lookup
constexpr int kLookupRows = 4;             // rows of a thread, all loaded before the first store

template <bool kWBf16, bool kOutBf16, bool kVec>
__global__ void __launch_bounds__(kMaxThreads) lookup_kernel(const __grid_constant__ LookupArgs a) {
  const int64_t c0 = (int64_t)blockIdx.y * blockDim.x * kCols;
  const int cols = (int)min((int64_t)blockDim.x * kCols, a.dim - c0);
  const int64_t t0 = (int64_t)blockIdx.x * blockDim.y * kLookupRows + threadIdx.y;
  int64_t id[kLookupRows];
#pragma unroll
  for (int r = 0; r < kLookupRows; ++r) {
    const int64_t t = t0 + r * blockDim.y;
    id[r] = -1;
    if (t < a.n) id[r] = a.ids64 ? static_cast<const int64_t*>(a.ids)[t] : static_cast<const int32_t*>(a.ids)[t];
    if (id[r] >= a.vocab) id[r] = -1;
  }
  Row8<kWBf16, kVec> row[kLookupRows];
#pragma unroll
  for (int r = 0; r < kLookupRows; ++r)
    if (id[r] >= 0) row[r].load(a.w, id[r] * a.w_ld + c0, threadIdx.x, blockDim.x, cols);
#pragma unroll
  for (int r = 0; r < kLookupRows; ++r) {
    const int64_t t = t0 + r * blockDim.y;
    if (t >= a.n) break;
    float x[8];
    row[r].get(x);
#pragma unroll
    for (int k = 0; k < kCols; ++k) x[k] = id[r] >= 0 ? a.scale * x[k] : 0.f;
    store8<kOutBf16, kVec>(a.out, t * a.out_ld + c0, threadIdx.x, blockDim.x, cols, x);
  }
}

// -------------------------------------------------------------------- gradient
constexpr int kStage = 256;                // positions of a slab staged at a time
constexpr int kFixCols = 128;              // columns of a CTA that adds partial rows
constexpr int kFixParts = 8;               // its warps: each adds an eighth of the slabs

// Slabs of the merged list of vocab rows and n positions: enough CTAs to fill
// the GPU a few times over, at least 16 entries each.
struct SlabPlan {
  int64_t slab;        // entries of a slab
  int64_t slabs;
};
SlabPlan plan_slabs(int64_t n, int64_t vocab) {
  const int64_t units = n + vocab, want = (int64_t)kSlabTarget;
  SlabPlan s;
  s.slab = std::max<int64_t>(16, (units + want - 1) / want);
  s.slabs = (units + s.slab - 1) / s.slab;
  return s;
}

// A row cut by slab ends: the slabs its positions start and end in.
struct CutRow {
  int32_t row, first, last;
};

struct GradKernelArgs {
  EmbedGradArgs a;
  int64_t slab;
  int64_t part_ld;     // floats of a partial row
  int32_t* n_cut;      // how many `cut` holds (zeroed by the sort)
  CutRow* cut;         // in no fixed order: each is added by itself
  float* parts;        // two rows a slab: [0] the row cut at its start, [1] the row cut at its end
};

// Rows whose own entry is among the first d of the merged list: the number of
// v with positions(key <= v) + v + 1 <= d.  A warp narrows [lo, hi) 32 ways a
// step; the same for d1 at once.
__device__ __forceinline__ void merge_search(const int32_t* keys, int64_t n, int64_t vocab, int64_t d0, int64_t d1,
                                             int64_t& v0, int64_t& v1) {
  const int lane = threadIdx.x & 31;
  int64_t lo[2] = {max((int64_t)0, d0 - n), max((int64_t)0, d1 - n)};
  int64_t hi[2] = {min(d0, vocab), min(d1, vocab)};       // first v not among them is in [lo, hi]
  lo[0] = min(lo[0], hi[0]);
  lo[1] = min(lo[1], hi[1]);
  while (hi[0] > lo[0] || hi[1] > lo[1]) {
    bool in[2];
    int64_t step[2];
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const int64_t d = q ? d1 : d0;
      step[q] = (hi[q] - lo[q] + 31) / 32;
      const int64_t v = lo[q] + lane * step[q];
      const int64_t i = d - v - 1;
      in[q] = v < hi[q] && (i >= n || keys[i] > v);
    }
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      if (hi[q] <= lo[q]) {
        __ballot_sync(0xffffffffu, in[q]);
        continue;
      }
      const int cnt = __popc(__ballot_sync(0xffffffffu, in[q]));   // probes 0 .. cnt-1 hold
      if (cnt == 0) {
        hi[q] = lo[q];
      } else {
        hi[q] = min(hi[q], lo[q] + cnt * step[q]);
        lo[q] = lo[q] + (cnt - 1) * step[q] + 1;
        if (lo[q] > hi[q]) lo[q] = hi[q];
      }
    }
  }
  v0 = lo[0];
  v1 = lo[1];
}

template <bool kInBf16, bool kOutBf16, bool kVec>
__global__ void __launch_bounds__(kMaxThreads) embed_grad_kernel(const __grid_constant__ GradKernelArgs p) {
  __shared__ int32_t keys[kStage], order[kStage];
  __shared__ int64_t split[2];
  constexpr int kBatch = kInBf16 && kVec ? 8 : 4;      // positions in flight
  const EmbedGradArgs& a = p.a;
  const int tid = threadIdx.x, threads = blockDim.x;
  const int64_t c0 = (int64_t)blockIdx.y * threads * kCols;
  const int cols = (int)min((int64_t)threads * kCols, a.dim - c0);
  const int64_t s = blockIdx.x;
  const int64_t d0 = s * p.slab, d1 = min(d0 + p.slab, a.n + a.vocab);
  ptx::wait_dependencies();
  if (tid < 32) {
    int64_t v0, v1;
    merge_search(a.keys, a.n, a.vocab, d0, d1, v0, v1);
    if (tid == 0) {
      split[0] = v0;
      split[1] = v1;
    }
  }
  __syncthreads();
  ptx::launch_dependents();
  const int64_t v0 = split[0], v1 = split[1], i0 = d0 - v0, i1 = d1 - v1;
  const bool cut = v0 < a.vocab && i0 > 0 && a.keys[i0 - 1] == v0;      // row v0 starts in an earlier slab
  if (tid < 32 && blockIdx.y == 0 && cut && v1 > v0) {
    // a row cut at the start ends here: it begins in the slab of its first position
    int64_t lo = 0, hi = i0;
    while (lo < hi) {
      const int64_t step = (hi - lo + 31) / 32, i = lo + tid * step;
      const int cnt = __popc(__ballot_sync(0xffffffffu, i < hi && a.keys[i] < v0));
      if (cnt == 0) {
        hi = lo;
      } else {
        hi = min(hi, lo + cnt * step);
        lo = lo + (cnt - 1) * step + 1;
      }
    }
    if (tid == 0) p.cut[atomicAdd(p.n_cut, 1)] = {(int32_t)v0, (int32_t)((lo + v0) / p.slab), (int32_t)s};
  }

  float acc[kCols] = {};
  int64_t v = v0;
  bool named = false;                                  // row v has a position in this slab
  float* const part0 = p.parts + 2 * s * p.part_ld + c0;
  // Row v is complete in this slab.
  auto finish = [&]() {
    if (v == v0 && cut) {
      store8<false, kVec>(part0, 0, tid, threads, cols, acc);
    } else if (named || !a.accumulate) {
      const int64_t at = v * a.grad_ld + c0;
#pragma unroll
      for (int k = 0; k < kCols; ++k) acc[k] *= a.scale;
      if (a.accumulate) {
        Row8<kOutBf16, kVec> old;
        float x[8];
        old.load(a.grad, at, tid, threads, cols);
        old.get(x);
#pragma unroll
        for (int k = 0; k < kCols; ++k) acc[k] += x[k];
      }
      store8<kOutBf16, kVec>(a.grad, at, tid, threads, cols, acc);
    }
    ++v;
    named = false;
#pragma unroll
    for (int k = 0; k < kCols; ++k) acc[k] = 0.f;
  };

  for (int64_t base = i0; base < i1; base += kStage) {
    const int cnt = (int)min((int64_t)kStage, i1 - base);
    __syncthreads();
    for (int j = tid; j < cnt; j += threads) {
      keys[j] = a.keys[base + j];
      order[j] = a.order[base + j];
    }
    __syncthreads();
    for (int j0 = 0; j0 < cnt; j0 += kBatch) {
      Row8<kInBf16, kVec> row[kBatch];
#pragma unroll
      for (int b = 0; b < kBatch; ++b)
        if (j0 + b < cnt && keys[j0 + b] < a.vocab)
          row[b].load(a.dout, (int64_t)order[j0 + b] * a.dout_ld + c0, tid, threads, cols);
#pragma unroll
      for (int b = 0; b < kBatch; ++b) {
        if (j0 + b >= cnt) break;
        const int key = keys[j0 + b];
        if (key >= a.vocab) break;                     // masked: after every row
        while (v < key) finish();
        float x[8];
        row[b].get(x);
#pragma unroll
        for (int k = 0; k < kCols; ++k) acc[k] += x[k];
        named = true;
      }
    }
  }
  while (v < v1) finish();
  // Row v1 goes on in the next slab.
  if (v1 < a.vocab && (named || (v1 == v0 && cut)))
    store8<false, kVec>(v1 == v0 && cut ? part0 : part0 + p.part_ld, 0, tid, threads, cols, acc);
}

// Adds the partial rows of the rows cut by slab ends: slab `first` holds a
// row's start (second row of its pair), the following slabs up to `last` the rest.
// A CTA takes 128 columns of one row at a time, each warp an eighth of the
// slabs (a token that fills the batch has one partial row in every slab).
template <bool kOutBf16>
__global__ void __launch_bounds__(32 * kFixParts) embed_fix_kernel(const __grid_constant__ GradKernelArgs p) {
  __shared__ float4 sum[kFixParts][32];
  const EmbedGradArgs& a = p.a;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int blocks = (int)((a.dim + kFixCols - 1) / kFixCols);
  ptx::wait_dependencies();
  const int items = *p.n_cut * blocks;
  for (int it = blockIdx.x; it < items; it += gridDim.x) {
    const CutRow cut = p.cut[it / blocks];
    const int64_t c = (int64_t)(it % blocks) * kFixCols + 4 * lane;
    const int slabs = cut.last - cut.first + 1;
    const int lo = cut.first + (int)((int64_t)slabs * warp / kFixParts);
    const int hi = cut.first + (int)((int64_t)slabs * (warp + 1) / kFixParts);
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    if (c < p.part_ld) {
#pragma unroll 8
      for (int s = lo; s < hi; ++s) {
        const float4 x = *reinterpret_cast<const float4*>(p.parts + (2 * (int64_t)s + (s == cut.first)) * p.part_ld + c);
        acc.x += x.x; acc.y += x.y; acc.z += x.z; acc.w += x.w;
      }
    }
    __syncthreads();
    sum[warp][lane] = acc;
    __syncthreads();
    if (warp != 0) continue;
#pragma unroll
    for (int w = 1; w < kFixParts; ++w) {
      const float4 x = sum[w][lane];
      acc.x += x.x; acc.y += x.y; acc.z += x.z; acc.w += x.w;
    }
    const float v[4] = {acc.x, acc.y, acc.z, acc.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (c + k >= a.dim) break;
      const int64_t at = cut.row * a.grad_ld + c + k;
      float x = v[k] * a.scale;
      if constexpr (kOutBf16) {
        __nv_bfloat16* g = static_cast<__nv_bfloat16*>(a.grad) + at;
        if (a.accumulate) x += __bfloat162float(*g);
        *g = __float2bfloat16_rn(x);
      } else {
        float* g = static_cast<float*>(a.grad) + at;
        if (a.accumulate) x += *g;
        *g = x;
      }
    }
  }
}

// Threads that cover `dim` columns, 8 each, in whole warps.
int threads_for(int64_t dim) {
  return (int)std::min<int64_t>(kMaxThreads, (dim + 32 * kCols - 1) / (32 * kCols) * 32);
}
// Rows of a tensor start on the vector's boundary: 16 bytes of bf16, 32 of fp32.
bool vec_rows(const void* p, int64_t ld, int64_t dim, int32_t bf16) {
  return ld % kCols == 0 && dim % kCols == 0 && aligned(p, bf16 ? 16 : 32);
}

template <bool kA, bool kB, bool kVec>
void lookup_launch(const LookupArgs& a, dim3 grid, dim3 block, cudaStream_t s) {
  lookup_kernel<kA, kB, kVec><<<grid, block, 0, s>>>(a);
}
template <bool kA, bool kB, bool kVec>
cudaError_t grad_launch(const GradKernelArgs& p, dim3 grid, int threads, cudaStream_t s) {
  return launch_overlapped(embed_grad_kernel<kA, kB, kVec>, grid, dim3((unsigned)threads), s, p);
}

}  // namespace

cudaError_t launch_lookup(const LookupArgs& a, cudaStream_t s) {
  const bool vec = vec_rows(a.w, a.w_ld, a.dim, a.w_bf16) && vec_rows(a.out, a.out_ld, a.dim, a.out_bf16);
  const int tx = threads_for(a.dim), ty = kMaxThreads / tx;
  const dim3 block(tx, ty);
  const dim3 grid((unsigned)((a.n + ty * kLookupRows - 1) / (ty * kLookupRows)),
                  (unsigned)((a.dim + tx * kCols - 1) / (tx * kCols)));
  const auto go = vec ? (a.w_bf16 ? (a.out_bf16 ? lookup_launch<true, true, true> : lookup_launch<true, false, true>)
                                  : (a.out_bf16 ? lookup_launch<false, true, true> : lookup_launch<false, false, true>))
                      : (a.w_bf16 ? (a.out_bf16 ? lookup_launch<true, true, false> : lookup_launch<true, false, false>)
                                  : (a.out_bf16 ? lookup_launch<false, true, false> : lookup_launch<false, false, false>));
  go(a, grid, block, s);
  return cudaGetLastError();
}

size_t embed_grad_partial_bytes(int64_t n, int64_t vocab, int64_t dim) {
  const SlabPlan sp = plan_slabs(n, vocab);
  return 256 + round_up(sp.slabs * sizeof(CutRow), 256) + (size_t)sp.slabs * 2 * round_up((size_t)dim, 8) * sizeof(float);
}

cudaError_t launch_embed_grad(const EmbedGradArgs& a, cudaStream_t s) {
  const SlabPlan sp = plan_slabs(a.n, a.vocab);
  GradKernelArgs p;
  p.a = a;
  p.slab = sp.slab;
  p.part_ld = (int64_t)round_up((size_t)a.dim, 8);
  uint8_t* at = reinterpret_cast<uint8_t*>(a.partials);
  p.n_cut = a.partials_count();
  p.cut = reinterpret_cast<CutRow*>(at + 256);
  p.parts = reinterpret_cast<float*>(at + 256 + round_up(sp.slabs * sizeof(CutRow), 256));
  const bool vec = vec_rows(a.dout, a.dout_ld, a.dim, a.dout_bf16) && vec_rows(a.grad, a.grad_ld, a.dim, a.grad_bf16);
  const int threads = threads_for(a.dim);
  const dim3 grid((unsigned)sp.slabs, (unsigned)((a.dim + threads * kCols - 1) / (threads * kCols)));
  const auto go = vec ? (a.dout_bf16 ? (a.grad_bf16 ? grad_launch<true, true, true> : grad_launch<true, false, true>)
                                     : (a.grad_bf16 ? grad_launch<false, true, true> : grad_launch<false, false, true>))
                      : (a.dout_bf16 ? (a.grad_bf16 ? grad_launch<true, true, false> : grad_launch<true, false, false>)
                                     : (a.grad_bf16 ? grad_launch<false, true, false> : grad_launch<false, false, false>));
  const cudaError_t e = go(p, grid, threads, s);
  if (e != cudaSuccess || a.n == 0) return e;
  const int64_t items = sp.slabs * ((a.dim + kFixCols - 1) / kFixCols);      // at most
  const dim3 fix((unsigned)std::min<int64_t>(items, 4 * std::max(1, sm_count())));
  return launch_overlapped(a.grad_bf16 ? embed_fix_kernel<true> : embed_fix_kernel<false>, fix, dim3(32 * kFixParts), s, p);
}

}  // namespace ops
}  // namespace mfsdp
