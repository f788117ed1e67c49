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
// Both are bound by how many loads are on their way, and the gradient of a batch by HBM's
// writes too.  A thread takes 8 columns with one 16- or 32-byte access a row.  Layouts whose
// rows do not start on such a boundary are read in the 16-byte words that hold their rows.
//
// Gradient, of more ids than a few, in three launches: the sort of positions by token
// (stable), the rows, and the rows that the division of work cut.
//   - Most of the vocabulary is unnamed in a batch, and its rows' zeros need no
//     order: the second kernel starts beside the sort (on 8 SMs, ~13 us),
//     finds the unnamed ones among its share of the rows from the ids
//     themselves, and writes them.
//   - Then every CTA adds up an equal run of the sorted positions (a slab): a token
//     may be named once or fill the batch, so rows are no fair share of work.  A row
//     whose positions lie in one slab is written there; a row cut by slab ends leaves
//     one partial row a slab in the workspace, and the third kernel adds them in slab
//     order.  The slabs depend on the sizes alone, so every sum has a fixed
//     order: no atomics on sums, bitwise reproducible, in fp32.
//   - Rows of dout arrive in shared memory as bulk copies, an instruction a row,
//     and a zero row leaves as one.  32768 ids, 32000 x 2048 fp32: 86 us in all, 396 MB.
//     The second kernel by itself, after the sort, takes 81 with DRAM at 55 % of its peak: its
//     17 warps an SM, all that the rings leave room for, wait for loads two thirds of the time.
//     With plain loads and stores after the sort, the rows alone took 72 us.
#include <cuda_bf16.h>

#include <atomic>
#include <type_traits>

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

template <bool kBf16>
__device__ __forceinline__ float load_one(const void* p, int64_t i) {
  return kBf16 ? __uint_as_float((uint32_t)static_cast<const uint16_t*>(p)[i] << 16) : static_cast<const float*>(p)[i];
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
          w[k] = kBf16 ? static_cast<const uint16_t*>(base)[at + c] : static_cast<const uint32_t*>(base)[at + c];
      }
    }
  }
  // From a row in shared memory whose first column is the block's.
  __device__ __forceinline__ void load_shared(const uint8_t* row, int tid, int threads, int cols) {
    if constexpr (kVec) {
      if (kCols * tid >= cols) return;
      const uint4* q = reinterpret_cast<const uint4*>(row) + (kBf16 ? tid : 2 * tid);
#pragma unroll
      for (int k = 0; k < (kBf16 ? 1 : 2); ++k) {
        const uint4 u = q[k];
        w[4 * k] = u.x; w[4 * k + 1] = u.y; w[4 * k + 2] = u.z; w[4 * k + 3] = u.w;
      }
    } else {
      load(row, 0, tid, threads, cols);
    }
  }
  __device__ __forceinline__ void get(float (&x)[8]) const {
    if constexpr (kBf16 && kVec) {
      unpack8(w, x);
    } else {
      // (shifted here: at the load it would wait)
#pragma unroll
      for (int k = 0; k < kCols; ++k) x[k] = __uint_as_float(kBf16 ? w[k] << 16 : w[k]);
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
      __stcs(reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(base) + at + kCols * tid),
             *reinterpret_cast<const uint4*>(h));
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
// 32768 rows of 2048, fp32 to bf16, with a text's frequencies: 36.5 us, 402 MB in and out of the
// SMs.  Bound by the loads' latency: the warps wait for a load in 57 % of their cycles, with DRAM at
// 53 %, L2 at 42 % and L1 at 51 % of their peaks; 60 registers allow 32 warps an SM, and 26
// are there.  (A call 39.6 us; 40.7 with stores that are not marked streaming.)  One row: 1.5 us.
constexpr int kLookupRows = 4;             // rows of a thread, all loaded before the first store

template <bool kWBf16, bool kOutBf16>
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
  Row8<kWBf16, true> row[kLookupRows];
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
    store8<kOutBf16, true>(a.out, t * a.out_ld + c0, threadIdx.x, blockDim.x, cols, x);
  }
}

// 8 columns from c on of a row of `dim` that may start anywhere: out of the 16-byte words that
// hold them, where those lie in the row, else one by one.
template <bool kBf16>
__device__ __forceinline__ void load8_any(const void* base, int64_t at, int64_t c, int64_t dim, float (&x)[8]) {
  constexpr int kPer = kBf16 ? 8 : 4, kWords = kBf16 ? 2 : 3;          // elements of a word; words that hold 8
  const uint8_t* const p = static_cast<const uint8_t*>(base) + (at + c) * (kBf16 ? 2 : 4);
  if (c >= kPer && c + kWords * kPer <= dim) {
    const uintptr_t a = reinterpret_cast<uintptr_t>(p);
    const uint4* const q = reinterpret_cast<const uint4*>(a & ~(uintptr_t)15);
    uint32_t w[4 * kWords];
#pragma unroll
    for (int k = 0; k < kWords; ++k) {
      const uint4 u = q[k];
      w[4 * k] = u.x; w[4 * k + 1] = u.y; w[4 * k + 2] = u.z; w[4 * k + 3] = u.w;
    }
    const bool by1 = a & 4, by2 = a & 8;
#pragma unroll
    for (int k = 0; k < 4 * kWords - 1; ++k) w[k] = by1 ? w[k + 1] : w[k];
#pragma unroll
    for (int k = 0; k < 4 * kWords - 3; ++k) w[k] = by2 ? w[k + 2] : w[k];
    if constexpr (kBf16) {
      const uint32_t shift = a & 2 ? 16 : 0;
      const uint32_t v[4] = {__funnelshift_r(w[0], w[1], shift), __funnelshift_r(w[1], w[2], shift),
                             __funnelshift_r(w[2], w[3], shift), __funnelshift_r(w[3], w[4], shift)};
      unpack8(v, x);
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k) x[k] = __uint_as_float(w[k]);
    }
    return;
  }
#pragma unroll
  for (int k = 0; k < 8; ++k) x[k] = load_one<kBf16>(base, at + c + k);
}

// Rows that do not start on vector boundaries: a thread takes the 8 columns of an output row
// that start on a 16-byte boundary of it, and the first threads its ends.  (35907 x 2709 of
// bf16: 88 us; columns one by one 166.)
constexpr int kAnyRows = 2;

template <bool kWBf16, bool kOutBf16>
__global__ void __launch_bounds__(kMaxThreads) lookup_any_kernel(const __grid_constant__ LookupArgs a) {
  const int64_t j = (int64_t)blockIdx.y * blockDim.x + threadIdx.x;
  const int64_t t0 = (int64_t)blockIdx.x * blockDim.y * kAnyRows + threadIdx.y;
  int64_t id[kAnyRows], c[kAnyRows];
  int head[kAnyRows];                                   // columns before the first boundary
  float x[kAnyRows][8];
#pragma unroll
  for (int r = 0; r < kAnyRows; ++r) {
    const int64_t t = t0 + r * blockDim.y;
    id[r] = -1;
    if (t < a.n) id[r] = a.ids64 ? static_cast<const int64_t*>(a.ids)[t] : static_cast<const int32_t*>(a.ids)[t];
    if (id[r] >= a.vocab) id[r] = -1;
    const uintptr_t o = reinterpret_cast<uintptr_t>(a.out) + t * a.out_ld * (kOutBf16 ? 2 : 4);
    head[r] = (int)min((int64_t)((16 - (o & 15)) & 15) / (kOutBf16 ? 2 : 4), a.dim);
    c[r] = head[r] + 8 * j;
#pragma unroll
    for (int k = 0; k < 8; ++k) x[r][k] = 0.f;
    if (id[r] >= 0 && c[r] + 8 <= a.dim) load8_any<kWBf16>(a.w, id[r] * a.w_ld, c[r], a.dim, x[r]);
  }
#pragma unroll
  for (int r = 0; r < kAnyRows; ++r) {
    const int64_t t = t0 + r * blockDim.y, row = t * a.out_ld;
    if (t >= a.n) break;
    if (c[r] + 8 <= a.dim) {
#pragma unroll
      for (int k = 0; k < 8; ++k) x[r][k] = id[r] >= 0 ? a.scale * x[r][k] : 0.f;
      if constexpr (kOutBf16) {
        store8<true, true>(a.out, row + c[r], 0, 1, kCols, x[r]);
      } else {
        float4* const o = reinterpret_cast<float4*>(static_cast<float*>(a.out) + row + c[r]);
        o[0] = make_float4(x[r][0], x[r][1], x[r][2], x[r][3]);
        o[1] = make_float4(x[r][4], x[r][5], x[r][6], x[r][7]);
      }
    }
    if (j >= 8) continue;
    const int64_t tail = head[r] + (a.dim - head[r]) / 8 * 8;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int64_t col = e == 0 ? j : tail + j;
      if (col >= (e == 0 ? head[r] : a.dim)) continue;
      const float v = id[r] >= 0 ? a.scale * load_one<kWBf16>(a.w, id[r] * a.w_ld + col) : 0.f;
      if constexpr (kOutBf16) static_cast<__nv_bfloat16*>(a.out)[row + col] = __float2bfloat16_rn(v);
      else static_cast<float*>(a.out)[row + col] = v;
    }
  }
}

// -------------------------------------------------------------------- gradient
constexpr int kMaxBatch = 32;              // a lane each
constexpr int kMaxStages = 8;
constexpr int kBatchBytes = 32768;         // a batch's rows, about
constexpr int kRingBytes = 98304;          // of the CTAs an SM holds: two, or more with less each
constexpr uint64_t kWaitNs = 2000000000ull;   // a stage is due within microseconds: longer is an error
constexpr int kFixCols = 128;              // columns of a CTA that adds partial rows
constexpr int kFixParts = 8;               // its warps: each adds an eighth of the slabs

// Threads that cover `dim` columns, 8 each, in whole warps.
int threads_for(int64_t dim) {
  return (int)std::min<int64_t>(kMaxThreads, (dim + 32 * kCols - 1) / (32 * kCols) * 32);
}

// CTAs an SM holds at once, by registers: their rings share 192 KB.
int ctas_per_sm(int64_t dim) { return std::max(2, std::min(3, 512 / threads_for(dim))); }

// Equal runs of the n sorted positions, one for each CTA that the GPU holds at
// once beside the sort, at least 4 each; and the CTAs, which share the vocabulary's
// rows too.  (CTAs that do not fit start when others end, with all their rows still to
// look for: 40 us instead of 27 for 22315 x 192, four an SM and in the sort's place too.)
struct SlabPlan {
  int64_t slab;        // positions of a slab
  int64_t slabs;
  int64_t ctas;
};
SlabPlan plan_slabs(int64_t n, int64_t vocab, int64_t dim) {
  const int64_t want = (kSms - kSortSms) * ctas_per_sm(dim);
  SlabPlan s;
  s.slab = std::max<int64_t>(4, (n + want - 1) / want);
  s.slabs = (n + s.slab - 1) / s.slab;
  s.ctas = std::max(s.slabs, std::min(want, (vocab + 15) / 16));
  return s;
}

// A row cut by slab ends: the slabs its positions start and end in.  It stands in
// the place of its last slab; the places of other slabs have no row.
struct CutRow {
  int32_t row, first, last;
};

struct GradKernelArgs {
  EmbedGradArgs a;
  int64_t slab;
  int64_t part_ld;     // floats of a partial row
  int64_t slabs;
  CutRow* cut;         // a place for each slab
  int32_t* status;     // first wait that gave up (0: none)
  int32_t threads;     // that add rows (the kernel may have more, which only look for unnamed rows)
  int32_t batch, stages, zero_bytes;   // rows of a batch, stages of the ring, bytes before it
  uint32_t row_slot, slot;   // bytes of a row of dout in the ring, and with the row of dW that accumulate adds to
  float* parts;        // two rows a slab: [0] of the row that began before it, [1] of the row that goes on after it
};

// First sorted position whose key is not below v; the whole warp narrows
// [0, n) 32 ways a step.
__device__ __forceinline__ int64_t warp_lower_bound(const int32_t* keys, int64_t n, int64_t v) {
  const int lane = threadIdx.x & 31;
  int64_t lo = 0, hi = n;
  while (lo < hi) {
    const int64_t step = (hi - lo + 31) / 32, i = lo + lane * step;
    const int below = __popc(__ballot_sync(0xffffffffu, i < hi && keys[i] < v));   // a prefix of the probes
    if (below == 0) {
      hi = lo;
    } else {
      hi = min(hi, lo + below * step);
      lo = lo + (below - 1) * step + 1;
    }
  }
  return lo;
}

// Calls zero(row) for the unnamed rows of this CTA's share of the vocabulary, each from
// one thread (or one whole warp), and waits for the sort: a short list of ids is read
// before the wait by every CTA; a long one would take longer than the sort, so then
// each CTA looks up its part of the sorted keys.  All threads call it.
constexpr int kWindow = 8192;              // rows marked at a time
constexpr int64_t kScanIds = 65536;

template <bool kWarpRow, typename Zero>
__device__ __forceinline__ void zero_unnamed(const EmbedGradArgs& a, Zero zero) {
  __shared__ uint32_t named[kWindow / 32];
  __shared__ int64_t range[2];
  const int64_t share = (a.vocab + gridDim.x - 1) / gridDim.x;
  const int64_t r0 = blockIdx.x * share, r1 = min(a.vocab, r0 + share);
  const bool early = a.n <= kScanIds && share <= kWindow;
  if (a.accumulate || !early) ptx::wait_dependencies();
  if (!a.accumulate) {
    for (int64_t w0 = r0; w0 < r1; w0 += kWindow) {
      const int len = (int)min((int64_t)kWindow, r1 - w0);
      __syncthreads();
      for (int i = threadIdx.x; i < (len + 31) / 32; i += blockDim.x) named[i] = 0;
      if (!early && threadIdx.x < 32) {
        const int64_t lo = warp_lower_bound(a.keys, a.n, w0), hi = warp_lower_bound(a.keys, a.n, w0 + len);
        if (threadIdx.x == 0) {
          range[0] = lo;
          range[1] = hi;
        }
      }
      __syncthreads();
      if (early) {
        constexpr int kAhead = 16;
        const int n = (int)a.n, step = blockDim.x;
        for (int i0 = threadIdx.x; i0 < n; i0 += kAhead * step) {
          int64_t id[kAhead];
#pragma unroll
          for (int k = 0; k < kAhead; ++k) {
            const int i = i0 + k * step;
            id[k] = -1;
            if (i < n) id[k] = a.ids64 ? static_cast<const int64_t*>(a.ids)[i] : static_cast<const int32_t*>(a.ids)[i];
          }
#pragma unroll
          for (int k = 0; k < kAhead; ++k) {
            const uint64_t r = (uint64_t)(id[k] - w0);
            if (r < (uint64_t)len) atomicOr(&named[r >> 5], 1u << (r & 31));
          }
        }
      } else {
        for (int64_t i = range[0] + threadIdx.x; i < range[1]; i += blockDim.x) {
          const int r = (int)(a.keys[i] - w0);
          atomicOr(&named[r >> 5], 1u << (r & 31));
        }
      }
      __syncthreads();
      for (int r = kWarpRow ? threadIdx.x >> 5 : threadIdx.x; r < len; r += kWarpRow ? blockDim.x >> 5 : blockDim.x)
        if (!(named[r >> 5] >> (r & 31) & 1)) zero(w0 + r);
    }
  }
  if (!a.accumulate && early) ptx::wait_dependencies();
}

// Where a slab's first and last rows reach beyond it.
struct Slab {
  int64_t i0, i1;      // its positions
  bool began;          // its first row has positions in earlier slabs
  bool goes_on;        // its last row has positions in later slabs
};
__device__ __forceinline__ Slab slab_of(const GradKernelArgs& p, int64_t s) {
  const EmbedGradArgs& a = p.a;
  Slab r;
  r.i0 = min(s * p.slab, a.n);
  r.i1 = min(r.i0 + p.slab, a.n);
  r.began = r.goes_on = false;
  if (r.i0 >= a.n) return r;
  // all four at once
  const int32_t k0 = a.keys[max(r.i0 - 1, (int64_t)0)], k1 = a.keys[r.i0], k2 = a.keys[r.i1 - 1],
                k3 = a.keys[min(r.i1, a.n - 1)];
  r.began = r.i0 > 0 && k0 == k1;
  r.goes_on = r.i1 < a.n && k2 == k3;
  return r;
}

// Notes, in the slab's place, the row that began in an earlier slab and ends in this one, or
// that there is none (whole warp).
__device__ __forceinline__ void note_cut(const GradKernelArgs& p, const Slab& sl, int64_t s) {
  const EmbedGradArgs& a = p.a;
  if (sl.i0 >= a.n) return;
  CutRow cut = {-1, 0, (int32_t)s};
  if (sl.began) {
    const int32_t v = a.keys[sl.i0];
    if (v < a.vocab && !(sl.goes_on && a.keys[sl.i1 - 1] == v))
      cut = {v, (int32_t)(warp_lower_bound(a.keys, sl.i0, v) / p.slab), (int32_t)s};
  }
  if ((threadIdx.x & 31) == 0) p.cut[s] = cut;
}

// A row's sum leaves the slab: into dW, with accumulate added to what it holds
// (`old`), or as a partial row.
template <bool kOutBf16, bool kVec>
__device__ __forceinline__ void put_row(const GradKernelArgs& p, const Slab& sl, int64_t s, int64_t c0, int64_t v,
                                        bool first, bool last, int tid, int threads, int cols, float (&acc)[kCols],
                                        const Row8<kOutBf16, kVec>& old) {
  const EmbedGradArgs& a = p.a;
  const bool began = first && sl.began;
  if (began || (last && sl.goes_on)) {
    store8<false, kVec>(p.parts + (2 * s + (began ? 0 : 1)) * p.part_ld + c0, 0, tid, threads, cols, acc);
    return;
  }
  if (a.accumulate) {
    float x[8];
    old.get(x);
#pragma unroll
    for (int k = 0; k < kCols; ++k) acc[k] += x[k];
  }
  store8<kOutBf16, kVec>(a.grad, v * a.grad_ld + c0, tid, threads, cols, acc);
}

// The rows.  Warp 0 copies the slab's rows of dout into the stages of a ring, a batch at a
// time (a lane each), and hands on their keys; the other warps add the rows up, 8
// columns a thread.  Layouts whose rows do not start on vector boundaries (not kVec): a row
// comes as the 16-byte words that hold it, except past the tensor's end, and is read from
// where it starts in them; with accumulate the adding threads fetch dW's row as theirs begins.
// (48890 x 1365 bf16 into 1703 rows: 76 us, added 94; element by element 738.)
template <bool kInBf16, bool kOutBf16, bool kVec>
__global__ void __launch_bounds__(32 + kMaxThreads, 3) embed_rows_kernel(const __grid_constant__ GradKernelArgs p) {
  extern __shared__ __align__(128) uint8_t smem[];     // a zero row, then the ring
  __shared__ __align__(8) uint64_t full[kMaxStages], empty[kMaxStages];
  __shared__ int32_t keys[kMaxStages][kMaxBatch];
  __shared__ uint8_t starts[kMaxStages][kMaxBatch];    // where a row starts in its first 16 bytes
  __shared__ int32_t count[kMaxStages];                // positions of the batch; the last one: ~positions
  const EmbedGradArgs& a = p.a;
  const int threads = p.threads, lane = threadIdx.x & 31;
  const int64_t c0 = (int64_t)blockIdx.y * threads * kCols;
  const int cols = (int)min((int64_t)threads * kCols, a.dim - c0);
  const uint32_t row_bytes = (uint32_t)cols * (kInBf16 ? 2 : 4), out_bytes = (uint32_t)cols * (kOutBf16 ? 2 : 4);
  const int64_t s = blockIdx.x;
  uint8_t* const ring = smem + p.zero_bytes;
  for (int i = threadIdx.x; i < p.zero_bytes / 16; i += blockDim.x)
    reinterpret_cast<uint4*>(smem)[i] = make_uint4(0, 0, 0, 0);
  if (threadIdx.x == 0) {
    for (int k = 0; k < p.stages; ++k) {
      ptx::mbar_init(ptx::smem_u32(&full[k]), 1);
      ptx::mbar_init(ptx::smem_u32(&empty[k]), (uint32_t)threads / 32);
    }
    ptx::fence_barrier_init();
  }
  ptx::fence_proxy_async_smem();
  __syncthreads();
  const uint64_t first_out = ptx::policy_evict_first();   // (90 us with it, 93 without)
  uint8_t* const out = static_cast<uint8_t*>(a.grad) + c0 * (kOutBf16 ? 2 : 4);
  const int64_t out_stride = a.grad_ld * (kOutBf16 ? 2 : 4);
  if constexpr (kVec) {
    const uint32_t zeros = ptx::smem_u32(smem);
    zero_unnamed<false>(a, [&](int64_t r) { ptx::bulk_store(out + r * out_stride, zeros, out_bytes, first_out); });
    ptx::bulk_commit();
  } else {
    zero_unnamed<true>(a, [&](int64_t r) {
      for (int c = lane; c < cols; c += 32) {
        if constexpr (kOutBf16) reinterpret_cast<uint16_t*>(out + r * out_stride)[c] = 0;
        else reinterpret_cast<float*>(out + r * out_stride)[c] = 0.f;
      }
    });
  }
  ptx::launch_dependents();
  const Slab sl = slab_of(p, s);

  if (threadIdx.x < 32) {
    const int64_t in_stride = a.dout_ld * (kInBf16 ? 2 : 4);
    const uint8_t* in = static_cast<const uint8_t*>(a.dout) + c0 * (kInBf16 ? 2 : 4);
    const uintptr_t in_end = reinterpret_cast<uintptr_t>(a.dout) + ((a.n - 1) * a.dout_ld + a.dim) * (kInBf16 ? 2 : 4);
    int stage = 0, use = 0;
    bool more = true;
    int64_t base = sl.i0;
    int key = 0, from = 0, before = -1;                // the key before the batch
    if (lane < p.batch && base + lane < sl.i1) {
      key = a.keys[base + lane];
      from = a.order[base + lane];
    }
    while (more) {
      const bool in_row = lane < p.batch && base + lane < sl.i1 && key < a.vocab;
      const int cnt = __popc(__ballot_sync(0xffffffffu, in_row));      // a prefix of the lanes: masked keys are last
      const int64_t next = base + p.batch;
      more = cnt == p.batch && next < sl.i1;
      const int this_key = key, this_from = from;
      if (more && lane < p.batch && next + lane < sl.i1) {             // in flight while this batch is queued
        key = a.keys[next + lane];
        from = a.order[next + lane];
      }
      if (!__all_sync(0xffffffffu, ptx::mbar_wait(ptx::smem_u32(&empty[stage]), (use & 1) ^ 1, kWaitNs))) {
        if (lane == 0) atomicCAS(p.status, 0, 1);
        break;
      }
      // with accumulate a row's first position brings what dW holds
      int left = __shfl_up_sync(0xffffffffu, this_key, 1);
      if (lane == 0) left = before;
      before = __shfl_sync(0xffffffffu, this_key, p.batch - 1);
      const bool brings = kVec && a.accumulate && in_row && this_key != left;
      const uint8_t* from_row = in + this_from * in_stride;
      uint8_t* const slot = ring + (size_t)(stage * p.batch + lane) * p.slot;
      uint32_t bytes = in_row ? row_bytes : 0;
      if (in_row) keys[stage][lane] = this_key;
      if (!kVec && in_row) {
        const uintptr_t at = reinterpret_cast<uintptr_t>(from_row), first = at & ~(uintptr_t)15, end = at + row_bytes;
        uintptr_t last = (end + 15) & ~(uintptr_t)15;
        if (last > in_end) {                                           // the rest one by one
          last = max(first, end & ~(uintptr_t)15);
          for (uintptr_t e = max(last, at); e < end; e += kInBf16 ? 2 : 4) {
            uint8_t* const to = slot + (e - first);
            if constexpr (kInBf16) *reinterpret_cast<uint16_t*>(to) = *reinterpret_cast<const uint16_t*>(e);
            else *reinterpret_cast<uint32_t*>(to) = *reinterpret_cast<const uint32_t*>(e);
          }
        }
        starts[stage][lane] = (uint8_t)(at - first);
        from_row = reinterpret_cast<const uint8_t*>(first);
        bytes = (uint32_t)(last - first);
      }
      const uint32_t all = __reduce_add_sync(0xffffffffu, bytes + (brings ? out_bytes : 0));
      __syncwarp();                                                    // the lanes' keys come before the arrival
      if (lane == 0) {
        count[stage] = more ? cnt : ~cnt;
        ptx::mbar_arrive_expect_tx(ptx::smem_u32(&full[stage]), all);
      }
      __syncwarp();
      if (bytes > 0) ptx::bulk_load(ptx::smem_u32(slot), from_row, bytes, ptx::smem_u32(&full[stage]));
      if (brings)
        ptx::bulk_load(ptx::smem_u32(slot) + p.row_slot, out + this_key * out_stride, out_bytes,
                       ptx::smem_u32(&full[stage]));
      if (++stage == p.stages) { stage = 0; ++use; }
      base = next;
    }
    if (blockIdx.y == 0) note_cut(p, sl, s);
  } else if ((int)threadIdx.x < 32 + threads) {
    const int tid = threadIdx.x - 32;
    float acc[kCols] = {};
    Row8<kOutBf16, kVec> old;                          // what row v of dW holds
    int v = -1;
    bool first = true;                                 // row v is the slab's first
    int stage = 0, use = 0;
    bool more = true, ok = true;
    while (more) {
      ok = __all_sync(0xffffffffu, ptx::mbar_wait(ptx::smem_u32(&full[stage]), use & 1, kWaitNs));
      if (!ok) {
        if (lane == 0) atomicCAS(p.status, 0, 2);
        break;
      }
      const int c = count[stage];
      more = c >= 0;
      const int cnt = more ? c : ~c;
      const uint8_t* rows = ring + (size_t)stage * p.batch * p.slot;
      constexpr int kAhead = kVec ? 4 : 1;
      for (int b0 = 0; b0 < cnt; b0 += kAhead) {
        Row8<kInBf16, kVec> row[kAhead];
#pragma unroll
        for (int b = 0; b < kAhead; ++b)
          if (b0 + b < cnt)
            row[b].load_shared(rows + (size_t)(b0 + b) * p.slot + (kVec ? 0 : starts[stage][b0 + b]), tid, threads,
                               cols);
#pragma unroll
        for (int b = 0; b < kAhead; ++b) {
          if (b0 + b >= cnt) break;
          const int key = keys[stage][b0 + b];
          if (key != v) {
            if (v >= 0) {
              put_row<kOutBf16, kVec>(p, sl, s, c0, v, first, false, tid, threads, cols, acc, old);
              first = false;
            }
            v = key;
            if (a.accumulate) {
              if constexpr (kVec) old.load_shared(rows + (size_t)(b0 + b) * p.slot + p.row_slot, tid, threads, cols);
              else old.load(a.grad, (int64_t)v * a.grad_ld + c0, tid, threads, cols);
            }
#pragma unroll
            for (int k = 0; k < kCols; ++k) acc[k] = 0.f;
          }
          float x[8];
          row[b].get(x);
#pragma unroll
          for (int k = 0; k < kCols; ++k) acc[k] = fmaf(a.scale, x[k], acc[k]);
        }
      }
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(ptx::smem_u32(&empty[stage]));
      if (++stage == p.stages) { stage = 0; ++use; }
    }
    // (a masked key that goes on is no row: v is the last row before it)
    if (ok && v >= 0)
      put_row<kOutBf16, kVec>(p, sl, s, c0, v, first, a.keys[sl.i1 - 1] == v, tid, threads, cols, acc, old);
  }
  ptx::bulk_wait_all();                                // the zero row is shared memory of this CTA
}

// Adds the partial rows of the rows cut by slab ends: slab `first` holds a
// row's start (second row of its pair), the following slabs up to `last` the
// rest.  An item is 128 columns of one row.  Most rows are cut once: a warp
// adds those by itself.  A frequent token's row goes through many slabs (one that
// fills the batch, through all): the warps of a CTA take an eighth of them each.
constexpr int kShortCut = 16;

__device__ __forceinline__ void add_parts(const GradKernelArgs& p, const CutRow& cut, int lo, int hi, int64_t c,
                                          float4& acc) {
#pragma unroll 8
  for (int s = lo; s < hi; ++s) {
    const float4 x = *reinterpret_cast<const float4*>(p.parts + (2 * (int64_t)s + (s == cut.first)) * p.part_ld + c);
    acc.x += x.x; acc.y += x.y; acc.z += x.z; acc.w += x.w;
  }
}

template <bool kOutBf16>
__device__ __forceinline__ void store_fix(const EmbedGradArgs& a, int64_t row, int64_t c, const float4& acc) {
  const float v[4] = {acc.x, acc.y, acc.z, acc.w};
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    if (c + k >= a.dim) break;
    const int64_t at = row * a.grad_ld + c + k;
    float x = v[k];
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

template <bool kOutBf16>
__global__ void __launch_bounds__(32 * kFixParts) embed_fix_kernel(const __grid_constant__ GradKernelArgs p) {
  __shared__ float4 sum[kFixParts][32];
  const EmbedGradArgs& a = p.a;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int blocks = (int)((a.dim + kFixCols - 1) / kFixCols);
  ptx::wait_dependencies();
  const int64_t items = p.slabs * blocks;
  // 32 items a look, one a lane: most places have no row
  const int64_t step = (int64_t)kFixParts * gridDim.x;
  for (int64_t at = (int64_t)warp * gridDim.x + blockIdx.x; at < items; at += 32 * step) {
    CutRow mine = {-1, 0, 0};
    if (at + lane * step < items) mine = p.cut[(at + lane * step) / blocks];
    unsigned found = __ballot_sync(0xffffffffu, mine.row >= 0 && mine.last - mine.first < kShortCut);
    for (; found; found &= found - 1) {
      const int k = __ffs(found) - 1;
      const CutRow cut = {__shfl_sync(0xffffffffu, mine.row, k), __shfl_sync(0xffffffffu, mine.first, k),
                          __shfl_sync(0xffffffffu, mine.last, k)};
      const int64_t c = (at + k * step) % blocks * kFixCols + 4 * lane;
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
      if (c < p.part_ld) add_parts(p, cut, cut.first, cut.last + 1, c, acc);
      store_fix<kOutBf16>(a, cut.row, c, acc);
    }
  }
  for (int64_t at = blockIdx.x; at < items; at += 32 * (int64_t)gridDim.x) {
    CutRow mine = {-1, 0, 0};
    if (at + lane * (int64_t)gridDim.x < items) mine = p.cut[(at + lane * (int64_t)gridDim.x) / blocks];
    unsigned found = __ballot_sync(0xffffffffu, mine.row >= 0 && mine.last - mine.first >= kShortCut);
    for (; found; found &= found - 1) {                // the same in every warp
      const int k = __ffs(found) - 1;
      const CutRow cut = {__shfl_sync(0xffffffffu, mine.row, k), __shfl_sync(0xffffffffu, mine.first, k),
                          __shfl_sync(0xffffffffu, mine.last, k)};
      const int64_t c = (at + k * (int64_t)gridDim.x) % blocks * kFixCols + 4 * lane;
      const int64_t slabs = cut.last - cut.first + 1;
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
      if (c < p.part_ld)
        add_parts(p, cut, cut.first + (int)(slabs * warp / kFixParts),
                  cut.first + (int)(slabs * (warp + 1) / kFixParts), c, acc);
      __syncthreads();
      sum[warp][lane] = acc;
      __syncthreads();
      if (warp != 0) continue;
#pragma unroll
      for (int w = 1; w < kFixParts; ++w) {
        const float4 x = sum[w][lane];
        acc.x += x.x; acc.y += x.y; acc.z += x.z; acc.w += x.w;
      }
      store_fix<kOutBf16>(a, cut.row, c, acc);
    }
  }
}

// Few ids: one launch, no sort.  A CTA takes a share of the vocabulary's rows and 256
// of the columns, reads all ids, lists those of its share in order, and writes its
// rows: the sum of a row's positions in ascending order, one row a warp, or zeros.  A row
// with many positions is added by the eight warps, an eighth of them each, and goes
// first.  Bound by latency (ids, positions, rows, stores: 3 us for 64 ids of 256 columns)
// or by writing zeros.
constexpr int kSmallIds = 1024;            // at most (see embed_grad_sorts)
constexpr int kSmallShare = 2048;          // rows of a share, at most: its bitmap
constexpr int kSmallWarps = 8;
constexpr int kSmallCols = 32 * kCols;
constexpr int kSmallRow = 32;              // positions of a row that one warp adds

template <bool kInBf16, bool kOutBf16, bool kVec>
__global__ void __launch_bounds__(32 * kSmallWarps, kVec ? 4 : 3)
    embed_small_kernel(const __grid_constant__ EmbedGradArgs a) {
  __shared__ int16_t pos[kSmallIds], row[kSmallIds];      // listed positions, and their rows in the share
  __shared__ uint32_t named[kSmallShare / 32];
  __shared__ int warp_count[kSmallWarps];
  __shared__ float sums[kSmallWarps][kSmallCols];
  __shared__ int16_t own[kSmallWarps][kSmallIds / kSmallWarps];    // positions that a warp adds
  constexpr int kAhead = 4;         // rows in flight
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t c0 = (int64_t)blockIdx.y * kSmallCols;
  const int cols = (int)min((int64_t)kSmallCols, a.dim - c0);
  const int64_t share = (a.vocab + gridDim.x - 1) / gridDim.x;
  const int64_t r0 = blockIdx.x * share;
  const int len = (int)max((int64_t)0, min(share, a.vocab - r0));
  if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) *a.header = 0;
  for (int i = threadIdx.x; i < (len + 31) / 32; i += blockDim.x) named[i] = 0;
  __syncthreads();
  int count = 0;
  for (int base = 0; base < (int)a.n; base += 32 * kSmallWarps) {
    const int t = base + threadIdx.x;
    uint64_t id = ~0ull;                                  // outside every share
    if (t < a.n)
      id = (uint64_t)(a.ids64 ? static_cast<const int64_t*>(a.ids)[t] : static_cast<const int32_t*>(a.ids)[t]) - r0;
    const bool in = id < (uint64_t)len;
    const unsigned mask = __ballot_sync(0xffffffffu, in);
    if (lane == 0) warp_count[warp] = __popc(mask);
    __syncthreads();
    int at = count;
#pragma unroll
    for (int w = 0; w < kSmallWarps; ++w) {
      if (w < warp) at += warp_count[w];
      count += warp_count[w];
    }
    if (in) {
      at += __popc(mask & ((1u << lane) - 1));
      pos[at] = (int16_t)t;
      row[at] = (int16_t)id;
      atomicOr(&named[id >> 5], 1u << (id & 31));
    }
    __syncthreads();
  }

  // adds the positions of row r from the first-th to the last-th
  float acc[kCols];
  auto add_positions = [&](int r, int first, int last) {
    int seen = 0;
    for (int base = 0; base < count && seen < last; base += 32) {
      const bool in = base + lane < count && row[base + lane] == r;
      const unsigned mask = __ballot_sync(0xffffffffu, in);
      const int nth = seen + __popc(mask & ((1u << lane) - 1));
      if (in && nth >= first && nth < last) own[warp][nth - first] = pos[base + lane];
      seen += __popc(mask);
    }
    __syncwarp();
    const int n = min(seen, last) - first;
#pragma unroll
    for (int k = 0; k < kCols; ++k) acc[k] = 0.f;
    for (int i = 0; i < n; i += kAhead) {
      Row8<kInBf16, kVec> x[kAhead];
#pragma unroll
      for (int b = 0; b < kAhead; ++b)
        if (i + b < n) x[b].load(a.dout, (int64_t)own[warp][i + b] * a.dout_ld + c0, lane, 32, cols);
#pragma unroll
      for (int b = 0; b < kAhead; ++b) {
        if (i + b >= n) break;
        float v[8];
        x[b].get(v);
#pragma unroll
        for (int k = 0; k < kCols; ++k) acc[k] = fmaf(a.scale, v[k], acc[k]);
      }
    }
    __syncwarp();
  };
  auto put = [&](int r) {
    const int64_t at = (r0 + r) * a.grad_ld + c0;
    if (a.accumulate) {
      Row8<kOutBf16, kVec> old;
      float v[8];
      old.load(a.grad, at, lane, 32, cols);
      old.get(v);
#pragma unroll
      for (int k = 0; k < kCols; ++k) acc[k] += v[k];
    }
    store8<kOutBf16, kVec>(a.grad, at, lane, 32, cols, acc);
  };
  auto positions_of = [&](int r) {
    int m = 0;
    for (int base = 0; base < count; base += 32)
      m += __popc(__ballot_sync(0xffffffffu, base + lane < count && row[base + lane] == r));
    return m;
  };

  // Rows of many positions, one at a time, first: theirs is the longest way.
  const int words = (len + 31) / 32;
  if (count > kSmallRow)
    for (int w = 0; w < words; ++w)
      for (uint32_t bits = named[w]; bits; bits &= bits - 1) {
        const int r = 32 * w + __ffs(bits) - 1, m = positions_of(r);
        if (m <= kSmallRow) continue;
        add_positions(r, m * warp / kSmallWarps, m * (warp + 1) / kSmallWarps);
        __syncthreads();
#pragma unroll
        for (int k = 0; k < kCols; ++k) sums[warp][32 * k + lane] = acc[k];
        __syncthreads();
        if (warp != 0) continue;
#pragma unroll
        for (int q = 1; q < kSmallWarps; ++q)
#pragma unroll
          for (int k = 0; k < kCols; ++k) acc[k] += sums[q][32 * k + lane];
        put(r);
      }
  // rows of a few, a warp each
  int turn = warp;
  for (int w = 0; w < words; ++w)
    for (uint32_t bits = named[w]; bits; bits &= bits - 1) {
      if (turn-- > 0) continue;
      turn = kSmallWarps - 1;
      const int r = 32 * w + __ffs(bits) - 1;
      if (count > kSmallRow && positions_of(r) > kSmallRow) continue;
      add_positions(r, 0, kSmallRow);
      put(r);
    }
  // rows of none
  if (a.accumulate) return;
#pragma unroll
  for (int k = 0; k < kCols; ++k) acc[k] = 0.f;
  for (int r = warp; r < len; r += kSmallWarps)
    if (!(named[r >> 5] >> (r & 31) & 1))
      store8<kOutBf16, kVec>(a.grad, (r0 + r) * a.grad_ld + c0, lane, 32, cols, acc);
}

// Rows of a tensor start on the vector's boundary: 16 bytes of bf16, 32 of fp32.
bool vec_rows(const void* p, int64_t ld, int64_t dim, int32_t bf16) {
  return ld % kCols == 0 && dim % kCols == 0 && aligned(p, bf16 ? 16 : 32);
}

template <bool kA, bool kB>
void lookup_launch(const LookupArgs& a, bool vec, cudaStream_t s) {
  const int64_t threads = vec ? threads_for(a.dim) : threads_for(a.dim + 8), rows = kMaxThreads / threads;
  const int64_t per = rows * (vec ? kLookupRows : kAnyRows);
  const dim3 block((unsigned)threads, (unsigned)rows);
  const dim3 grid((unsigned)((a.n + per - 1) / per), (unsigned)((a.dim + threads * kCols - 1) / (threads * kCols)));
  if (vec) lookup_kernel<kA, kB><<<grid, block, 0, s>>>(a);
  else lookup_any_kernel<kA, kB><<<grid, block, 0, s>>>(a);
}
// Shares of the vocabulary for few ids: four CTAs an SM, more where a share would
// not fit its bitmap.
int64_t small_shares(int64_t vocab, int64_t dim) {
  const int64_t blocks = (dim + kSmallCols - 1) / kSmallCols;
  const int64_t want = std::min((vocab + 7) / 8, std::max<int64_t>(1, 4 * kSms / blocks));
  return std::max((vocab + kSmallShare - 1) / kSmallShare, want);
}

template <bool kIn, bool kOut>
cudaError_t small_launch(const EmbedGradArgs& all, bool vec, cudaStream_t s) {
  constexpr int64_t kMost = (int64_t)65535 * kSmallCols;      // columns of a launch
  for (int64_t c = 0; c < all.dim; c += kMost) {
    EmbedGradArgs a = all;
    a.dim = std::min(kMost, all.dim - c);
    a.dout = static_cast<const uint8_t*>(all.dout) + c * (kIn ? 2 : 4);
    a.grad = static_cast<uint8_t*>(all.grad) + c * (kOut ? 2 : 4);
    const dim3 grid((unsigned)small_shares(a.vocab, a.dim), (unsigned)((a.dim + kSmallCols - 1) / kSmallCols));
    if (vec) embed_small_kernel<kIn, kOut, true><<<grid, 32 * kSmallWarps, 0, s>>>(a);
    else embed_small_kernel<kIn, kOut, false><<<grid, 32 * kSmallWarps, 0, s>>>(a);
  }
  return cudaGetLastError();
}

template <bool kIn, bool kOut, bool kVec>
cudaError_t grad_launch(GradKernelArgs& p, int64_t ctas, cudaStream_t s) {
  const EmbedGradArgs& a = p.a;
  const int threads = threads_for(a.dim);
  const dim3 grid((unsigned)ctas, (unsigned)((a.dim + threads * kCols - 1) / (threads * kCols)));
  // The kernel writes dW before its wait, beside the sort, which is the kernel before it.
  p.threads = threads;
  const int cols = (int)std::min<int64_t>(a.dim, (int64_t)threads * kCols);
  p.row_slot = (uint32_t)round_up((size_t)cols * (kIn ? 2 : 4) + (kVec ? 0 : 30), 128);
  p.zero_bytes = kVec ? (int32_t)round_up((size_t)cols * (kOut ? 2 : 4), 128) : 0;
  p.slot = p.row_slot + (a.accumulate ? (uint32_t)p.zero_bytes : 0);
  const int ring = 2 * kRingBytes / ctas_per_sm(a.dim);
  p.batch = (int32_t)std::max<int64_t>(2, std::min<int64_t>({kMaxBatch, kBatchBytes / p.slot, ring / (2 * p.slot)}));
  p.stages = (int32_t)std::max<int64_t>(2, std::min<int64_t>(kMaxStages, ring / (p.batch * p.slot)));
  const size_t smem = p.zero_bytes + (size_t)p.stages * p.batch * p.slot;
  static std::atomic<bool> ready[kMaxDevices];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
  if (!ready[dev].load()) {
    e = cudaFuncSetAttribute(embed_rows_kernel<kIn, kOut, kVec>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             kRingBytes + 16384);
    if (e != cudaSuccess) return e;
    ready[dev].store(true);
  }
  const dim3 block((unsigned)std::max(256, 32 + threads));
  return launch_overlapped(embed_rows_kernel<kIn, kOut, kVec>, grid, block, smem, s,
                           true, p);
}

}  // namespace

cudaError_t launch_lookup(const LookupArgs& a, cudaStream_t s) {
  const bool vec = vec_rows(a.w, a.w_ld, a.dim, a.w_bf16) && vec_rows(a.out, a.out_ld, a.dim, a.out_bf16);
  a.w_bf16 ? (a.out_bf16 ? lookup_launch<true, true>(a, vec, s) : lookup_launch<true, false>(a, vec, s))
           : (a.out_bf16 ? lookup_launch<false, true>(a, vec, s) : lookup_launch<false, false>(a, vec, s));
  return cudaGetLastError();
}

size_t embed_grad_partial_bytes(int64_t n, int64_t vocab, int64_t dim) {
  const SlabPlan sp = plan_slabs(n, vocab, dim);
  return round_up(sp.slabs * sizeof(CutRow), 256) + (size_t)sp.slabs * 2 * round_up((size_t)dim, 8) * sizeof(float);
}

bool embed_grad_vec(const EmbedGradArgs& a) {
  return vec_rows(a.dout, a.dout_ld, a.dim, a.dout_bf16) && vec_rows(a.grad, a.grad_ld, a.dim, a.grad_bf16);
}

// Few ids go in one launch; more, or many rows of zeros beside more than half of as many (a
// quarter, off the vectors' boundaries), through the sort and two more.  The one launch's zeros wait
// for the ids' list and its named rows, the sort hides behind the zeros.  From cold caches, GPU time
// in us, one launch / sorted, fp32 rows, a text's ids (and half of the ids one token):
//   512 ids,  2048 columns into  1000 rows    15.5 / 21.6  (23.6 / 19.6)
//             2048              32000         50.3 / 54.4  (59.6 / 54.4)
//   600,      2048              32000         51.3 / 55.4  (64.6 / 55.4)
//   1024,      256               1000         17.5 / 21.6  (33.9 / 21.6)
//              256              32000 (33 MB) 19.6 / 21.6  (31.9 / 21.6)
//             2048               5000 (41 MB) 25.7 / 23.7  (40.1 / 23.7)
//             2048              32000         56.4 / 56.4  (77.0 / 58.5)
//             2048              32000, added  23.7 / 23.7  (40.1 / 23.7)
//   off the vectors' boundaries
//   1024,      375               1000         17.5 / 22.7  (28.8 / 24.7)
//             1365               5000 (27 MB) 21.7 / 24.7  (34.0 / 25.7)
//              375              32000 (48 MB) 23.7 / 23.6  (34.0 / 25.7)
//             1365               5000, added  21.7 / 27.7  (31.9 / 27.8)
//   512,       375              32000         21.7 / 23.7  (24.7 / 23.6)
//             1365              32000, bf16 (87 MB) 33.9 / 31.9 (37.0 / 29.8)
//             1365              32000         46.2 / 43.2  (50.3 / 42.1)
//   256 (warm), 1365            32000         37.8 / 36.4  (all one token 41.9 / 36.2)
bool embed_grad_sorts(const EmbedGradArgs& a) {
  if (a.n > kSmallIds || a.accumulate) return a.n > kSmallIds;
  const int64_t zeros = a.vocab * a.dim * (a.grad_bf16 ? 2 : 4);                  // bytes, at most
  if (a.n > kSmallIds / 2) return zeros > 1 << 25;
  return a.n > kSmallIds / 4 && zeros > 1 << 26 && !embed_grad_vec(a);
}

cudaError_t launch_embed_grad(const EmbedGradArgs& a, cudaStream_t s) {
  const bool vec = embed_grad_vec(a);
  if (!embed_grad_sorts(a))
    return a.dout_bf16 ? (a.grad_bf16 ? small_launch<true, true>(a, vec, s) : small_launch<true, false>(a, vec, s))
                       : (a.grad_bf16 ? small_launch<false, true>(a, vec, s) : small_launch<false, false>(a, vec, s));
  const SlabPlan sp = plan_slabs(a.n, a.vocab, a.dim);
  GradKernelArgs p;
  p.a = a;
  p.slab = sp.slab;
  p.part_ld = (int64_t)round_up((size_t)a.dim, 8);
  uint8_t* at = reinterpret_cast<uint8_t*>(a.partials);
  p.status = a.header;
  p.slabs = sp.slabs;
  p.cut = reinterpret_cast<CutRow*>(at);
  p.parts = reinterpret_cast<float*>(at + round_up(sp.slabs * sizeof(CutRow), 256));
  const auto go = [&](auto in, auto out) {
    return vec ? grad_launch<decltype(in)::value, decltype(out)::value, true>(p, sp.ctas, s)
               : grad_launch<decltype(in)::value, decltype(out)::value, false>(p, sp.ctas, s);
  };
  const std::true_type yes;
  const std::false_type no;
  const cudaError_t e = a.dout_bf16 ? (a.grad_bf16 ? go(yes, yes) : go(yes, no))
                                    : (a.grad_bf16 ? go(no, yes) : go(no, no));
  if (e != cudaSuccess) return e;
  const int64_t items = sp.slabs * ((a.dim + kFixCols - 1) / kFixCols);      // at most
  const dim3 fix((unsigned)std::min<int64_t>(items, 4 * std::max(1, sm_count())));
  return launch_overlapped(a.grad_bf16 ? embed_fix_kernel<true> : embed_fix_kernel<false>, fix, dim3(32 * kFixParts),
                           0, s, true, p);
}

}  // namespace ops
}  // namespace mfsdp
