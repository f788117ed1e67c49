// AdamW over a set of tensors, with states in 32 bits or in 8.
//
//   g' = coef g,  m <- b1 m + (1-b1) g',  v <- b2 v + (1-b2) g'^2
//   p <- p (1 - lr wd) - lr/(1-b1^t) m / (sqrt(v)/sqrt(1-b2^t) + eps)
//
// Matrices go to Muon; what is left for AdamW is an embedding, a head and many
// short vectors, each with its own decay and rate.  One launch takes up to 384 of them, cut
// into chunks of 2048 elements; a chunk is found by bisection in the launch's table.
//
// State in 8 bits: 256 elements share a scale.  e4m3 has 3 bits of mantissa over 2^18 of range;
// the second moment is kept as its root, which has half the powers of two and is
// what the step divides by.  A warp has one block, so its largest magnitude is one
// warp reduction over the bits of the magnitudes (ordered as whole numbers, NaN the largest).
// The scale is fp32 and not a power of two: with a decay as slow as 0.999 a
// rounded state would otherwise stand still; so the block's largest element, and with it
// the scale, always follows the formula.
//
// With 8-bit states the instructions count as much as the bytes, so sums and products run on pairs of elements, and the
// quotient is the hardware's reciprocal's (2^-22).  A code has to be what the formula in fp32 gives, whoever
// computes it, since the next step's quotient may hang on it: the moments take no fused operations, and their root is
// the IEEE one (ptx::root).
//
// Bound by HBM: 28 bytes an element (fp32), 16 with a bf16 gradient, an 8-bit state and a bf16
// copy.  Measured: 131 M elements, fp32 states: 513 us at 7.2 TB/s; 8-bit states, 2.1 GB: 325 us at 6.5 TB/s.
// A lane takes elements 4l .. 4l+3 of each half of a block: every warp access is
// contiguous, and needs 4 elements' alignment.  All loads of a chunk go out before the first is
// used.  Tensors off that alignment go element by element, still contiguous over a warp.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstring>

#include "ops_internal.h"
#include "ops_ptx.cuh"

namespace mfsdp {
namespace ops {
namespace {

using ptx::both;
using ptx::fma2;
using ptx::mul2;

constexpr int kThreads = 256;
constexpr int kPerLane = 8;
static_assert(kThreads * kPerLane == kAdamwChunk && 32 * kPerLane == MFSDP_STATE_BLOCK, "a warp has one block");
constexpr float kTop8 = 448.0f;                    // the largest e4m3 value
constexpr float kDeadBlock = 0x1p-100f;            // a block below is stored as zeros: 448 / it stays finite

// The tensor of a chunk, which is none before `from`: a CTA's chunks ascend, and most lie where the last one lay.
template <int kN>
__device__ __forceinline__ int find_tensor(const AdamwBatch<kN>& b, int chunk, int from) {
  if (from + 1 >= b.n || b.t[from + 1].chunk0 > chunk) return from;
  int lo = from + 1, hi = b.n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (b.t[mid].chunk0 <= chunk) lo = mid; else hi = mid - 1;
  }
  return lo;
}

// Four e4m3 codes to fp32, and back with rounding to nearest even (past 448: 448).
__device__ __forceinline__ void decode4(uint32_t c, float2 (&x)[2]) {
  uint32_t lo, hi;
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(c));
  x[0] = __half22float2(*reinterpret_cast<const __half2*>(&lo));
  x[1] = __half22float2(*reinterpret_cast<const __half2*>(&hi));
}
__device__ __forceinline__ uint32_t encode4(const float2 (&x)[2]) {
  uint32_t c;
  asm("{\n\t.reg .b16 a, b;\n\tcvt.rn.satfinite.e4m3x2.f32 a, %2, %1;\n\tcvt.rn.satfinite.e4m3x2.f32 b, %4, %3;\n\t"
      "mov.b32 %0, {a, b};\n\t}"
      : "=r"(c)
      : "f"(x[0].x), "f"(x[0].y), "f"(x[1].x), "f"(x[1].y));
  return c;
}

__device__ __forceinline__ float bf16_bits(uint32_t u) { return __uint_as_float(u << 16); }

// A lane has two runs of 4 elements of its warp's block: 4l + j and 128 + 4l + j where the tensor lies on 4
// elements' boundaries (kVec), else every 32nd element from l on.
template <bool kVec>
__device__ __forceinline__ int place(int lane, int h, int j) {
  return kVec ? h * 128 + lane * 4 + j : lane + 32 * (4 * h + j);
}

// Four elements as they come from memory.
template <bool kBf16>
struct Raw {
  uint32_t w[kBf16 ? 2 : 4];
  __device__ __forceinline__ void get(float2 (&x)[2]) const {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      if constexpr (kBf16) x[j] = make_float2(bf16_bits(w[j]), __uint_as_float(w[j] & 0xFFFF0000u));
      else x[j] = make_float2(__uint_as_float(w[2 * j]), __uint_as_float(w[2 * j + 1]));
    }
  }
};

// Run h of the block that starts at element `at`, `left` of whose elements exist (zeros past them).
template <bool kBf16, bool kVec>
__device__ __forceinline__ Raw<kBf16> load4(const void* src, int64_t at, int left, int lane, int h) {
  Raw<kBf16> r;
  if (kVec && place<kVec>(lane, h, 3) < left) {
    if constexpr (kBf16) {
      const uint2 q = __ldcs(reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(src) + at + place<kVec>(lane, h, 0)));
      r.w[0] = q.x;
      r.w[1] = q.y;
    } else {
      const uint4 q = __ldcs(reinterpret_cast<const uint4*>(static_cast<const float*>(src) + at + place<kVec>(lane, h, 0)));
      r.w[0] = q.x;
      r.w[1] = q.y;
      r.w[2] = q.z;
      r.w[3] = q.w;
    }
    return r;
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int e = place<kVec>(lane, h, j);
    if constexpr (kBf16) {
      const uint32_t x = e < left ? static_cast<const uint16_t*>(src)[at + e] : 0;
      r.w[j >> 1] = j & 1 ? r.w[j >> 1] | x << 16 : x;
    } else {
      r.w[j] = e < left ? static_cast<const uint32_t*>(src)[at + e] : 0;
    }
  }
  return r;
}

template <bool kBf16, bool kVec>
__device__ __forceinline__ void store4(void* dst, int64_t at, int left, int lane, int h, const float2 (&x)[2]) {
  if (kVec && place<kVec>(lane, h, 3) < left) {
    if constexpr (kBf16) {
      __nv_bfloat162 w[2] = {__float22bfloat162_rn(x[0]), __float22bfloat162_rn(x[1])};
      __stcs(reinterpret_cast<uint2*>(static_cast<uint16_t*>(dst) + at + place<kVec>(lane, h, 0)),
             *reinterpret_cast<const uint2*>(w));
    } else {
      __stcs(reinterpret_cast<float4*>(static_cast<float*>(dst) + at + place<kVec>(lane, h, 0)),
             make_float4(x[0].x, x[0].y, x[1].x, x[1].y));
    }
    return;
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int e = place<kVec>(lane, h, j);
    if (e >= left) continue;
    const float xj = j & 1 ? x[j >> 1].y : x[j >> 1].x;
    if constexpr (kBf16) static_cast<__nv_bfloat16*>(dst)[at + e] = __float2bfloat16_rn(xj);
    else static_cast<float*>(dst)[at + e] = xj;
  }
}

template <bool kVec>
__device__ __forceinline__ uint32_t load_codes(const void* src, int64_t at, int left, int lane, int h) {
  const uint8_t* s = static_cast<const uint8_t*>(src) + at;
  if (kVec && place<kVec>(lane, h, 3) < left)
    return __ldcs(reinterpret_cast<const uint32_t*>(s + place<kVec>(lane, h, 0)));
  uint32_t c = 0;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int e = place<kVec>(lane, h, j);
    if (e < left) c |= (uint32_t)s[e] << (8 * j);
  }
  return c;
}

template <bool kVec>
__device__ __forceinline__ void store_codes(void* dst, int64_t at, int left, int lane, int h, uint32_t c) {
  uint8_t* d = static_cast<uint8_t*>(dst) + at;
  if (kVec && place<kVec>(lane, h, 3) < left) {
    __stcs(reinterpret_cast<uint32_t*>(d + place<kVec>(lane, h, 0)), c);
    return;
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int e = place<kVec>(lane, h, j);
    if (e < left) d[e] = (uint8_t)(c >> (8 * j));
  }
}

// A sum that is not fused with a product before it (the assembler fuses a pair's).
__device__ __forceinline__ float2 add_apart(float2 a, float2 b) {
  return make_float2(__fadd_rn(a.x, b.x), __fadd_rn(a.y, b.y));
}

// The block's codes and scale of x (kRoot: x >= 0, and what is not zero keeps a code that is not).
template <bool kRoot>
__device__ __forceinline__ float encode_block(const float2 (&x)[2][2], uint32_t (&c)[2]) {
  float top = 0.0f;
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int j = 0; j < 2; ++j) top = ptx::max_nan(ptx::max_nan(top, fabsf(x[h][j].x)), fabsf(x[h][j].y));
  top = __uint_as_float(__reduce_max_sync(0xFFFFFFFFu, __float_as_uint(top)));       // magnitudes order as whole numbers
  if (top < kDeadBlock) {                            // not a NaN: that block's scale is one
    c[0] = c[1] = 0;
    return 0.0f;
  }
  const float2 inv = both(__fdiv_rn(kTop8, top));
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    float2 q[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      q[j] = mul2(x[h][j], inv);
      if (kRoot) {
        if (x[h][j].x > 0.0f) q[j].x = fmaxf(q[j].x, 0x1p-9f);
        if (x[h][j].y > 0.0f) q[j].y = fmaxf(q[j].y, 0x1p-9f);
      }
    }
    c[h] = encode4(q);
  }
  return __fdiv_rn(top, kTop8);
}

// One block of 256 elements, a warp's: all loads first, as they are, then run by run.
template <bool kP16, bool kG16, bool k8, bool kVec>
__device__ __forceinline__ void step_block(const AdamwTensor& t, const AdamwHead& a, int64_t at, int lane, float coef) {
  const int left = (int)min((int64_t)MFSDP_STATE_BLOCK, t.numel - at);
  Raw<kP16> rp[2];
  Raw<kG16> rg[2];
  Raw<false> rm[2], rv[2];
  uint32_t cm[2], cv[2];
  float sm = 0.0f, sv = 0.0f;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    rp[h] = load4<kP16, kVec>(t.p, at, left, lane, h);
    rg[h] = load4<kG16, kVec>(t.g, at, left, lane, h);
    if (k8) {
      cm[h] = load_codes<kVec>(t.m, at, left, lane, h);
      cv[h] = load_codes<kVec>(t.v, at, left, lane, h);
    } else {
      rm[h] = load4<false, kVec>(t.m, at, left, lane, h);
      rv[h] = load4<false, kVec>(t.v, at, left, lane, h);
    }
  }
  if (k8) {
    sm = t.m_scale[at / MFSDP_STATE_BLOCK];
    sv = t.v_scale[at / MFSDP_STATE_BLOCK];
  }
  float2 new_m[2][2], new_r[2][2];                   // 8-bit states: kept for the block's scales
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    float2 p[2], g[2], m[2], v[2];
    rp[h].get(p);
    rg[h].get(g);
    if (k8) {
      decode4(cm[h], m);
      decode4(cv[h], v);
    } else {
      rm[h].get(m);
      rv[h].get(v);
    }
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      if (k8) {
        m[j] = mul2(m[j], both(sm));
        v[j] = mul2(v[j], both(sv));
        v[j] = mul2(v[j], v[j]);
      }
      g[j] = mul2(g[j], both(coef));
      m[j] = add_apart(mul2(m[j], both(a.beta1)), mul2(g[j], both(a.omb1)));
      v[j] = add_apart(mul2(v[j], both(a.beta2)), mul2(mul2(g[j], both(a.omb2)), g[j]));
      const float2 root = k8 ? ptx::root(v[j]) : make_float2(ptx::sqrt_approx(v[j].x), ptx::sqrt_approx(v[j].y));
      const float2 den = fma2(root, both(a.inv_sqrt_bc2), both(a.eps));
      const float2 inv = make_float2(ptx::rcp_approx(den.x), ptx::rcp_approx(den.y));
      p[j] = fma2(mul2(m[j], inv), both(-t.step_size), mul2(p[j], both(t.decay)));
      new_m[h][j] = m[j];
      new_r[h][j] = root;
    }
    store4<kP16, kVec>(t.p, at, left, lane, h, p);
    if (t.copy) store4<true, kVec>(t.copy, at, left, lane, h, p);
    if (!k8) {
      store4<false, kVec>(t.m, at, left, lane, h, m);
      store4<false, kVec>(t.v, at, left, lane, h, v);
    }
  }
  if (k8) {
    if (left < MFSDP_STATE_BLOCK) {                  // places past the end count for nothing
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          if (place<kVec>(lane, h, 2 * j) >= left) new_m[h][j].x = new_r[h][j].x = 0.0f;
          if (place<kVec>(lane, h, 2 * j + 1) >= left) new_m[h][j].y = new_r[h][j].y = 0.0f;
        }
    }
    sm = encode_block<false>(new_m, cm);
    sv = encode_block<true>(new_r, cv);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      store_codes<kVec>(t.m, at, left, lane, h, cm[h]);
      store_codes<kVec>(t.v, at, left, lane, h, cv[h]);
    }
    if (lane == 0) {
      t.m_scale[at / MFSDP_STATE_BLOCK] = sm;
      t.v_scale[at / MFSDP_STATE_BLOCK] = sv;
    }
  }
}

// What a launch's tensors are: 32-bit states alone, which have more bytes on their way in each thread and take their
// registers from a fourth CTA (131 M elements: 513 us, with four 516); 8-bit ones too, all on 4 elements' boundaries,
// which gain by more warps (324 us with six CTAs, 337 with five, 359 with four); or any, whose single elements would
// not have the registers (4 x 10 M off the boundaries: 118 with five, 123 with six).
enum Set { kWide, kEightOnFour, kAll };
constexpr int kCtas[] = {3, 6, 5};
template <int kN, Set kSet>
__global__ void __launch_bounds__(kThreads, kCtas[kSet]) adamw_set_kernel(const __grid_constant__ AdamwBatch<kN> b) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const float coef = b.norm ? b.norm[1] : 1.0f;
  int which = 0;
  for (int ch = blockIdx.x; ch < b.chunks; ch += gridDim.x) {
    which = find_tensor(b, ch, which);
    const AdamwTensor& t = b.t[which];
    const int64_t at = (int64_t)(ch - t.chunk0) * kAdamwChunk + warp * MFSDP_STATE_BLOCK;
    if (at >= t.numel) continue;
    switch (t.form) {
#define MFSDP_FORM(f) \
  case f: \
    if constexpr (kSet == kWide ? !(f & 4) : kSet == kAll || (f & 8)) \
      step_block<(f & 1) != 0, (f & 2) != 0, (f & 4) != 0, (f & 8) != 0>(t, b, at, lane, coef); \
    break;
      MFSDP_FORM(0) MFSDP_FORM(1) MFSDP_FORM(2) MFSDP_FORM(3) MFSDP_FORM(4) MFSDP_FORM(5) MFSDP_FORM(6)
      MFSDP_FORM(7) MFSDP_FORM(8) MFSDP_FORM(9) MFSDP_FORM(10) MFSDP_FORM(11) MFSDP_FORM(12) MFSDP_FORM(13)
      MFSDP_FORM(14) MFSDP_FORM(15)
#undef MFSDP_FORM
    }
  }
}

// Far more CTAs than run at once: a chunk of a fresh CTA is under way before the last of another's is written (131 M
// elements, fp32 states: one CTA a chunk 513 us, 64 an SM 524, 8 an SM 540, one round of them 572; 8 bits, with what a
// CTA looks up first: 50 an SM 337, 100 an SM 341, one a chunk 351, 8 an SM 364).
template <int kN>
cudaError_t launch(const AdamwBatch<kN>& b, Set set, int sms, cudaStream_t s) {
  const int blocks = set == kWide ? b.chunks : std::min(b.chunks, 50 * sms);
  if (set == kWide) adamw_set_kernel<kN, kWide><<<blocks, kThreads, 0, s>>>(b);
  else if (set == kEightOnFour) adamw_set_kernel<kN, kEightOnFour><<<blocks, kThreads, 0, s>>>(b);
  else adamw_set_kernel<kN, kAll><<<blocks, kThreads, 0, s>>>(b);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_adamw_set(const AdamwBatch<kAdamwTable>& b, int sms, cudaStream_t s) {
  bool eight = false, on_four = true;
  for (int i = 0; i < b.n; ++i) {
    eight = eight || (b.t[i].form & 4);
    on_four = on_four && (b.t[i].form & 8);
  }
  const Set set = !eight ? kWide : on_four ? kEightOnFour : kAll;
  if (b.n > kAdamwShort) return launch(b, set, sms, s);
  AdamwBatch<kAdamwShort> sb;                        // a launch copies its parameters: 30 KB or 1
  static_cast<AdamwHead&>(sb) = b;
  std::memcpy(sb.t, b.t, sizeof(AdamwTensor) * b.n);
  return launch(sb, set, sms, s);
}

}  // namespace ops
}  // namespace mfsdp
