// Log-probabilities of given tokens, with entropy and top alternatives, and their gradient.
//
//   z = scale x,  M = max z,  S = sum exp(z - M),  T = sum exp(z - M) (z - M)
//   lse = M + log S,   logprob = (z_y - M) - log S,   entropy = log S - T / S
//   dx_j = scale (dlogprob ([j = y] - p_j) - dentropy p_j (log p_j + entropy))
//
// A sure token's S is barely above 1, and its logprob is -log S.  So what threads, warps and CTAs hand on is R = S - 1, the
// sum without one of the largest logit's terms, which is 1 whatever that logit: log S = log1p(R).
//
// The embedding's other end: a training batch has gigabytes of logits, which go by once
// (forward) or once in and once out (gradient).
//
// Forward: batches without alternatives go by teams of warps, as many to a row as leave each team some turns; with
// alternatives a row is a CTA's or, where there are few rows, a cluster's of up to 16 CTAs,
// each of which takes a run of the row's vectors.  A thread keeps its own
// running M (in powers of two: exp2 is what the hardware has), S and T; a new maximum scales the other two, once for
// a batch of vectors.  Threads, warps and CTAs are joined in a fixed order.
//
// Top alternatives without another pass: the threads' maxima, taken over 64 groups of
// threads, bound the k-th largest logit from below (k <= 32 groups' maxima are k
// elements).  Only the elements of threads whose own maximum reaches that bound are read again, by all threads,
// and what reaches the bound is sorted by counting: some 20 to 50 candidates as a rule.  Where more
// than the list holds reach it, the k largest are taken one by one over the row, which is slow and right: a row of
// equal logits, or one with fewer than k groups that have a live logit, whose bound is -inf (20 alternatives of 32000 logits:
// 10 live 26.7 us for one row and 3.1 ms for 8000, 300 live 10.3 and 120).  A cluster's CTAs sort their own, the first merges.
//
// Bound by HBM: 32768 x 32000 bf16 take 308 us forward (6.8 TB/s) and 623 us for the gradient (6.7 TB/s, the issue slots
// some 80 % full).  One row of a generated token is latency: 7.7 us in a graph.
#include <cuda_bf16.h>

#include <algorithm>
#include <type_traits>

#include "ops_internal.h"
#include "ops_ptx.cuh"

namespace mfsdp {
namespace ops {
namespace {

constexpr int kWideThreads = 512, kNarrowThreads = 128;      // of a CTA that has a row, or a part of one
constexpr int kMaxCluster = 16;
constexpr int kGroups = 64;                   // groups of threads whose maxima bound the alternatives
constexpr int kCandidates = 1024;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr float kLeast = -1000.0f;            // exp2 of less is 0; keeps 0 * -inf out of T
constexpr float kFloor = -0x1p101f;           // what a masked logit becomes; the same twice in bf16
constexpr uint32_t kFloorPair = 0xF200F200u;
constexpr float kRange = 0x1p100f;            // a logit below -2^100 is masked, a row with one above 2^100 has no sum

using ptx::add2;
using ptx::both;
using ptx::fma2;
using ptx::mul2;

__device__ __forceinline__ float lo16(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi16(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// Elements of a 16-byte vector.
template <bool kBf16>
constexpr int kPer = kBf16 ? 8 : 4;

template <bool kBf16>
__device__ __forceinline__ void unpack(const uint4& q, float (&x)[kPer<kBf16>]) {
  if constexpr (kBf16) {
    x[0] = lo16(q.x); x[1] = hi16(q.x); x[2] = lo16(q.y); x[3] = hi16(q.y);
    x[4] = lo16(q.z); x[5] = hi16(q.z); x[6] = lo16(q.w); x[7] = hi16(q.w);
  } else {
    x[0] = __uint_as_float(q.x); x[1] = __uint_as_float(q.y); x[2] = __uint_as_float(q.z); x[3] = __uint_as_float(q.w);
  }
}

template <bool kBf16>
__device__ __forceinline__ float load_one(const void* p, int64_t i) {
  if constexpr (kBf16) return __uint_as_float((uint32_t)__ldg(static_cast<const uint16_t*>(p) + i) << 16);
  else return __ldg(static_cast<const float*>(p) + i);
}

// A running maximum (of x, not scaled), the sum without one of the maximum's terms (-1 where there is none: no live
// logit yet), and the weighted sum, in which that term is 0.  The maximum starts at -2^100, so that it
// times k2 is finite: an element below is 2^77 below at least, and adds nothing.
struct Stats {
  float m, rest, t;
};

// Here and below the difference comes before the product: the largest logit's is then 0 and its term 1, whatever its size.
__device__ __forceinline__ Stats join(const Stats& a, const Stats& b, float k2) {
  const bool first = a.m >= b.m;
  const float d = (first ? b.m - a.m : a.m - b.m) * k2;      // <= 0; NaN only where both are +inf, and R is NaN already
  const float c = ptx::exp2_approx(d), less = 1.0f + (first ? b.rest : a.rest);
  return {fmaxf(a.m, b.m), fmaf(c, less, first ? a.rest : b.rest),
          fmaf(c, fmaf(less, fmaxf(d, kLeast), first ? b.t : a.t), first ? a.t : b.t)};
}

// A thread's own sums: of pairs of elements, so that they take two operations an instruction.  kApart: the batch of vectors
// that has the maximum is summed apart, so that no sum of many terms has the maximum's 1 beside them.
template <bool kEntropy, bool kApart>
struct Sums {
  float m;
  float2 s, t;       // s: without that batch, whose sum is b
  float b;
  int at;            // its first vector; -1: it is a single element, or none
  __device__ __forceinline__ Sums() : m(-kRange), s(make_float2(0.0f, 0.0f)), t(make_float2(0.0f, 0.0f)), b(0.0f), at(-1) {}
  __device__ __forceinline__ void raise(float to, float k2) {          // to > m
    const float d = (m - to) * k2;             // NaN only where both are +inf, and the sum is NaN already
    const float2 c = both(ptx::exp2_approx(d));
    if (kApart) s.x += b;
    if (kEntropy) t = mul2(c, fma2(s, both(fmaxf(d, kLeast)), t));
    s = mul2(c, s);
    m = to;
  }
  __device__ __forceinline__ void add(float2 x, float k2, float2 less_m, float2& sum) {
    const float2 d = mul2(add2(x, less_m), both(k2));
    const float2 e = make_float2(ptx::exp2_approx(d.x), ptx::exp2_approx(d.y));
    sum = add2(sum, e);
    if (kEntropy) t = fma2(e, d, t);
  }
  __device__ __forceinline__ void add_one(float x, float k2) {
    if (kEntropy) x = ptx::max_nan(x, kFloor);
    const bool up = x > m;
    if (up) raise(x, k2);
    const float d = (x - m) * k2, e = ptx::exp2_approx(d);
    if (kEntropy) t.x = fmaf(e, d, t.x);
    if (kApart && up) {
      b = e;
      at = -1;
    } else {
      s.x += e;
    }
  }
  // Some vectors at once, the first of them vector i: one look for a new maximum.  With the entropy, masked logits
  // become -2^101, which adds 0 times a finite number.
  template <bool kBf16, int kVecs>
  __device__ __forceinline__ void add(uint4 (&v)[kVecs], float k2, int64_t i) {
    float top;
    if constexpr (kBf16) {
      uint32_t mm = 0xFF7FFF7Fu;               // the lowest number twice
#pragma unroll
      for (int b = 0; b < kVecs; ++b) {
        if (kEntropy) {
          v[b].x = ptx::max_nan_bf16x2(v[b].x, kFloorPair);
          v[b].y = ptx::max_nan_bf16x2(v[b].y, kFloorPair);
          v[b].z = ptx::max_nan_bf16x2(v[b].z, kFloorPair);
          v[b].w = ptx::max_nan_bf16x2(v[b].w, kFloorPair);
        }
        mm = ptx::max_bf16x2(mm, ptx::max_bf16x2(ptx::max_bf16x2(v[b].x, v[b].y), ptx::max_bf16x2(v[b].z, v[b].w)));
      }
      top = fmaxf(lo16(mm), hi16(mm));
    } else {
      top = -kRange;
#pragma unroll
      for (int b = 0; b < kVecs; ++b) {
        if (kEntropy) {
          v[b].x = __float_as_uint(ptx::max_nan(__uint_as_float(v[b].x), kFloor));
          v[b].y = __float_as_uint(ptx::max_nan(__uint_as_float(v[b].y), kFloor));
          v[b].z = __float_as_uint(ptx::max_nan(__uint_as_float(v[b].z), kFloor));
          v[b].w = __float_as_uint(ptx::max_nan(__uint_as_float(v[b].w), kFloor));
        }
        top = fmaxf(top, fmaxf(fmaxf(__uint_as_float(v[b].x), __uint_as_float(v[b].y)),
                               fmaxf(__uint_as_float(v[b].z), __uint_as_float(v[b].w))));
      }
    }
    const bool up = top > m;
    if (up) raise(top, k2);
    const float2 less_m = both(-m);
    float2 sum = kApart ? make_float2(0.0f, 0.0f) : s;
#pragma unroll
    for (int b = 0; b < kVecs; ++b) {
      const uint32_t w[4] = {v[b].x, v[b].y, v[b].z, v[b].w};
      if constexpr (kBf16) {
#pragma unroll
        for (int j = 0; j < 4; ++j) add(make_float2(lo16(w[j]), hi16(w[j])), k2, less_m, sum);
      } else {
        add(make_float2(__uint_as_float(w[0]), __uint_as_float(w[1])), k2, less_m, sum);
        add(make_float2(__uint_as_float(w[2]), __uint_as_float(w[3])), k2, less_m, sum);
      }
    }
    if (!kApart) {
      s = sum;
    } else if (up) {
      b = sum.x + sum.y;
      at = (int)i;
    } else {
      s = add2(s, sum);
    }
  }
  __device__ __forceinline__ Stats stats() const { return {m, s.x + s.y + (b - 1.0f), t.x + t.y}; }
};

// A run of a row: `head` single elements up to the first 16-byte boundary, vectors, and `tail`
// single elements, from element `from` on.
struct Span {
  int64_t from;
  int head, tail;
  int64_t vecs;
};
template <bool kBf16>
__device__ __forceinline__ Span span_of(const void* row, int64_t vocab, int part, int parts) {
  constexpr int kSize = kBf16 ? 2 : 4;
  const int64_t head = min((int64_t)(((16 - (reinterpret_cast<uintptr_t>(row) & 15)) & 15) / kSize), vocab);
  const int64_t vecs = (vocab - head) / kPer<kBf16>;
  const int64_t v0 = vecs * part / parts, v1 = vecs * (part + 1) / parts;
  Span s;
  s.from = part == 0 ? 0 : head + v0 * kPer<kBf16>;
  s.head = part == 0 ? (int)head : 0;
  s.vecs = v1 - v0;
  s.tail = part == parts - 1 ? (int)(vocab - head - vecs * kPer<kBf16>) : 0;
  return s;
}

// Calls f(element index, value) for each of this thread's elements of the span.
template <bool kBf16, int kThreads, typename F>
__device__ __forceinline__ void each_element(const void* row, const Span& sp, F&& f) {
  const int tid = threadIdx.x;
  if (tid < sp.head) f(sp.from + tid, load_one<kBf16>(row, sp.from + tid));
  const int64_t v = sp.from + sp.head, end = v + sp.vecs * kPer<kBf16>;
  const uint4* q = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(row) + v * (kBf16 ? 2 : 4));
  for (int64_t i = tid; i < sp.vecs; i += kThreads) {
    float x[kPer<kBf16>];
    unpack<kBf16>(__ldg(q + i), x);
#pragma unroll
    for (int j = 0; j < kPer<kBf16>; ++j) f(v + i * kPer<kBf16> + j, x[j]);
  }
  if (tid < sp.tail) f(end + tid, load_one<kBf16>(row, end + tid));
}

// This thread's sums over a span that `threads` threads share, kVecs vectors at a time.
template <bool kBf16, bool kEntropy, int kVecs, bool kApart>
__device__ __forceinline__ Sums<kEntropy, kApart> sums_of(const uint8_t* row, const Span& sp, int tid, int threads, float k2) {
  Sums<kEntropy, kApart> st;
  const uint4* q = reinterpret_cast<const uint4*>(row + (sp.from + sp.head) * (kBf16 ? 2 : 4));
  int64_t i = tid;
  for (; i + (int64_t)(kVecs - 1) * threads < sp.vecs; i += (int64_t)kVecs * threads) {
    uint4 v[kVecs];
#pragma unroll
    for (int b = 0; b < kVecs; ++b) v[b] = __ldg(q + i + b * threads);
    st.template add<kBf16>(v, k2, i);
  }
  if (i < sp.vecs) {                           // fewer: vectors that are not there are masked
    uint4 v[kVecs];
#pragma unroll
    for (int b = 0; b < kVecs; ++b)
      v[b] = i + b * threads < sp.vecs ? __ldg(q + i + b * threads)
             : kBf16                   ? make_uint4(0xFF80FF80u, 0xFF80FF80u, 0xFF80FF80u, 0xFF80FF80u)
                                       : make_uint4(0xFF800000u, 0xFF800000u, 0xFF800000u, 0xFF800000u);
    st.template add<kBf16>(v, k2, i);
  }
  if (tid < sp.head) st.add_one(load_one<kBf16>(row, sp.from + tid), k2);
  if (tid < sp.tail) st.add_one(load_one<kBf16>(row, sp.from + sp.head + sp.vecs * kPer<kBf16> + tid), k2);
  return st;
}

// A row's joined sums as what they stand for.
struct Row {
  bool empty, bad;
  float m, logs;
  __device__ __forceinline__ explicit Row(const Stats& st)
      : empty(st.rest < -0.5f),                // -1: every logit is masked
        bad(!(st.rest < INFINITY) || st.m > kRange),         // a NaN or +inf
        m(st.m), logs(log1pf(st.rest)) {}
  __device__ __forceinline__ float logprob(float x, float scale) const {
    if (bad) return NAN;
    if (empty || x < -kRange) return -INFINITY;
    return fmaf(x - m, scale, -logs);
  }
};

// What a row has one of.
template <bool kBf16, bool kEntropy>
__device__ __forceinline__ void put_row(const LogprobArgs& a, int64_t t, const void* row, const Stats& st) {
  const Row r(st);
  // From the rounded product, as the gradient takes it: a sure token's is then lse itself.
  if (a.lse) a.lse[t] = r.bad ? NAN : r.empty ? -INFINITY : __fadd_rn(__fmul_rn(r.m, a.scale), r.logs);
  if (kEntropy) a.entropy[t] = r.bad ? NAN : r.empty ? 0.0f : fmaf(st.t / (1.0f + st.rest), -kLn2, r.logs);
  if (a.logprob) {
    const int64_t y = a.ids64 ? static_cast<const int64_t*>(a.targets)[t] : static_cast<const int32_t*>(a.targets)[t];
    a.logprob[t] = y < 0 || y >= a.vocab ? 0.0f : r.logprob(load_one<kBf16>(row, y), a.scale);
  }
}

// The sums of a warp from its threads', each over a span's vectors tid, tid + threads and so on, kVecs at a time.  The thread
// with the largest logit has that one's 1 among its terms, which lose what is below 2^-24 beside it.  Where all else is
// small against the 1, they are summed once more without it: the vectors of one thread, near as a rule, or (kApart) one
// batch of them.
constexpr float kSmallRest = 0.5f;
template <bool kBf16, int kVecs, bool kEntropy, bool kApart>
__device__ __forceinline__ Stats warp_sums(const Sums<kEntropy, kApart>& sums, const uint8_t* row, const Span& sp, int tid,
                                           int threads, float k2) {
  constexpr uint32_t kAll = 0xFFFFFFFFu;
  const int lane = tid & 31;
  const Stats mine = sums.stats();
  const int order = __float_as_int(mine.m) ^ (__float_as_int(mine.m) >> 31 & 0x7FFFFFFF);      // ordered as the maxima are
  const bool largest = order == __reduce_max_sync(kAll, order);
  const int owner = __ffs(__ballot_sync(kAll, largest)) - 1;
  Stats st;
  st.m = __shfl_sync(kAll, mine.m, owner);
  const float d = (mine.m - st.m) * k2, c = ptx::exp2_approx(d), all = 1.0f + mine.rest;       // d: see join
  st.rest = lane == owner ? 0.0f : c * all;
  st.t = lane == owner ? mine.t : c * fmaf(all, fmaxf(d, kLeast), mine.t);
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    st.rest += __shfl_xor_sync(kAll, st.rest, o);
    if (kEntropy) st.t += __shfl_xor_sync(kAll, st.t, o);
  }
  const float others = st.rest;
  st.rest += __shfl_sync(kAll, mine.rest, owner);
  if (!(st.m > -kRange && st.rest < kSmallRest)) return st;  // (a maximum at -2^100 came in no batch)
  const int at = kApart ? __shfl_sync(kAll, sums.at, owner) : tid - lane + owner;
  float sum = kApart && lane == owner ? sums.s.x + sums.s.y : 0.0f;
  const auto add = [&](float x) {
    if (x != st.m) sum += ptx::exp2_approx((x - st.m) * k2);   // one element is st.m: of two the rest would be 1
  };
  const auto add_vector = [&](int64_t i) {
    float x[kPer<kBf16>];
    unpack<kBf16>(__ldg(reinterpret_cast<const uint4*>(row + (sp.from + sp.head) * (kBf16 ? 2 : 4)) + i), x);
#pragma unroll
    for (int j = 0; j < kPer<kBf16>; ++j) add(x[j]);
  };
  const int64_t i = at + (int64_t)lane * threads;
  if constexpr (kApart) {
    if (at >= 0 && lane < kVecs && i < sp.vecs) add_vector(i);
  } else {
    for (int64_t k = i; k < sp.vecs; k += (int64_t)32 * threads) add_vector(k);
    if (lane == 0 && at < sp.head) add(load_one<kBf16>(row, sp.from + at));
    if (lane == 0 && at < sp.tail) add(load_one<kBf16>(row, sp.from + sp.head + sp.vecs * kPer<kBf16> + at));
  }
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) sum += __shfl_xor_sync(kAll, sum, o);
  st.rest = others + sum;
  return st;
}

// Many rows without alternatives: a team of 1 to 8 warps a row, each team on its own, so that no row's end
// stops the loads of the others.
constexpr int kRowThreads = 256;
constexpr int kRowTurns = 6;                  // rows that a team takes at least, before it grows
// CTAs for every one that runs at once: a fresh CTA's loads are under way while others end (32768 x 32000 bf16, when this
// was chosen: 302 us, with one 308, with 16 303; gradient 624, with one 641, two 635,
// 16 624; few long rows lose 2 to 3 %: 2000 x 100000 74.5, with one 72.3).
constexpr int kRounds = 4;
template <bool kBf16, bool kEntropy>
__global__ void __launch_bounds__(kRowThreads, 4) logprob_rows_kernel(const LogprobArgs a, int team_warps) {
  __shared__ Stats warp_stats[2][kRowThreads / 32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, team = warp / team_warps, teams = kRowThreads / 32 / team_warps;
  const int threads = team_warps * 32, tid = threadIdx.x - team * threads;
  int turn = 0;
  for (int64_t t = (int64_t)blockIdx.x * teams + team; t < a.n; t += (int64_t)gridDim.x * teams) {
    const uint8_t* row = static_cast<const uint8_t*>(a.x) + t * a.x_ld * (kBf16 ? 2 : 4);
    const Span sp = span_of<kBf16>(row, a.vocab, 0, 1);
    constexpr int kVecs = kBf16 ? 4 : 8;
    Stats st = warp_sums<kBf16, kVecs>(sums_of<kBf16, kEntropy, kVecs, true>(row, sp, tid, threads, a.k2), row, sp, tid,
                                       threads, a.k2);
    if (team_warps > 1) {                      // in turns: one barrier a row
      if (lane == 0) warp_stats[turn][warp] = st;
      asm volatile("bar.sync %0, %1;" ::"r"(team + 1), "r"(threads) : "memory");
      if (tid == 0)
        for (int w = 1; w < team_warps; ++w) st = join(st, warp_stats[turn][warp + w], a.k2);
      turn ^= 1;
    }
    if (tid == 0) put_row<kBf16, kEntropy>(a, t, row, st);
  }
}

// Logit and index as one whole number: a larger logit, then a smaller index, is larger.  No logit gives 0.
__device__ __forceinline__ uint64_t key_of(float x, int64_t i) {
  const uint32_t b = __float_as_uint(x + 0.0f);              // -0 counts as 0
  const uint32_t o = b & 0x80000000u ? ~b : b | 0x80000000u;
  return (uint64_t)o << 32 | (0xFFFFFFFFu - (uint32_t)i);
}
__device__ __forceinline__ float logit_of(uint64_t key) {
  const uint32_t o = (uint32_t)(key >> 32);
  return __uint_as_float(o & 0x80000000u ? o & 0x7FFFFFFFu : ~o);
}
__device__ __forceinline__ int32_t index_of(uint64_t key) { return (int32_t)(0xFFFFFFFFu - (uint32_t)key); }

template <int kThreads>
struct Shared {
  Stats warp[kThreads / 32];
  Stats part[kMaxCluster];                    // of the cluster's CTAs, in the first one
  Stats row;
  alignas(16) float group[kGroups];
  float bound;
  int count, owners;
  uint16_t owner[kThreads];                   // threads whose maximum reaches the bound
  uint64_t best[kThreads / 32];
  uint64_t list[kCandidates];
  uint64_t top[MFSDP_MAX_TOP];                // this CTA's largest
  uint64_t merge[kMaxCluster * MFSDP_MAX_TOP];
};

// The `k` largest keys of the span into sh.top, from the largest down; 0 where there are no more.
// m: this thread's largest logit.
template <bool kBf16, int kThreads>
__device__ void find_top(Shared<kThreads>& sh, const void* row, const Span& sp, float m, int k) {
  const int tid = threadIdx.x;
  constexpr int kGroup = kThreads / kGroups;
  float g = m;
#pragma unroll
  for (int o = 1; o < kGroup; o <<= 1) g = fmaxf(g, __shfl_xor_sync(0xFFFFFFFFu, g, o));
  if (tid % kGroup == 0) sh.group[tid / kGroup] = g;
  if (tid == 0) sh.count = sh.owners = 0;
  if (tid < k) sh.top[tid] = 0;
  __syncthreads();
  if (tid < kGroups) {                        // the k-th largest of the groups' maxima
    const float mine = sh.group[tid];
    int above = 0;
#pragma unroll
    for (int i = 0; i < kGroups; i += 4) {
      const float4 q = *reinterpret_cast<const float4*>(&sh.group[i]);
      above += (q.x > mine || (q.x == mine && i < tid)) + (q.y > mine || (q.y == mine && i + 1 < tid)) +
               (q.z > mine || (q.z == mine && i + 2 < tid)) + (q.w > mine || (q.w == mine && i + 3 < tid));
    }
    if (above == k - 1) sh.bound = mine > -kRange ? mine : -INFINITY;   // masked logits are in no maximum
  }
  __syncthreads();
  const float bound = sh.bound;
  if (m >= bound) sh.owner[atomicAdd(&sh.owners, 1)] = (uint16_t)tid;
  __syncthreads();
  // The owners' vectors, dealt out over all threads: some 20 to 50 owners as a rule.
  const auto note = [&](int64_t i, float x) {
    if (x >= bound) {
      const int at = atomicAdd(&sh.count, 1);
      if (at < kCandidates) sh.list[at] = key_of(x, i);
    }
  };
  const int64_t first = sp.from + sp.head;
  const uint4* q = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(row) + first * (kBf16 ? 2 : 4));
  const uint32_t owners = sh.owners;
  const uint32_t runs = (uint32_t)((sp.vecs + kThreads - 1) / kThreads);       // vectors of a thread
#pragma unroll 2
  for (uint32_t c = tid; c < owners * runs; c += kThreads) {  // at most (2^29 + kThreads) of them
    const int64_t i = sh.owner[c % owners] + (int64_t)(c / owners) * kThreads;
    if (i >= sp.vecs) continue;
    float x[kPer<kBf16>];
    unpack<kBf16>(__ldg(q + i), x);
#pragma unroll
    for (int j = 0; j < kPer<kBf16>; ++j) note(first + i * kPer<kBf16> + j, x[j]);
  }
  if (tid < sp.head) note(sp.from + tid, load_one<kBf16>(row, sp.from + tid));
  const int64_t end = first + sp.vecs * kPer<kBf16>;
  if (tid < sp.tail) note(end + tid, load_one<kBf16>(row, end + tid));
  __syncthreads();
  const int count = sh.count;
  if (count <= kCandidates) {                 // a key's place is the number of larger ones: all keys differ
    for (int c = tid; c < count; c += kThreads) {
      const uint64_t mine = sh.list[c];
      int above = 0;
#pragma unroll 4
      for (int i = 0; i < count; ++i) above += sh.list[i] > mine;
      if (above < k) sh.top[above] = mine;
    }
    __syncthreads();
    return;
  }
  uint64_t last = ~0ull;
  for (int r = 0; r < k; ++r) {
    uint64_t best = 0;
    each_element<kBf16, kThreads>(row, sp, [&](int64_t i, float x) {
      const uint64_t key = key_of(x, i);
      if (key < last && key > best) best = key;
    });
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) best = max(best, __shfl_xor_sync(0xFFFFFFFFu, best, o));
    if ((tid & 31) == 0) sh.best[tid >> 5] = best;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) best = max(best, sh.best[w]);
    if (tid == 0) sh.top[r] = best;
    last = best;
    __syncthreads();
  }
}

template <bool kBf16, bool kEntropy, int kThreads>
__global__ void __launch_bounds__(kThreads) logprob_kernel(const LogprobArgs a, int parts) {
  __shared__ Shared<kThreads> sh;
  const int tid = threadIdx.x;
  const int part = parts > 1 ? (int)ptx::cluster_ctarank() : 0;
  const int64_t t = blockIdx.x / parts;
  const uint8_t* row = static_cast<const uint8_t*>(a.x) + t * a.x_ld * (kBf16 ? 2 : 4);
  const Span sp = span_of<kBf16>(row, a.vocab, part, parts);
  if (parts > 1) ptx::cluster_arrive();
  // Apart in narrow CTAs of bf16 (8000 x 32000: 98.8 us, else 101.2; 30000 x 150: 96.4, else 102.5).  An fp32 batch has half the
  // elements for the same selects (517 x 31999: 22.1 apart, 21.2 not), a wide CTA few batches and no register to spare.
  constexpr bool kApart = kBf16 && kThreads == kNarrowThreads;
  const Sums<kEntropy, kApart> sums = sums_of<kBf16, kEntropy, 4, kApart>(row, sp, tid, kThreads, a.k2);
  const float mine = sums.m;
  Stats st = warp_sums<kBf16, 4>(sums, row, sp, tid, kThreads, a.k2);
  if ((tid & 31) == 0) sh.warp[tid >> 5] = st;
  __syncthreads();
  if (parts > 1) ptx::cluster_wait();         // every CTA runs: the first one's shared memory may be written
  if (tid == 0) {
    for (int w = 1; w < kThreads / 32; ++w) st = join(st, sh.warp[w], a.k2);
    if (parts == 1) {
      sh.row = st;
    } else {
      const uint32_t to = ptx::mapa_shared(ptx::smem_u32(&sh.part[part]), 0);
      ptx::st_shared_cluster_s32(to, __float_as_int(st.m));
      ptx::st_shared_cluster_s32(to + 4, __float_as_int(st.rest));
      ptx::st_shared_cluster_s32(to + 8, __float_as_int(st.t));
    }
  }
  if (a.top_k > 0) {
    find_top<kBf16, kThreads>(sh, row, sp, mine, a.top_k);
    if (parts > 1 && tid < a.top_k)
      ptx::st_shared_cluster_u64(ptx::mapa_shared(ptx::smem_u32(&sh.merge[part * a.top_k + tid]), 0), sh.top[tid]);
  }
  if (parts > 1) {
    ptx::cluster_sync();                      // the first CTA alone goes on; nothing of the others' is read after it
    if (part != 0) return;
    if (tid == 0) {
      st = sh.part[0];
      for (int p = 1; p < parts; ++p) st = join(st, sh.part[p], a.k2);
      sh.row = st;
    }
    if (a.top_k > 0) {                        // keys differ but for the zeros of CTAs with less than k elements
      for (int c = tid; c < parts * a.top_k; c += kThreads) {
        const uint64_t key = sh.merge[c];
        int above = 0;
        for (int i = 0; i < parts * a.top_k; ++i) above += sh.merge[i] > key;
        if (key != 0 && above < a.top_k) sh.top[above] = key;
      }
    }
  }
  __syncthreads();
  st = sh.row;
  if (tid == 0) put_row<kBf16, kEntropy>(a, t, row, st);
  if (tid < a.top_k) {
    const Row r(st);
    const uint64_t key = sh.top[tid];
    if (a.top_ids) a.top_ids[t * a.top_k + tid] = r.bad ? -1 : index_of(key);
    if (a.top_logprob) a.top_logprob[t * a.top_k + tid] = r.logprob(logit_of(key), a.scale);
  }
}

// ------------------------------------------------------------------ gradient
constexpr int kGradThreads = 256;
constexpr int kGradVecs = 8;                  // vectors that a thread loads at once (4: 690 us, 2: 777; 32768 x 32000 bf16)

struct RowTerms {
  float lse;
  float dlp, dent;   // the gradients of the log-probability and the entropy
  float entropy;
  int64_t y;         // the target, -1 where it is masked
};

// Of elements i and i + 1.  The product with the scale is rounded before lse is taken away, as it was when lse was made: the
// two roundings of a row's largest logit are one and the same, and p of a sure token is 1.  (Not on pairs: the assembler
// would fuse them.)
__device__ __forceinline__ float2 grad_of(float2 x, int64_t i, const LogprobGradArgs& a, const RowTerms& r) {
  const float2 logp = make_float2(__fsub_rn(__fmul_rn(x.x, a.scale), r.lse), __fsub_rn(__fmul_rn(x.y, a.scale), r.lse));
  const float2 power = mul2(logp, both(kLog2e));
  const float2 p = make_float2(ptx::exp2_approx(power.x), ptx::exp2_approx(power.y));
  float2 c = both(-r.dlp);
  if (r.dent != 0.0f) c = fma2(both(-r.dent), add2(logp, both(r.entropy)), c);
  float2 d = mul2(p, c);
  d.x = p.x > 0.0f || p.x != p.x ? d.x : 0.0f;               // c may be infinite; a NaN stays one
  d.y = p.y > 0.0f || p.y != p.y ? d.y : 0.0f;
  if (i == r.y) d.x = __fadd_rn(d.x, r.dlp);
  if (i + 1 == r.y) d.y = __fadd_rn(d.y, r.dlp);
  return mul2(d, both(a.scale));
}

// Not by the read-only path (load_one): in place, other threads write the same line.
template <bool kBf16>
__device__ __forceinline__ float load_own(const void* p, int64_t i) {
  if constexpr (kBf16) return __uint_as_float((uint32_t)static_cast<const uint16_t*>(p)[i] << 16);
  else return static_cast<const float*>(p)[i];
}

template <bool kBf16>
__device__ __forceinline__ void store_one(void* p, int64_t i, float v) {
  if constexpr (kBf16) static_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(v);
  else static_cast<float*>(p)[i] = v;
}

template <bool kBf16>
__device__ __forceinline__ uint4 pack(const float (&x)[kPer<kBf16>]) {
  if constexpr (kBf16) {
    __nv_bfloat162 h[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) h[j] = __floats2bfloat162_rn(x[2 * j], x[2 * j + 1]);
    return *reinterpret_cast<const uint4*>(h);
  } else {
    return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
  }
}

// A warp takes a row, or one of `parts` equal runs of it, by itself: the row's terms are fetched once for all of it, and
// no warp waits for another.
template <bool kBf16>
__global__ void __launch_bounds__(kGradThreads) logprob_grad_kernel(const LogprobGradArgs a, int parts) {
  constexpr int kSize = kBf16 ? 2 : 4, kStep = kPer<kBf16>;
  const int lane = threadIdx.x & 31;
  const int64_t warps = (int64_t)gridDim.x * (kGradThreads / 32), items = a.n * parts;
  for (int64_t item = (int64_t)blockIdx.x * (kGradThreads / 32) + (threadIdx.x >> 5); item < items; item += warps) {
    const int64_t t = item / parts;
    const int part = (int)(item - t * parts);
    const uint8_t* row = static_cast<const uint8_t*>(a.x) + t * a.x_ld * kSize;
    uint8_t* out = static_cast<uint8_t*>(a.dx) + t * a.dx_ld * kSize;
    RowTerms r;
    r.y = -1;
    if (a.targets) {
      r.y = a.ids64 ? static_cast<const int64_t*>(a.targets)[t] : static_cast<const int32_t*>(a.targets)[t];
      if (r.y < 0 || r.y >= a.vocab) r.y = -1;
    }
    r.dlp = a.dlogprob ? a.dlogprob[t] : 0.0f;
    r.dent = a.dentropy ? a.dentropy[t] : 0.0f;
    r.entropy = a.dentropy ? a.entropy[t] : 0.0f;
    r.lse = a.lse[t];
    if (r.y < 0) r.dlp = 0.0f;
    const bool zero = (r.dlp == 0.0f && r.dent == 0.0f) || r.lse == -INFINITY;
    const auto single = [&](int64_t i) {
      store_one<kBf16>(out, i, zero ? 0.0f : grad_of(both(load_own<kBf16>(row, i)), i, a, r).x);
    };
    // vectors where both rows reach their 16-byte boundaries together
    if (((reinterpret_cast<uintptr_t>(row) ^ reinterpret_cast<uintptr_t>(out)) & 15) != 0) {
      const int64_t end = a.vocab * (part + 1) / parts;
      for (int64_t i = a.vocab * part / parts + lane; i < end; i += 32) single(i);
      continue;
    }
    const Span sp = span_of<kBf16>(row, a.vocab, part, parts);
    const int64_t first = sp.from + sp.head, end = first + sp.vecs * kStep;
    if (lane < sp.head) single(sp.from + lane);
    if (lane < sp.tail) single(end + lane);
    const uint4* q = reinterpret_cast<const uint4*>(row + first * kSize) + lane;
    uint4* o = reinterpret_cast<uint4*>(out + first * kSize) + lane;
    if (zero) {
      for (int64_t i = lane; i < sp.vecs; i += 32, o += 32) __stcs(o, make_uint4(0, 0, 0, 0));
      continue;
    }
    for (int64_t i = lane; i < sp.vecs; i += 32 * kGradVecs, q += 32 * kGradVecs, o += 32 * kGradVecs) {
      uint4 v[kGradVecs];
#pragma unroll
      for (int b = 0; b < kGradVecs; ++b)
        if (i + b * 32 < sp.vecs) v[b] = __ldcs(q + b * 32);
#pragma unroll
      for (int b = 0; b < kGradVecs; ++b) {
        if (i + b * 32 >= sp.vecs) break;
        float x[kStep];
        unpack<kBf16>(v[b], x);
#pragma unroll
        for (int j = 0; j < kStep; j += 2) {
          const float2 d = grad_of(make_float2(x[j], x[j + 1]), first + (i + b * 32) * kStep + j, a, r);
          x[j] = d.x;
          x[j + 1] = d.y;
        }
        __stcs(o + b * 32, pack<kBf16>(x));
      }
    }
  }
}

}  // namespace

cudaError_t launch_logprob(const LogprobArgs& a, int sms, cudaStream_t s) {
  const int64_t resident = (int64_t)sms * 4 * (kRowThreads / 32);      // warps
  if (a.top_k == 0 && a.n * 8 >= resident) {
    int warps = 1;
    while (warps < 8 && a.n * warps < kRowTurns * resident) warps *= 2;
    const int teams = kRowThreads / 32 / warps;
    const unsigned blocks = (unsigned)std::min<int64_t>((a.n + teams - 1) / teams, (int64_t)sms * 4 * kRounds);
    const auto rows = a.x_bf16 ? (a.entropy ? logprob_rows_kernel<true, true> : logprob_rows_kernel<true, false>)
                               : (a.entropy ? logprob_rows_kernel<false, true> : logprob_rows_kernel<false, false>);
    rows<<<blocks, kRowThreads, 0, s>>>(a, warps);
    return cudaGetLastError();
  }
  // Rows alone fill the GPU from a few per SM on; fewer are split, down to some 256 vectors a CTA.
  const int64_t vecs = a.vocab / (a.x_bf16 ? 8 : 4);
  int parts = 1;
  while (parts < kMaxCluster && a.n * parts * 2 <= 2 * sms && vecs / (parts * 2) >= kWideThreads / 2) parts *= 2;
  // Narrow CTAs leave more rows in flight while some are at their ends (8000 x 32000 with 5 alternatives: 99 us, wide 174;
  // 30000 x 150: 99 and 619; 517 x 31999 fp32: 21 both).
  const bool narrow = parts == 1 && (vecs <= 1024 || a.n >= 2 * sms);
  const int threads = narrow ? kNarrowThreads : kWideThreads;
  const auto pick = [&](auto bf16, auto entropy) {
    return narrow ? logprob_kernel<bf16(), entropy(), kNarrowThreads> : logprob_kernel<bf16(), entropy(), kWideThreads>;
  };
  using std::false_type;
  using std::true_type;
  const auto kernel = a.x_bf16 ? (a.entropy ? pick(true_type{}, true_type{}) : pick(true_type{}, false_type{}))
                               : (a.entropy ? pick(false_type{}, true_type{}) : pick(false_type{}, false_type{}));
  if (parts > 8) {
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
  }
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = (unsigned)parts;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(a.n * parts));
  cfg.blockDim = dim3((unsigned)threads);
  cfg.stream = s;
  cfg.attrs = &attr;
  cfg.numAttrs = parts > 1 ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kernel, a, parts);
}

cudaError_t launch_logprob_grad(const LogprobGradArgs& a, int sms, cudaStream_t s) {
  // Rows are divided until there are some turns of them for every resident warp, down to 64 vectors each.
  const int64_t resident = (int64_t)sms * 48, vecs = a.vocab / (a.x_bf16 ? 8 : 4);
  int parts = 1;
  while (a.n * parts < kRowTurns * resident && vecs / (parts * 2) >= 64) parts *= 2;
  const int64_t warps = kGradThreads / 32;
  const unsigned blocks = (unsigned)std::min<int64_t>((a.n * parts + warps - 1) / warps, kRounds * resident / warps);
  if (a.x_bf16) logprob_grad_kernel<true><<<blocks, kGradThreads, 0, s>>>(a, parts);
  else logprob_grad_kernel<false><<<blocks, kGradThreads, 0, s>>>(a, parts);
  return cudaGetLastError();
}

}  // namespace ops
}  // namespace mfsdp
