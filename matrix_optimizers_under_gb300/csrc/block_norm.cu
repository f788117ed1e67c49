// The norms around a block, fused with its gate and the residual scale, and their gradient.
//
//   hat_b = (branch - mean_b) rstd_b,  u = hat_b w_post + b_post
//   out   = a residual + b gate u,     hat_r = (out - mean_r) rstd_r,  normed = hat_r w_pre + b_pre
//
//   e = d_normed w_pre,   D = d_out + rstd_r (e - mean(e) - hat_r mean(e hat_r))
//   d_residual = a D,     q = b gate D,   f = q w_post
//   d_branch = rstd_b (f - mean(f) - hat_b mean(f hat_b))
//   d_w_pre = sum d_normed hat_r, d_b_pre = sum d_normed, d_gate = sum b D u,
//   d_w_post = sum q hat_b, d_b_post = sum q                 (sums over the rows)
// (without the means of e and f for RMS).
//
// Each row is read once and written once.  A row belongs to a team of warps, 8 columns a thread, so that it stays in
// registers; a CTA holds as many teams as fit 16 warps, and each team takes a run of rows.  Rows past 4096 columns
// are shared by a cluster of CTAs, which exchange their sums.  Statistics are taken from the row in registers,
// squares around the mean.  The gradient recomputes `out` from residual and branch in fp32, as the forward
// pass had it before its rounding, and sums the vectors' gradients in registers over the team's run; teams, then
// CTAs, are joined in a fixed order.
//
// Rows arrive ahead of their use in a ring of stages: forward by asynchronous copies of single threads, each of which
// copies the columns that it will read itself, so that neither arrival nor reuse needs a barrier; in the gradient
// by bulk copies, a row and tensor each.  Arithmetic runs on pairs of columns (two fp32 operations an instruction).
//
// 32768 x 2048 bf16 with RMS: forward 90 us (537 MB, 5.9 TB/s), gradient 142 (805 MB, 5.7 TB/s).  HBM bounds
// neither alone: a warp has 270 and 330 instructions a row, at 0.7 and 0.5 of the issue rate, and a row's one (RMS
// forward: two) exchange between warps is latency that the gradient's 16 warps an SM, all that its registers allow, do
// not hide.  Before: sums by single columns with looked up forms took 404 and 622 instructions, 141 and 248 us.
#include <cuda_bf16.h>

#include <algorithm>
#include <atomic>
#include <initializer_list>
#include <type_traits>

#include "ops_internal.h"
#include "ops_ptx.cuh"

namespace mfsdp {
namespace ops {
namespace {

constexpr int kMaxWarps = 16;                 // of a CTA
constexpr int kMaxThreads = kMaxWarps * 32;
constexpr int kCols = 8;                      // columns of a thread
constexpr int kPairs = kCols / 2;
constexpr int kCtaCols = kMaxThreads * kCols; // columns that a CTA takes of a row
constexpr int kMaxCluster = MFSDP_MAX_NORM_DIM / kCtaCols;
// Of a tensor in a stage: 16 bytes a thread (fp32: twice), and room for the words that rows off 16-byte boundaries
// begin and end in, for each team.
template <bool kAligned>
constexpr int kChunk = kMaxThreads * 16 + (kAligned ? 0 : kMaxWarps * 32);
constexpr int kChunkBytes = kChunk<true>;
constexpr size_t kSharedBytes = 220 * 1024;

using ptx::add2;
using ptx::bits;
using ptx::both;
using ptx::fma2;
using ptx::mul2;

struct Cols {
  float2 p[kPairs];
  __device__ __forceinline__ void fill(float x) {
#pragma unroll
    for (int k = 0; k < kPairs; ++k) p[k] = both(x);
  }
  __device__ __forceinline__ float at(int i) const { return i & 1 ? p[i >> 1].y : p[i >> 1].x; }
  __device__ __forceinline__ void set(int i, float x) { (i & 1 ? p[i >> 1].y : p[i >> 1].x) = x; }
};

// ------------------------------------------------------------------- teams
// The sums that warps hand to each other, in two turns so that one barrier a sum is enough; places past a
// team's warps stay zero.
template <bool kMany>      // whether several values are summed at once
struct Exchange {
  float one[2][kMaxWarps * 4];
  float2 part[2][kMaxCluster][4];
};
template <>
struct Exchange<true> : Exchange<false> {
  float many[2][kMaxWarps * 4][8];
};

template <bool kAligned, bool kCluster, bool kMany>
struct Team {
  static constexpr bool kVectors = kAligned;
  int unit;          // its run of rows
  int id;            // in the CTA
  int tid;           // this thread in the team
  int warps, threads;
  int c0, end;       // columns [c0, end) of the row are this CTA's
  int parts;         // CTAs that share a row
  bool active;       // aligned rows: this thread has columns; others read the first ones and count for nothing
  int place;         // of the team in the exchange
  int turn;
  Exchange<kMany>* ex;

  __device__ __forceinline__ Team(int dim, int team_warps, int row_parts, int part_cols, Exchange<kMany>* exchange) {
    warps = team_warps;
    threads = warps * 32;
    id = threadIdx.x / threads;
    tid = threadIdx.x % threads;
    parts = row_parts;
    c0 = kCluster ? (int)ptx::cluster_ctarank() * part_cols : 0;
    end = kCluster ? min(dim, c0 + part_cols) : dim;
    unit = (int)(blockIdx.x / parts) * (int)(blockDim.x / threads) + id;
    active = c0 + tid * kCols < end;
    place = id * ((warps + 3) & ~3);
    turn = 0;
    ex = exchange;
    for (int k = threadIdx.x; k < (int)(sizeof(Exchange<kMany>) / 4); k += blockDim.x) reinterpret_cast<float*>(ex)[k] = 0.0f;
  }

  // The column of this thread's element i: 8 in a row where rows consist of 16-byte vectors, else single
  // ones, a warp's side by side.
  __device__ __forceinline__ int column(int i) const {
    return c0 + (kAligned ? (active ? tid * kCols : 0) + i : i * threads + tid);
  }
  __device__ __forceinline__ bool has(int i) const { return kAligned ? active : c0 + i * threads + tid < end; }

  __device__ __forceinline__ void meet() const {
    if (warps == 1) __syncwarp();
    else asm volatile("bar.sync %0, %1;" ::"r"(id + 1), "r"(threads) : "memory");
  }
  // The sums of the cluster's CTAs, in order.
  template <int kN>
  __device__ __forceinline__ void across(float2 (&v)[kN]) {
    if (tid < parts) {
      const uint32_t to = ptx::mapa_shared(ptx::smem_u32(&ex->part[turn][ptx::cluster_ctarank()][0]), tid);
#pragma unroll
      for (int i = 0; i < kN; ++i) ptx::st_shared_cluster_u64(to + 8 * i, bits(v[i]));
    }
    ptx::cluster_sync();
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      v[i] = ex->part[turn][0][i];
      for (int k = 1; k < parts; ++k) v[i] = add2(v[i], ex->part[turn][k][i]);
    }
  }

  // Sums over a row's threads, the same in each of them.
  __device__ __forceinline__ float sum(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    if (warps > 1) {
      float* const to = ex->one[turn] + place;
      if ((threadIdx.x & 31) == 0) to[tid >> 5] = v;
      meet();
      v = 0.0f;
      for (int k = 0; k < warps; k += 4) {
        const float4 q = *reinterpret_cast<const float4*>(to + k);
        v += (q.x + q.y) + (q.z + q.w);
      }
    } else {
      __syncwarp();                            // as the barrier does: what the team has read may be written over
    }
    if (kCluster) {
      float2 w[1] = {make_float2(v, 0.0f)};
      across(w);
      v = w[0].x;
    }
    turn ^= 1;
    return v;
  }
  // Of 4 or 8 values at once: each step of the exchange halves what a lane still has to add up.
  template <int kN>
  __device__ __forceinline__ void sum(float (&v)[kN]) {
    const int lane = threadIdx.x & 31;
    int o = 16;
#pragma unroll
    for (int half = kN / 2; half > 0; half >>= 1, o >>= 1) {
      const bool upper = lane & o;
#pragma unroll
      for (int i = 0; i < half; ++i) {
        const float give = upper ? v[i] : v[i + half];
        v[i] = (upper ? v[i + half] : v[i]) + __shfl_xor_sync(0xFFFFFFFFu, give, o);
      }
    }
    float x = v[0];                            // of value lane / (32 / kN)
#pragma unroll
    for (int r = 16 / kN; r > 0; r >>= 1) x += __shfl_xor_sync(0xFFFFFFFFu, x, r);
    float2 w[kN / 2];
    if (warps > 1) {
      float(*const to)[8] = ex->many[turn] + place;
      if (lane % (32 / kN) == 0) to[tid >> 5][lane / (32 / kN)] = x;
      meet();
#pragma unroll
      for (int i = 0; i < kN / 2; ++i) w[i] = make_float2(0.0f, 0.0f);
      for (int k = 0; k < warps; k += 4) {
#pragma unroll
        for (int i = 0; i < kN / 4; ++i) {
          const float4 p = *reinterpret_cast<const float4*>(&to[k][4 * i]);
          const float4 q = *reinterpret_cast<const float4*>(&to[k + 1][4 * i]);
          const float4 r = *reinterpret_cast<const float4*>(&to[k + 2][4 * i]);
          const float4 u = *reinterpret_cast<const float4*>(&to[k + 3][4 * i]);
          w[2 * i] = add2(w[2 * i], add2(add2(make_float2(p.x, p.y), make_float2(q.x, q.y)),
                                         add2(make_float2(r.x, r.y), make_float2(u.x, u.y))));
          w[2 * i + 1] = add2(w[2 * i + 1], add2(add2(make_float2(p.z, p.w), make_float2(q.z, q.w)),
                                                 add2(make_float2(r.z, r.w), make_float2(u.z, u.w))));
        }
      }
    } else {
      __syncwarp();
#pragma unroll
      for (int i = 0; i < kN / 2; ++i)
        w[i] = make_float2(__shfl_sync(0xFFFFFFFFu, x, 2 * i * (32 / kN)), __shfl_sync(0xFFFFFFFFu, x, (2 * i + 1) * (32 / kN)));
    }
    if (kCluster) across(w);
#pragma unroll
    for (int i = 0; i < kN; ++i) v[i] = i & 1 ? w[i >> 1].y : w[i >> 1].x;
    turn ^= 1;
  }
  // This thread's share of a sum over pairs.
  __device__ __forceinline__ float share(float2 v) const { return !kAligned || active ? v.x + v.y : 0.0f; }
  // Columns past the row's end, which a sum must not count (aligned rows: see share).
  __device__ __forceinline__ void clear_past(Cols& x) const {
    if constexpr (!kAligned) {
#pragma unroll
      for (int i = 0; i < kCols; ++i)
        if (!has(i)) x.set(i, 0.0f);
    }
  }
};

// An element type known when the kernel is compiled, or (kAny) when it runs.
constexpr int kF32 = 0, kBf16 = 1, kAny = 2;
template <int kType>
__device__ __forceinline__ bool is_bf16(int flag) { return kType == kAny ? flag != 0 : kType == kBf16; }

__device__ __forceinline__ float load_at(const void* p, int64_t i, bool bf16) {
  return bf16 ? __uint_as_float((uint32_t)static_cast<const uint16_t*>(p)[i] << 16) : static_cast<const float*>(p)[i];
}

__device__ __forceinline__ void widen(const uint4& q, Cols& x) {
  const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
  for (int k = 0; k < kPairs; ++k)
    x.p[k] = make_float2(__uint_as_float(w[k] << 16), __uint_as_float(w[k] & 0xFFFF0000u));
}
__device__ __forceinline__ void as_floats(const uint4& lo, const uint4& hi, Cols& x) {
  x.p[0] = make_float2(__uint_as_float(lo.x), __uint_as_float(lo.y));
  x.p[1] = make_float2(__uint_as_float(lo.z), __uint_as_float(lo.w));
  x.p[2] = make_float2(__uint_as_float(hi.x), __uint_as_float(hi.y));
  x.p[3] = make_float2(__uint_as_float(hi.z), __uint_as_float(hi.w));
}

// This thread's columns of a vector that starts at element `at`; `none` where it has none, or there is no vector.
template <bool kAligned, bool kCluster, bool kMany>
__device__ __forceinline__ void load_vector(const void* p, int64_t at, bool bf16, const Team<kAligned, kCluster, kMany>& t,
                                            float none, Cols& x) {
  x.fill(none);
  if (p == nullptr) return;
  if constexpr (kAligned) {
    const uint4* q = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(p) + (at + t.column(0)) * (bf16 ? 2 : 4));
    if (bf16) widen(q[0], x);
    else as_floats(q[0], q[1], x);
  } else {
#pragma unroll
    for (int i = 0; i < kCols; ++i)
      if (t.has(i)) x.set(i, load_at(p, at + t.column(i), bf16));
  }
}

// Vectors kept in shared memory, where a warp reads them without conflicts.
template <bool kAligned, bool kCluster, bool kMany>
__device__ __forceinline__ void keep(float* to, const Cols& x, const Team<kAligned, kCluster, kMany>& t) {
#pragma unroll
  for (int i = 0; i < kCols; ++i) to[kAligned ? ((i >> 2) * t.threads + t.tid) * 4 + (i & 3) : i * t.threads + t.tid] = x.at(i);
}
template <bool kAligned, bool kCluster, bool kMany>
__device__ __forceinline__ void kept(const float* from, const Team<kAligned, kCluster, kMany>& t, Cols& x) {
  if constexpr (kAligned) {
    const float4 lo = reinterpret_cast<const float4*>(from)[t.tid];
    const float4 hi = reinterpret_cast<const float4*>(from)[t.threads + t.tid];
    x.p[0] = make_float2(lo.x, lo.y);
    x.p[1] = make_float2(lo.z, lo.w);
    x.p[2] = make_float2(hi.x, hi.y);
    x.p[3] = make_float2(hi.z, hi.w);
  } else {
#pragma unroll
    for (int i = 0; i < kCols; ++i) x.set(i, from[i * t.threads + t.tid]);
  }
}

// --------------------------------------------------------------------- rows
// A tensor's rows as a thread goes over them: its first column in the present row (aligned), or the
// row's start.
template <int kType, bool kAligned>
struct Rows {
  uint8_t* p;
  const RowStep& step;   // and whether the type is bf16 where it is not known: the kernel's parameters, which
  const int32_t& flag;   // need no registers
  template <typename T>
  __device__ __forceinline__ Rows(const void* base, const RowStep& bytes, const int32_t& bf16, int64_t row, const T& t)
      : step(bytes), flag(bf16) {
    p = base == nullptr ? nullptr
                        : static_cast<uint8_t*>(const_cast<void*>(base)) + row * step.row +
                              (kAligned ? t.column(0) * (is_bf16<kType>(bf16) ? 2 : 4) : 0);
  }
  __device__ __forceinline__ bool bf16() const { return is_bf16<kType>(flag); }
  __device__ __forceinline__ int chunks() const { return bf16() ? 1 : 2; }
  __device__ __forceinline__ void next() { p += step.next; }
  template <typename T>
  __device__ __forceinline__ void store(const Cols& x, const T& t) const {
    if constexpr (kAligned) {
      if (!t.active) return;
      uint4* q = reinterpret_cast<uint4*>(p);
      if (bf16()) {
        __nv_bfloat162 h[kPairs];
#pragma unroll
        for (int k = 0; k < kPairs; ++k) h[k] = __float22bfloat162_rn(x.p[k]);
        __stcs(q, *reinterpret_cast<const uint4*>(h));
      } else {
        __stcs(q, make_uint4(__float_as_uint(x.p[0].x), __float_as_uint(x.p[0].y), __float_as_uint(x.p[1].x),
                             __float_as_uint(x.p[1].y)));
        __stcs(q + 1, make_uint4(__float_as_uint(x.p[2].x), __float_as_uint(x.p[2].y), __float_as_uint(x.p[3].x),
                                 __float_as_uint(x.p[3].y)));
      }
    } else {
#pragma unroll
      for (int i = 0; i < kCols; ++i) {
        if (!t.has(i)) continue;
        const int c = t.column(i);
        if (bf16()) reinterpret_cast<__nv_bfloat16*>(p)[c] = __float2bfloat16_rn(x.at(i));
        else reinterpret_cast<float*>(p)[c] = x.at(i);
      }
    }
  }
};

// The 16-byte words that hold this CTA's columns of a row.
struct Words {
  const uint8_t* from;
  uint32_t bytes;
  template <typename T>
  __device__ __forceinline__ Words(const void* p, int64_t offset, int size, const T& t) {
    from = static_cast<const uint8_t*>(p) + offset + t.c0 * size;
    const uint32_t o = (uint32_t)reinterpret_cast<uintptr_t>(from) & 15;
    from -= o;
    bytes = (o + (t.end - t.c0) * size + 15) & ~15u;
  }
};

// Rows on their way: a ring of stages, in which a thread has 16 bytes (bf16) or twice 16 (fp32) of
// each tensor.  The copies run kStages rows ahead of the row in hand.  A row off 16-byte boundaries comes as the words
// that hold it, dealt out over the team, which meets before it reads them; the first and last rows of a tensor, whose
// words may reach past it, do not come by the ring.
template <int kStages, bool kAligned>
struct Ring {
  uint32_t at;                // the present row's stage
  uint32_t first, past;       // of the ring
  uint32_t stage_bytes;
  __device__ __forceinline__ Ring(const void* base, int chunks) {
    stage_bytes = chunks * kChunk<kAligned>;
    at = first = ptx::smem_u32(base) + (kAligned ? threadIdx.x * 16 : 0);
    past = first + kStages * stage_bytes;
  }
  __device__ __forceinline__ void next() {
    at += stage_bytes;
    if (at == past) at = first;
  }
  template <typename R>
  __device__ __forceinline__ void fetch(R& rows, bool there, int chunk) const {
    if (!there) return;
    const uint32_t to = at + chunk * kChunkBytes;
    ptx::copy_async_16(to, rows.p);
    if (!rows.bf16()) ptx::copy_async_16(to + kChunkBytes, rows.p + 16);
    rows.next();
  }
  template <typename T>
  __device__ __forceinline__ void fetch_words(const void* p, int64_t offset, int chunk, int size, const T& t) const {
    if (p == nullptr) return;
    const Words w(p, offset, size, t);
    const uint32_t to = at + chunk * kChunk<kAligned> + t.id * (t.threads * kCols * size + 32);
    for (uint32_t k = t.tid * 16; k < w.bytes; k += t.threads * 16) ptx::copy_async_16(to + k, w.from + k);
  }
  __device__ __forceinline__ void wait() const { ptx::copy_async_wait<kStages - 1>(); }
  __device__ __forceinline__ uint32_t mine(int chunk, bool) const { return at + chunk * kChunkBytes; }
  static __device__ constexpr uint32_t second() { return kChunkBytes; }      // from a thread's first 16 bytes to its others
};

// The same by bulk copies, one a team and tensor, issued by the team's first thread once the team has met in an
// earlier row's sums.  (A copy for each warp's columns keeps the copy engine busy without need: 174 us against 148,
// 32768 x 2048.)
constexpr uint64_t kWaitNs = 2000000000;
template <int kStages, bool kAligned>
struct BulkRing {
  uint32_t at;                // of the present stage
  uint32_t bar;               // its barrier, this team's
  int stage;
  uint32_t phase;
  bool broken;                // a wait gave up: no more copies, and short waits for those on their way
  const uint32_t first, stage_bytes, bar_first;
  template <typename T>
  __device__ __forceinline__ BulkRing(const void* base, int chunks, uint64_t (*bars)[kMaxWarps], const T& t)
      : first(ptx::smem_u32(base)), stage_bytes(chunks * kChunk<kAligned>), bar_first(ptx::smem_u32(&bars[0][t.id])) {
    at = first;
    bar = bar_first;
    stage = 0;
    phase = 0;
    broken = false;
    if (t.tid == 0) {
#pragma unroll
      for (int k = 0; k < kStages; ++k) ptx::mbar_init(bar + k * kMaxWarps * 8, 1);
      ptx::fence_barrier_init();
      ptx::fence_proxy_async_smem();
    }
  }
  __device__ __forceinline__ void next() {
    at += stage_bytes;
    bar += kMaxWarps * 8;
    if (++stage == kStages) {
      stage = 0;
      at = first;
      bar = bar_first;
      phase ^= 1;
    }
  }
  // The first thread's: a row of a tensor.
  __device__ __forceinline__ void fetch(const void* p, bool there, int64_t offset, int chunk, int bytes_a_thread,
                                        uint32_t bytes) const {
    if (!there) return;
    ptx::bulk_load(at + chunk * kChunkBytes + threadIdx.x * bytes_a_thread, static_cast<const uint8_t*>(p) + offset, bytes, bar);
  }
  template <typename T>
  __device__ __forceinline__ void fetch_words(const void* p, const Words& w, int chunk, int size, const T& t) const {
    if (p != nullptr)
      ptx::bulk_load(at + chunk * kChunk<kAligned> + t.id * (t.threads * kCols * size + 32), w.from, w.bytes, bar);
  }
  __device__ __forceinline__ void wait(int32_t* status) {
    if (ptx::mbar_wait(bar, phase, broken ? kWaitNs / 2000 : kWaitNs) || broken) return;
    broken = true;
    atomicCAS(status, 0, 1);
  }
  __device__ __forceinline__ uint32_t mine(int chunk, bool bf16) const {
    return at + chunk * kChunkBytes + threadIdx.x * (bf16 ? 16 : 32);
  }
  static __device__ constexpr uint32_t second() { return 16; }
};

__device__ __forceinline__ uint16_t ld_shared_2(uint32_t addr) {
  uint16_t x;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(x) : "r"(addr) : "memory");
  return x;
}
__device__ __forceinline__ float ld_shared_4(uint32_t addr) {
  float x;
  asm volatile("ld.shared.f32 %0, [%1];" : "=f"(x) : "r"(addr) : "memory");
  return x;
}
__device__ __forceinline__ uint4 ld_shared_16(uint32_t addr) {
  uint4 q;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(q.x), "=r"(q.y), "=r"(q.z), "=r"(q.w) : "r"(addr) : "memory");
  return q;
}

// The present row's columns: from the ring, or (rows off 16-byte boundaries that are not on it) from memory.  No
// tensor: zeros.
template <bool kAligned, typename G, typename R, typename T>
__device__ __forceinline__ void take(const G& ring, R& rows, bool there, int chunk, const T& t, bool ringed, Cols& x) {
  if (!there) {
    x.fill(0.0f);
    return;
  }
  if constexpr (kAligned) {
    const uint32_t from = ring.mine(chunk, rows.bf16());
    const uint4 lo = ld_shared_16(from);
    if (rows.bf16()) widen(lo, x);
    else as_floats(lo, ld_shared_16(from + G::second()), x);
  } else {
    x.fill(0.0f);
    const int size = rows.bf16() ? 2 : 4;
    const uint32_t o = ((uint32_t)reinterpret_cast<uintptr_t>(rows.p) + t.c0 * size) & 15;
    const uint32_t from = ring.at + chunk * kChunk<false> + t.id * (t.threads * kCols * size + 32) + o + t.tid * size;
    if (!ringed) {
#pragma unroll
      for (int i = 0; i < kCols; ++i)
        if (t.has(i)) x.set(i, load_at(rows.p, t.column(i), rows.bf16()));
    } else if (rows.bf16()) {
#pragma unroll
      for (int i = 0; i < kCols; ++i)
        if (t.has(i)) x.set(i, __uint_as_float((uint32_t)ld_shared_2(from + i * t.threads * 2) << 16));
    } else {
#pragma unroll
      for (int i = 0; i < kCols; ++i)
        if (t.has(i)) x.set(i, ld_shared_4(from + i * t.threads * 4));
    }
    rows.next();
  }
}

// What a call has, known when the kernel is compiled, or (kMixed) looked up in every row.  The known forms have every
// tensor of rows that goes with them and the norms' weights, and with LAYER their biases:
//   kRms, kLayer             a block between two norms of one kind
//   kAddRms, kAddLayer       a block without a norm after it
//   kFirstRms, kFirstLayer   no block before
// Each looked up fact costs a warp some four instructions a row (forward: 404 in all, 271 in a known form).
enum Form { kMixed, kRms, kLayer, kAddRms, kAddLayer, kFirstRms, kFirstLayer };
template <Form kForm>
struct Known {
  static constexpr bool kAll = kForm != kMixed, kPost = kForm == kRms || kForm == kLayer;
  static constexpr bool kBlock = kPost || kForm == kAddRms || kForm == kAddLayer;
  static constexpr bool kBias = kForm == kLayer || kForm == kAddLayer || kForm == kFirstLayer;
  // rows that every form has, and the weight of the norm before the next block
  static __device__ __forceinline__ bool has(const void* p) { return kAll || p != nullptr; }
  static __device__ __forceinline__ bool block(const void* p) { return kAll ? kBlock : p != nullptr; }
  static __device__ __forceinline__ bool post_weight(const void* p) { return kAll ? kPost : p != nullptr; }
  static __device__ __forceinline__ bool post_bias(const void* p) { return kAll ? kForm == kLayer : p != nullptr; }
  static __device__ __forceinline__ bool pre_bias(const void* p) { return kAll ? kBias : p != nullptr; }
  static __device__ __forceinline__ int post_kind(int given) {
    return !kAll ? given : kForm == kRms ? MFSDP_NORM_RMS : kForm == kLayer ? MFSDP_NORM_LAYER : MFSDP_NORM_NONE;
  }
  static __device__ __forceinline__ int pre_kind(int given) {
    return !kAll ? given : kBias ? MFSDP_NORM_LAYER : MFSDP_NORM_RMS;
  }
};

struct NormPlan {
  int warps;         // of a team
  int units;         // runs of rows, one a team
  int stride;        // rows from one of a run to its next: 1, or as many as there are runs
  int parts;         // CTAs that share a row (then a CTA is a team)
  int part_cols;
  int margin;        // rows off 16-byte boundaries: so many first and last ones do not come by the ring
};

// First row of a run (there are no more runs than rows; teams past them have none).
__device__ __forceinline__ int run_start(int unit, int64_t n, int units) {
  return (int)(unit < units ? unit * n / units : n);
}

// Mean and 1/sqrt of a row in registers (rows not made of vectors: zeros past its end).
template <typename T>
__device__ __forceinline__ float2 statistics(const Cols& x, int kind, const NormArgs& a, T& t) {
  float mean = 0.0f;
  float2 s;
  if (kind == MFSDP_NORM_LAYER) {
    mean = t.sum(t.share(add2(add2(x.p[0], x.p[1]), add2(x.p[2], x.p[3])))) * a.inv_dim;
    Cols d;
#pragma unroll
    for (int k = 0; k < kPairs; ++k) d.p[k] = add2(x.p[k], both(-mean));
    t.clear_past(d);
    s = mul2(d.p[0], d.p[0]);
#pragma unroll
    for (int k = 1; k < kPairs; ++k) s = fma2(d.p[k], d.p[k], s);
  } else {
    s = mul2(x.p[0], x.p[0]);
#pragma unroll
    for (int k = 1; k < kPairs; ++k) s = fma2(x.p[k], x.p[k], s);
  }
  return make_float2(mean, rsqrtf(fmaf(t.sum(t.share(s)), a.inv_dim, a.eps)));
}

// x becomes (x - mean) rstd.  The difference first: a row may lie close to its mean.
__device__ __forceinline__ void standardise(Cols& x, int kind, float mean, float rstd) {
  if (kind == MFSDP_NORM_LAYER) {
#pragma unroll
    for (int k = 0; k < kPairs; ++k) x.p[k] = add2(x.p[k], both(-mean));
  }
#pragma unroll
  for (int k = 0; k < kPairs; ++k) x.p[k] = mul2(x.p[k], both(rstd));
}

__device__ __forceinline__ float2 total(const Cols& x) { return add2(add2(x.p[0], x.p[1]), add2(x.p[2], x.p[3])); }
__device__ __forceinline__ float2 dot(const Cols& x, const Cols& y) {
  float2 s = mul2(x.p[0], y.p[0]);
#pragma unroll
  for (int k = 1; k < kPairs; ++k) s = fma2(x.p[k], y.p[k], s);
  return s;
}

// x times a weight, x plus a bias, where there is one.
template <typename T>
__device__ __forceinline__ void scale_by(Cols& x, bool there, const float* kept_w, const T& t) {
  if (!there) return;
  Cols v;
  kept(kept_w, t, v);
#pragma unroll
  for (int k = 0; k < kPairs; ++k) x.p[k] = mul2(x.p[k], v.p[k]);
}
template <typename T>
__device__ __forceinline__ void shift_by(Cols& x, bool there, const float* kept_b, const T& t) {
  if (!there) return;
  Cols v;
  kept(kept_b, t, v);
#pragma unroll
  for (int k = 0; k < kPairs; ++k) x.p[k] = add2(x.p[k], v.p[k]);
}

// ----------------------------------------------------------------- forward
constexpr int kForwardStages = 2;

template <Form kForm, bool kAligned, bool kCluster, int kR, int kB>
__global__ void __launch_bounds__(kMaxThreads, 2) norm_kernel(const __grid_constant__ NormArgs a, const NormPlan plan) {
  extern __shared__ __align__(16) uint8_t shared[];
  __shared__ __align__(16) Exchange<false> exchange;
  using T = Team<kAligned, kCluster, false>;
  using K = Known<kForm>;
  T t(a.dim, plan.warps, plan.parts, plan.part_cols, &exchange);
  float* const w_post = reinterpret_cast<float*>(shared);
  const int vector = t.threads * kCols;
  float* const b_post = w_post + (a.w_post ? vector : 0);
  float* const w_pre = b_post + (a.b_post ? vector : 0);
  float* const b_pre = w_pre + (a.w_pre ? vector : 0);
  float* const end = b_pre + (a.b_pre ? vector : 0);
  const bool apart = plan.stride > 1;
  const int r0 = apart ? (t.unit < plan.units ? t.unit : (int)a.n) : run_start(t.unit, a.n, plan.units);
  const int r1 = apart ? (int)a.n : run_start(t.unit + 1, a.n, plan.units);
  Rows<kR, kAligned> residual(a.residual, a.residual_step, a.r_bf16, r0, t), out(a.out, a.out_step, a.r_bf16, r0, t);
  Rows<kB, kAligned> branch(a.branch, a.branch_step, a.b_bf16, r0, t), normed(a.normed, a.normed_step, a.b_bf16, r0, t);
  const int bc = residual.chunks();            // of branch in a stage
  Ring<kForwardStages, kAligned> ring(end, bc + branch.chunks());
  const auto ringed = [&](int row) { return kAligned || (row >= plan.margin && row < a.n - plan.margin); };
  const auto fetch = [&](int row) {
    if (row < r1 && ringed(row)) {
      if constexpr (kAligned) {
        ring.fetch(residual, true, 0);
        ring.fetch(branch, K::block(a.branch), bc);
      } else {
        ring.fetch_words(a.residual, row * a.residual_step.row, 0, a.r_bf16 ? 2 : 4, t);
        ring.fetch_words(a.branch, row * a.branch_step.row, bc, a.b_bf16 ? 2 : 4, t);
      }
    }
    ptx::copy_async_commit();
    ring.next();
  };
#pragma unroll
  for (int k = 0; k < kForwardStages; ++k) fetch(r0 + k * plan.stride);
  if (t.id == 0) {
    Cols v;
    const auto keep_one = [&](float* to, const void* p) {
      if (p == nullptr) return;
      load_vector(p, 0, a.w_bf16, t, 0.0f, v);
      keep(to, v, t);
    };
    keep_one(w_post, a.w_post);
    keep_one(b_post, a.b_post);
    keep_one(w_pre, a.w_pre);
    keep_one(b_pre, a.b_pre);
  }
  __syncthreads();
  if (kCluster) ptx::cluster_sync();
  Cols gate;
  int group_end = r0;
  for (int row = r0; row < r1; row += plan.stride) {
    ring.wait();
    if (!kAligned) t.meet();                   // all threads' words are there
    Cols x, y;
    take<kAligned>(ring, residual, true, 0, t, ringed(row), x);
    float4 st = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (K::block(a.branch)) {
      take<kAligned>(ring, branch, true, bc, t, ringed(row), y);
      if (row == group_end) {
        const int64_t g = a.gate ? (uint32_t)row / (uint32_t)a.gate_rows : 0;
        load_vector(a.gate, g * a.dim, a.w_bf16, t, 1.0f, gate);
#pragma unroll
        for (int k = 0; k < kPairs; ++k) gate.p[k] = mul2(gate.p[k], both(a.branch_scale));
        group_end = a.gate ? (int)min((int64_t)r1, (g + 1) * a.gate_rows) : r1;
      }
      if (K::post_kind(a.post) != MFSDP_NORM_NONE) {
        const float2 s = statistics(y, K::post_kind(a.post), a, t);
        st.x = s.x;
        st.y = s.y;
        standardise(y, K::post_kind(a.post), s.x, s.y);
        scale_by(y, K::post_weight(a.w_post), w_post, t);
        shift_by(y, K::post_bias(a.b_post), b_post, t);
      }
#pragma unroll
      for (int k = 0; k < kPairs; ++k) x.p[k] = fma2(both(a.residual_scale), x.p[k], mul2(gate.p[k], y.p[k]));
      t.clear_past(x);
    }
    if (!kAligned) t.meet();
    fetch(row + kForwardStages * plan.stride);               // this row's stage is in registers
    if (K::block(a.out)) {
      out.store(x, t);
      out.next();
    }
    if (K::pre_kind(a.pre) != MFSDP_NORM_NONE) {
      const float2 s = statistics(x, K::pre_kind(a.pre), a, t);
      st.z = s.x;
      st.w = s.y;
      if (K::has(a.normed)) {
        standardise(x, K::pre_kind(a.pre), s.x, s.y);
        scale_by(x, K::has(a.w_pre), w_pre, t);
        shift_by(x, K::pre_bias(a.b_pre), b_pre, t);
        normed.store(x, t);
        normed.next();
      }
    }
    if (a.stats && t.tid == 0 && t.c0 == 0) a.stats[row] = st;
  }
}

// ------------------------------------------------------------------ gradient
// Vectors whose gradients are summed, in the order of the parts: and a gate that all rows share.
enum { kSumWPost, kSumBPost, kSumWPre, kSumBPre, kSumGate };
static_assert(kSumGate + 1 == kNormParts, "a part has these");

__device__ __forceinline__ void put(float* p, float x, int accumulate) { *p = accumulate ? *p + x : x; }

// This thread's columns of a vector's gradient that starts at `p`, or of a part of one.
template <typename T>
__device__ __forceinline__ void put_vector(float* p, const Cols& x, int accumulate, const T& t) {
  if constexpr (T::kVectors) {
    if (!t.active) return;
    float4* q = reinterpret_cast<float4*>(p + t.column(0));
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float4 v = make_float4(x.p[2 * h].x, x.p[2 * h].y, x.p[2 * h + 1].x, x.p[2 * h + 1].y);
      if (accumulate) {
        const float4 o = q[h];
        v = make_float4(o.x + v.x, o.y + v.y, o.z + v.z, o.w + v.w);
      }
      q[h] = v;
    }
  } else {
#pragma unroll
    for (int i = 0; i < kCols; ++i)
      if (t.has(i)) put(p + t.column(i), x.at(i), accumulate);
  }
}

// A place of shared memory for 8 numbers of each thread.
struct Aside {
  float4* at;
  __device__ __forceinline__ explicit Aside(float* base) : at(reinterpret_cast<float4*>(base) + threadIdx.x) {}
  __device__ __forceinline__ void put(const Cols& x) const {
    at[0] = make_float4(x.p[0].x, x.p[0].y, x.p[1].x, x.p[1].y);
    at[kMaxThreads] = make_float4(x.p[2].x, x.p[2].y, x.p[3].x, x.p[3].y);
  }
  __device__ __forceinline__ void get(Cols& x) const {
    const float4 lo = at[0], hi = at[kMaxThreads];
    x.p[0] = make_float2(lo.x, lo.y);
    x.p[1] = make_float2(lo.z, lo.w);
    x.p[2] = make_float2(hi.x, hi.y);
    x.p[3] = make_float2(hi.z, hi.w);
  }
};
constexpr int kAsideFloats = kMaxThreads * kCols;
// Those of the gradient's kernels: gb, where there can be a bias, and with all sums two of them.
template <Form kForm, int kSums>
constexpr int kAsides = kForm != kMixed && kForm != kLayer ? 0 : kSums == 2 ? 3 : 1;
// Stages of the gradient's ring: what leaves room for those and a vector beside it.
template <Form kForm, int kR, int kB, int kSums>
constexpr int kGradStages =
    std::min(3, (int)((kSharedBytes - (1 + kAsides<kForm, kSums>) * kAsideFloats * 4) /
                      (kChunk<false> * (2 * (kR == kBf16 ? 1 : 2) + 2 * (kB == kBf16 ? 1 : 2)))));

// Adds up what the CTA's teams left of the wanted vectors.  By itself, so that the rows' loop has the registers.
template <bool kAligned>
__device__ __noinline__ void join_teams(const float* left, float* part, uint32_t wanted, int teams, int threads, int dim) {
  for (int job = threadIdx.x; job < kNormParts * threads; job += blockDim.x) {
    const int which = job / threads, tid = job - which * threads;
    if (!(wanted >> which & 1)) continue;
    const float4* from = reinterpret_cast<const float4*>(left + which * kAsideFloats) + tid;
    float4 lo = from[0], hi = from[kMaxThreads];
    for (int k = 1; k < teams; ++k) {
      from += threads;
      const float4 u = from[0], v = from[kMaxThreads];
      lo = make_float4(lo.x + u.x, lo.y + u.y, lo.z + u.z, lo.w + u.w);
      hi = make_float4(hi.x + v.x, hi.y + v.y, hi.z + v.z, hi.w + v.w);
    }
    float* to = part + which * dim;
    if constexpr (kAligned) {
      if (tid * kCols >= dim) continue;
      reinterpret_cast<float4*>(to + tid * kCols)[0] = lo;
      reinterpret_cast<float4*>(to + tid * kCols)[1] = hi;
    } else {
      const float x[kCols] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
#pragma unroll
      for (int i = 0; i < kCols; ++i)
        if (i * threads + tid < dim) to[i * threads + tid] = x[i];
    }
  }
}

// The rows of a group share the gate, so all that the block's side needs of them is P = sum D hat_b and
// R = sum D: d_gate = b (w_post P + b_post R), and a group adds b gate P to d_w_post and b gate R to
// d_b_post.  The row itself needs only the products gw = b gate w_post and gb = b gate b_post.
// kSums: 0 rows only, 1 without R and d_b_pre, 2 all.
template <Form kForm, bool kAligned, bool kCluster, int kR, int kB, int kSums>
__global__ void __launch_bounds__(kMaxThreads, 1) norm_grad_kernel(const __grid_constant__ NormGradArgs g,
                                                                   const NormPlan plan) {
  extern __shared__ __align__(16) uint8_t shared[];
  __shared__ __align__(16) Exchange<true> exchange;
  const NormArgs& a = g.f;
  using T = Team<kAligned, kCluster, true>;
  using K = Known<kForm>;
  constexpr bool kSumsR = kSums == 2 && (kForm == kMixed || kForm == kLayer);      // R, and d_b_post
  T t(a.dim, plan.warps, plan.parts, plan.part_cols, &exchange);
  float* const w_pre = reinterpret_cast<float*>(shared);
  // Beside the sums there is no room in registers for gb and the two sums that only a group's end changes.
  float* const places = w_pre + (a.w_pre ? t.threads * kCols : 0);
  const Aside gb_aside(places), wpost_aside(places + kAsideFloats), bpost_aside(places + 2 * kAsideFloats);
  float* const end = places + kAsides<kForm, kSums> * kAsideFloats;
  const bool apart = plan.stride > 1;
  const int r0 = apart ? (t.unit < plan.units ? t.unit : (int)a.n) : run_start(t.unit, a.n, plan.units);
  const int r1 = apart ? (int)a.n : run_start(t.unit + 1, a.n, plan.units);
  // Where rows are made of vectors they come by the ring, and these pointers are not used.
  Rows<kR, kAligned> residual(a.residual, a.residual_step, a.r_bf16, r0, t), d_out(g.d_out, g.d_out_step, a.r_bf16, r0, t),
      d_residual(g.d_residual, g.d_residual_step, a.r_bf16, r0, t);
  Rows<kB, kAligned> branch(a.branch, a.branch_step, a.b_bf16, r0, t),
      d_normed(g.d_normed, g.d_normed_step, a.b_bf16, r0, t), d_branch(g.d_branch, g.d_branch_step, a.b_bf16, r0, t);
  const int rc = residual.chunks(), bc = branch.chunks();
  constexpr int kStages = kGradStages<kForm, kR, kB, kSums>;
  __shared__ __align__(8) uint64_t bars[kStages][kMaxWarps];
  __shared__ __align__(16) float4 row_stats[kStages][kMaxWarps];       // of a team
  BulkRing<kStages, kAligned> ring(end, 2 * rc + 2 * bc, bars, t);
  const auto ringed = [&](int row) { return kAligned || (row >= plan.margin && row < a.n - plan.margin); };
  // Fills the present stage and goes on to the next.
  const auto fetch = [&](int row) {
    if (row < r1 && t.tid == 0 && !ring.broken && !ringed(row)) {
      ptx::mbar_arrive(ring.bar);              // nothing comes: the stage's phases go on all the same
    } else if (row < r1 && t.tid == 0 && !ring.broken) {
      const int r_size = a.r_bf16 ? 2 : 4, b_size = a.b_bf16 ? 2 : 4;
      if constexpr (!kAligned) {
        const Words w0(a.residual, row * a.residual_step.row, r_size, t), w1(g.d_out, row * g.d_out_step.row, r_size, t),
            w2(a.branch, row * a.branch_step.row, b_size, t), w3(g.d_normed, row * g.d_normed_step.row, b_size, t);
        ptx::mbar_arrive_expect_tx(ring.bar, 16 + w0.bytes + (g.d_out ? w1.bytes : 0) + (a.branch ? w2.bytes : 0) +
                                                 (g.d_normed ? w3.bytes : 0));
        ptx::bulk_load(ptx::smem_u32(&row_stats[ring.stage][t.id]), g.stats + row, 16, ring.bar);
        ring.fetch_words(a.residual, w0, 0, r_size, t);
        ring.fetch_words(g.d_out, w1, rc, r_size, t);
        ring.fetch_words(a.branch, w2, 2 * rc, b_size, t);
        ring.fetch_words(g.d_normed, w3, 2 * rc + bc, b_size, t);
      } else {
        const uint32_t r_bytes = (t.end - t.c0) * r_size, b_bytes = (t.end - t.c0) * b_size;
        const int64_t r_at = t.c0 * r_size, b_at = t.c0 * b_size;
        ptx::mbar_arrive_expect_tx(ring.bar, 16 + r_bytes * (1 + K::has(g.d_out)) +
                                                 b_bytes * (K::block(a.branch) + K::has(g.d_normed)));
        ptx::bulk_load(ptx::smem_u32(&row_stats[ring.stage][t.id]), g.stats + row, 16, ring.bar);
        ring.fetch(a.residual, true, row * a.residual_step.row + r_at, 0, 8 * r_size, r_bytes);
        ring.fetch(g.d_out, K::has(g.d_out), row * g.d_out_step.row + r_at, rc, 8 * r_size, r_bytes);
        ring.fetch(a.branch, K::block(a.branch), row * a.branch_step.row + b_at, 2 * rc, 8 * b_size, b_bytes);
        ring.fetch(g.d_normed, K::has(g.d_normed), row * g.d_normed_step.row + b_at, 2 * rc + bc, 8 * b_size, b_bytes);
      }
    }
    ring.next();
  };
  if (blockIdx.x == 0 && threadIdx.x == 0) *g.status = 0;
#pragma unroll
  for (int k = 0; k < kStages; ++k) fetch(r0 + k * plan.stride);
  ring.phase = 0;
  Cols s_p, s_r, s_wpre, s_bpre, s_wpost, gw;
  s_p.fill(0.0f);
  s_r.fill(0.0f);
  s_wpre.fill(0.0f);
  s_bpre.fill(0.0f);
  s_wpost.fill(0.0f);
  if (t.id == 0 && a.w_pre) {
    load_vector(a.w_pre, 0, a.w_bf16, t, 0.0f, gw);
    keep(w_pre, gw, t);
  }
  if (kSumsR) {
    wpost_aside.put(s_p);
    bpost_aside.put(s_p);
  }
  __syncthreads();
  if (kCluster) ptx::cluster_sync();
  const int post_kind = K::post_kind(a.post), pre_kind = K::pre_kind(a.pre);
  const bool post = post_kind != MFSDP_NORM_NONE, pre = pre_kind != MFSDP_NORM_NONE && K::has(g.d_normed);
  const bool one_gate = a.gate_rows >= a.n;
  const float d_scale = K::block(a.branch) ? a.residual_scale : 1.0f;
  int group = 0, group_end = r0;
  // Takes the present group's sums to where they belong.
  const auto close_group = [&]() {
    Cols v, w;
    load_vector(a.gate, (int64_t)group * a.dim, a.w_bf16, t, 1.0f, v);
#pragma unroll
    for (int k = 0; k < kPairs; ++k) v.p[k] = mul2(v.p[k], both(a.branch_scale));
    if (kSumsR) wpost_aside.get(s_wpost);
#pragma unroll
    for (int k = 0; k < kPairs; ++k) s_wpost.p[k] = fma2(v.p[k], s_p.p[k], s_wpost.p[k]);
    if (kSumsR) {
      wpost_aside.put(s_wpost);
      bpost_aside.get(w);
#pragma unroll
      for (int k = 0; k < kPairs; ++k) w.p[k] = fma2(v.p[k], s_r.p[k], w.p[k]);
      bpost_aside.put(w);
    }
    if (!g.d_gate) {
      s_p.fill(0.0f);
      s_r.fill(0.0f);
      return;
    }
    load_vector(post ? a.w_post : nullptr, 0, a.w_bf16, t, 1.0f, w);
#pragma unroll
    for (int k = 0; k < kPairs; ++k) s_p.p[k] = mul2(s_p.p[k], w.p[k]);
    if (kSumsR) {
      load_vector(post ? a.b_post : nullptr, 0, a.w_bf16, t, 0.0f, w);
#pragma unroll
      for (int k = 0; k < kPairs; ++k) s_p.p[k] = fma2(s_r.p[k], w.p[k], s_p.p[k]);
    }
    if (one_gate) return;                      // joined with the other runs' below
    const int64_t first = (int64_t)group * a.gate_rows;
    const int side = first < r0 ? 0 : group_end > r1 ? 1 : 2;
    float* const to = side == 2 ? g.d_gate + (int64_t)group * a.dim : g.gate_parts + ((int64_t)t.unit * 2 + side) * a.dim;
#pragma unroll
    for (int k = 0; k < kPairs; ++k) s_p.p[k] = mul2(s_p.p[k], both(a.branch_scale));
    put_vector(to, s_p, side == 2 && g.accumulate, t);
    s_p.fill(0.0f);
    s_r.fill(0.0f);
  };
  for (int row = r0; row < r1; row += plan.stride) {
    float4 st;
    if (ringed(row)) {
      ring.wait(g.status);
      st = row_stats[ring.stage][t.id];
    } else {
      st = g.stats[row];
    }
    if (K::block(a.branch) && row == group_end) {
      Cols v;
      group = a.gate ? (int)((uint32_t)row / (uint32_t)a.gate_rows) : 0;
      load_vector(a.gate, (int64_t)group * a.dim, a.w_bf16, t, 1.0f, v);
#pragma unroll
      for (int k = 0; k < kPairs; ++k) v.p[k] = mul2(v.p[k], both(a.branch_scale));
      load_vector(post ? a.w_post : nullptr, 0, a.w_bf16, t, 1.0f, gw);
#pragma unroll
      for (int k = 0; k < kPairs; ++k) gw.p[k] = mul2(gw.p[k], v.p[k]);
      t.clear_past(gw);
      if (post && K::post_bias(a.b_post)) {
        Cols b;
        load_vector(a.b_post, 0, a.w_bf16, t, 0.0f, b);
#pragma unroll
        for (int k = 0; k < kPairs; ++k) b.p[k] = mul2(b.p[k], v.p[k]);
        gb_aside.put(b);
      }
      group_end = (int)(a.gate ? min(a.n, (group + 1) * a.gate_rows) : a.n);
    }
    // d goes from d_out over d_out + rstd_r e to D; what is 0 past a row's end keeps its sums right (rows made
    // of vectors: see share).
    Cols hat_b, hat_r, e, d;
    take<kAligned>(ring, residual, true, 0, t, ringed(row), hat_r);
    const bool block = K::block(a.branch), to_branch = block && K::block(g.d_branch) && post;
    if (block) {
      take<kAligned>(ring, branch, true, 2 * rc, t, ringed(row), hat_b);
      if (post) standardise(hat_b, post_kind, st.x, st.y);
#pragma unroll
      for (int k = 0; k < kPairs; ++k) e.p[k] = mul2(gw.p[k], hat_b.p[k]);
#pragma unroll
      for (int k = 0; k < kPairs; ++k) hat_r.p[k] = fma2(both(a.residual_scale), hat_r.p[k], e.p[k]);
      if (post && K::post_bias(a.b_post)) {
        gb_aside.get(d);
#pragma unroll
        for (int k = 0; k < kPairs; ++k) hat_r.p[k] = add2(hat_r.p[k], d.p[k]);
      }
    } else {
      hat_b.fill(0.0f);
      e.fill(0.0f);
    }
    if (pre) standardise(hat_r, pre_kind, st.z, st.w);
    // The sums of both norms in one exchange: with t = d_out + rstd_r e, w = gw hat_b and the means m of e and e hat_r,
    //   sum f       = sum gw t - rstd_r (m1 sum gw + m2 sum gw hat_r)
    //   sum f hat_b = sum w t  - rstd_r (m1 sum w  + m2 sum w hat_r)
    // (values 0 and 3 are the sums of e hat_r and e, 1 and 2 those of w t and w hat_r).
    constexpr int kMany = kForm == kMixed || kForm == kLayer ? 8 : 4;
    constexpr bool kMean = kForm == kMixed || K::kBias, kBoth = kForm == kMixed || K::kPost;
    float v[kMany] = {};
    if constexpr (kBoth) v[2] = t.share(dot(e, hat_r));      // e: w so far
    if constexpr (kMany == 8) {
      v[4] = t.share(total(e));
      v[5] = t.share(total(gw));
      v[6] = t.share(dot(gw, hat_r));
    }
    take<kAligned>(ring, d_out, K::has(g.d_out), rc, t, ringed(row), d);
    if (pre) {
      Cols w = e;
      take<kAligned>(ring, d_normed, true, 2 * rc + bc, t, ringed(row), e);
      if (kSums > 0) {
#pragma unroll
        for (int k = 0; k < kPairs; ++k) s_wpre.p[k] = fma2(e.p[k], hat_r.p[k], s_wpre.p[k]);
      }
      if (kSums > 1) {
#pragma unroll
        for (int k = 0; k < kPairs; ++k) s_bpre.p[k] = add2(s_bpre.p[k], e.p[k]);
      }
      scale_by(e, K::has(a.w_pre), w_pre, t);
      v[0] = t.share(dot(e, hat_r));
      if constexpr (kMean) v[3] = t.share(total(e));
#pragma unroll
      for (int k = 0; k < kPairs; ++k) d.p[k] = fma2(both(st.w), e.p[k], d.p[k]);
      if constexpr (kBoth) v[1] = t.share(dot(w, d));
    } else {
      v[1] = t.share(dot(e, d));
    }
    if constexpr (kMany == 8) v[7] = t.share(dot(gw, d));
    if constexpr (!kBoth && !kMean) v[0] = t.sum(v[0]);
    else if (pre || to_branch) t.sum(v);
    else t.meet();                             // the sums' exchange, or this: the team has read the stage
    const float m2 = pre ? v[0] * a.inv_dim * st.w : 0.0f;             // times rstd_r
    const float m1 = kMean && pre_kind == MFSDP_NORM_LAYER && pre ? v[3] * a.inv_dim * st.w : 0.0f;
    if (pre) {
#pragma unroll
      for (int k = 0; k < kPairs; ++k) d.p[k] = fma2(hat_r.p[k], both(-m2), d.p[k]);
      if (kMean && pre_kind == MFSDP_NORM_LAYER) {
#pragma unroll
        for (int k = 0; k < kPairs; ++k) d.p[k] = add2(d.p[k], both(-m1));
      }
    }
    fetch(row + kStages * plan.stride);
    if (K::has(g.d_residual)) {
#pragma unroll
      for (int k = 0; k < kPairs; ++k) e.p[k] = mul2(d.p[k], both(d_scale));
      d_residual.store(e, t);
      d_residual.next();
    }
    if (!block) continue;
    if (kSums > 0) {
#pragma unroll
      for (int k = 0; k < kPairs; ++k) s_p.p[k] = fma2(d.p[k], hat_b.p[k], s_p.p[k]);
      if (kSumsR) {
#pragma unroll
        for (int k = 0; k < kPairs; ++k) s_r.p[k] = add2(s_r.p[k], d.p[k]);
      }
      if (!one_gate && (row + 1 == group_end || row + 1 == r1)) close_group();
    }
    if (!K::block(g.d_branch)) continue;
#pragma unroll
    for (int k = 0; k < kPairs; ++k) d.p[k] = mul2(d.p[k], gw.p[k]);
    if (post) {
      const float f2 = v[1] - m1 * v[kMany == 8 ? 4 : 0] - m2 * v[2];  // m1 is 0 where there are 4 values
#pragma unroll
      for (int k = 0; k < kPairs; ++k) d.p[k] = fma2(hat_b.p[k], both(-f2 * a.inv_dim), d.p[k]);
      if (kMany == 8 && post_kind == MFSDP_NORM_LAYER) {
        const float f1 = v[kMany - 1] - m1 * v[kMany == 8 ? 5 : 0] - m2 * v[kMany == 8 ? 6 : 0];
#pragma unroll
        for (int k = 0; k < kPairs; ++k) d.p[k] = add2(d.p[k], both(-f1 * a.inv_dim));
      }
#pragma unroll
      for (int k = 0; k < kPairs; ++k) d.p[k] = mul2(both(st.y), d.p[k]);
    }
    d_branch.store(d, t);
    d_branch.next();
  }
  if (kSums == 0) return;
  if (one_gate && K::block(a.branch)) close_group();     // of a run without rows: zeros
  // The CTA's teams are added in order, through the ring's place, whose copies have all arrived: every team leaves its
  // sums of all vectors, and all threads add them up.
  ptx::launch_dependents();
  const int teams = blockDim.x / t.threads;
  float* const part = g.parts + (int64_t)(blockIdx.x / plan.parts) * kNormParts * a.dim;
  const auto leave = [&](int which, const Cols& s) {
    if (teams == 1) put_vector(part + which * a.dim, s, 0, t);
    else Aside(end + which * kAsideFloats).put(s);
  };
  if (teams > 1) __syncthreads();              // the last rows have been read
  if (g.d_w_pre) leave(kSumWPre, s_wpre);
  if (kSums > 1 && g.d_b_pre) leave(kSumBPre, s_bpre);
  if (g.d_gate && one_gate) {
#pragma unroll
    for (int k = 0; k < kPairs; ++k) s_p.p[k] = mul2(s_p.p[k], both(a.branch_scale));
    leave(kSumGate, s_p);
  }
  if (g.d_w_post) {
    if (kSumsR) wpost_aside.get(s_wpost);
    leave(kSumWPost, s_wpost);
  }
  if (kSumsR && g.d_b_post) {
    bpost_aside.get(s_r);
    leave(kSumBPost, s_r);
  }
  if (teams == 1) return;
  __syncthreads();
  const uint32_t wanted = (g.d_w_pre ? 1u << kSumWPre : 0) | (kSums > 1 && g.d_b_pre ? 1u << kSumBPre : 0) |
                          (g.d_gate && one_gate ? 1u << kSumGate : 0) | (g.d_w_post ? 1u << kSumWPost : 0) |
                          (kSumsR && g.d_b_post ? 1u << kSumBPost : 0);
  join_teams<kAligned>(end, part, wanted, teams, t.threads, a.dim);
}

// The run that has a row.
__device__ __forceinline__ int run_of(int64_t row, int64_t n, int units) {
  int k = (int)(row * units / n);
  while (run_start(k + 1, n, units) <= row) ++k;
  while (run_start(k, n, units) > row) --k;
  return k;
}

// Adds up the parts, in order: 128 columns a CTA, 4 a lane, its warps a share of the parts each.  blockIdx.y: first
// the vectors, then the groups of a gate that lie in more than one run.
constexpr int kJoinWarps = 32, kJoinCols = 128;        // at most
__global__ void __launch_bounds__(kJoinWarps * 32) norm_join_kernel(const NormGradArgs g, int ctas, int units, int jobs) {
  __shared__ float sum[kJoinWarps][kJoinCols];
  const NormArgs& a = g.f;
  ptx::wait_dependencies();
  if (a.n == 0 && blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) *g.status = 0;       // no other kernel runs
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  float* to = nullptr;
  const float* parts = nullptr;
  int64_t step = 0;                           // floats between parts
  int count = 0;
  const float* head = nullptr;                // a part that comes before these
  if (blockIdx.y < kNormParts) {
    to = blockIdx.y == kSumWPost ? g.d_w_post : blockIdx.y == kSumBPost ? g.d_b_post : blockIdx.y == kSumWPre ? g.d_w_pre
         : blockIdx.y == kSumBPre ? g.d_b_pre : a.gate_rows >= a.n ? g.d_gate : nullptr;
    parts = g.parts + (int64_t)blockIdx.y * a.dim;
    step = (int64_t)kNormParts * a.dim;
    count = ctas;
  } else {
    // with few groups a job is a group, with many it is a border of two runs and the group that it cuts
    const int job = blockIdx.y - kNormParts;
    const bool by_group = (a.n + a.gate_rows - 1) / a.gate_rows <= units;
    const int64_t group = by_group ? job : run_start(job + 1, a.n, units) / a.gate_rows;
    const int64_t first = group * a.gate_rows, last = min(a.n, first + a.gate_rows) - 1;
    if (first >= a.n) return;
    const int u0 = run_of(first, a.n, units), u1 = run_of(last, a.n, units);
    if (u0 == u1 || (!by_group && u0 != job)) return;
    to = g.d_gate + group * a.dim;
    head = g.gate_parts + ((int64_t)u0 * 2 + 1) * a.dim;
    parts = g.gate_parts + (int64_t)(u0 + 1) * 2 * a.dim;
    step = 2 * (int64_t)a.dim;
    count = u1 - u0;
  }
  if (to == nullptr) return;
  const int c0 = blockIdx.x * kJoinCols + lane;
  float s[kJoinCols / 32] = {};
  const int k0 = count * warp / warps, k1 = count * (warp + 1) / warps;
#pragma unroll
  for (int i = 0; i < kJoinCols / 32; ++i)
    if (head && warp == 0 && c0 + 32 * i < a.dim) s[i] = head[c0 + 32 * i];
#pragma unroll 4
  for (int k = k0; k < k1; ++k) {
#pragma unroll
    for (int i = 0; i < kJoinCols / 32; ++i)
      if (c0 + 32 * i < a.dim) s[i] += parts[k * step + c0 + 32 * i];
  }
#pragma unroll
  for (int i = 0; i < kJoinCols / 32; ++i) sum[warp][lane + 32 * i] = s[i];
  __syncthreads();
  const int c = blockIdx.x * kJoinCols + threadIdx.x;
  if (threadIdx.x >= kJoinCols || c >= a.dim) return;
  float x = sum[0][threadIdx.x];
  for (int w = 1; w < warps; ++w) x += sum[w][threadIdx.x];
  put(to + c, x, g.accumulate);
}

// ------------------------------------------------------------------ launches
// How rows are divided: by their number and width alone.
struct NormDivision {
  int parts, part_cols, warps, teams;
  int rows_at_once;  // CTAs, or clusters, that have a team each at least
  int units;
};
NormDivision divide(int64_t dim, int64_t n, int ctas_per_sm) {
  NormDivision d;
  d.parts = (int)((dim + kCtaCols - 1) / kCtaCols);
  d.part_cols = d.parts > 1 ? (int)round_up((size_t)((dim + d.parts - 1) / d.parts), 8) : (int)dim;
  d.warps = (d.part_cols + 32 * kCols - 1) / (32 * kCols);
  d.teams = d.parts > 1 ? 1 : kMaxWarps / d.warps;
  d.rows_at_once = (int)std::min<int64_t>(ctas_per_sm * kSms / d.parts, (n + d.teams - 1) / d.teams);
  d.units = (int)std::min<int64_t>(n, (int64_t)d.rows_at_once * d.teams);
  return d;
}

// A launch: `chunks`, 16-byte pieces of a thread in a stage, and `vectors`, those kept.
struct NormLaunch {
  NormPlan plan;
  int ctas, threads;
  size_t vector_bytes, stage_bytes;
};
NormLaunch plan_of(const NormArgs& a, int chunks, int vectors, int ctas_per_sm) {
  const NormDivision d = divide(a.dim, a.n, ctas_per_sm);
  NormLaunch l;
  const bool apart = a.gate == nullptr || a.gate_rows >= a.n;
  l.plan = {d.warps, d.units, apart ? d.units : 1, d.parts, d.part_cols, 0};
  l.threads = d.teams * d.warps * 32;
  l.ctas = d.rows_at_once * d.parts;
  l.vector_bytes = (size_t)vectors * d.warps * 32 * kCols * 4;
  l.stage_bytes = (size_t)chunks * (a.vec ? kChunk<true> : kChunk<false>);
  return l;
}

// Rows until 16 bytes before or after one are still its tensor's (steps of 0: no tensor).
int margin_of(std::initializer_list<RowStep> steps) {
  int64_t margin = 1;
  for (const RowStep& s : steps)
    if (s.row > 0) margin = std::max(margin, (16 + s.row - 1) / s.row);
  return (int)margin;
}

template <typename A>
cudaError_t launch(void (*kernel)(A, NormPlan), std::atomic<bool> (&ready)[kMaxDevices], const A& args,
                   const NormLaunch& l, int stages, cudaStream_t s) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
  if (!ready[dev].load()) {
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSharedBytes);
    if (e != cudaSuccess) return e;
    ready[dev].store(true);
  }
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = (unsigned)l.plan.parts;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)l.ctas);
  cfg.blockDim = dim3((unsigned)l.threads);
  cfg.dynamicSmemBytes = l.vector_bytes + stages * l.stage_bytes;
  cfg.stream = s;
  cfg.attrs = &attr;
  cfg.numAttrs = l.plan.parts > 1 ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kernel, args, l.plan);
}

// Calls f with the kernel's variant.  Rows made of vectors with a bf16 block, in a known form, have their types known
// too (a cluster's: with RMS); so has an fp32 block between two norms.  Else it is as it comes.
template <typename F>
cudaError_t with_variant(const NormArgs& a, Form form, bool cluster, F&& f) {
  using std::false_type;
  using std::integral_constant;
  using std::true_type;
  using Any = integral_constant<int, kAny>;
  using Mixed = integral_constant<Form, kMixed>;
  if (!a.vec)
    return cluster ? f(Mixed{}, false_type{}, true_type{}, Any{}, Any{}) : f(Mixed{}, false_type{}, false_type{}, Any{}, Any{});
  const auto mixed = [&]() {
    return cluster ? f(Mixed{}, true_type{}, true_type{}, Any{}, Any{}) : f(Mixed{}, true_type{}, false_type{}, Any{}, Any{});
  };
  using F32 = integral_constant<int, kF32>;
  using Bf16 = integral_constant<int, kBf16>;
  const auto typed = [&](auto known, auto many) {
    return a.r_bf16 ? f(known, true_type{}, many, Bf16{}, Bf16{}) : f(known, true_type{}, many, F32{}, Bf16{});
  };
  const auto wide = [&](auto known) {
    return a.r_bf16 ? f(known, true_type{}, false_type{}, Bf16{}, F32{}) : f(known, true_type{}, false_type{}, F32{}, F32{});
  };
  using Rms = integral_constant<Form, kRms>;
  using Layer = integral_constant<Form, kLayer>;
  using AddRms = integral_constant<Form, kAddRms>;
  using FirstRms = integral_constant<Form, kFirstRms>;
  if (!a.b_bf16) return cluster || (form != kRms && form != kLayer) ? mixed() : form == kRms ? wide(Rms{}) : wide(Layer{});
  if (cluster)
    return form == kRms        ? typed(Rms{}, true_type{})
           : form == kAddRms   ? typed(AddRms{}, true_type{})
           : form == kFirstRms ? typed(FirstRms{}, true_type{})
                               : mixed();
  switch (form) {
    case kRms: return typed(Rms{}, false_type{});
    case kLayer: return typed(Layer{}, false_type{});
    case kAddRms: return typed(AddRms{}, false_type{});
    case kAddLayer: return typed(integral_constant<Form, kAddLayer>{}, false_type{});
    case kFirstRms: return typed(FirstRms{}, false_type{});
    case kFirstLayer: return typed(integral_constant<Form, kFirstLayer>{}, false_type{});
    default: return mixed();
  }
}

// The form of a call that has all rows that a form asks for.
Form form_of(const NormArgs& a, bool all_rows) {
  const bool layer = a.pre == MFSDP_NORM_LAYER;
  if (!all_rows || a.pre == MFSDP_NORM_NONE || !a.w_pre || (a.b_pre != nullptr) != layer) return kMixed;
  if (!a.branch) return layer ? kFirstLayer : kFirstRms;
  if (a.post == MFSDP_NORM_NONE) return layer ? kAddLayer : kAddRms;
  if (a.post != a.pre || !a.w_post || (a.b_post != nullptr) != layer) return kMixed;
  return layer ? kLayer : kRms;
}

template <Form kForm, bool kAligned, bool kCluster, int kR, int kB, int kSums>
cudaError_t run_grad(const NormGradArgs& g, NormLaunch l, cudaStream_t s) {
  l.vector_bytes += (size_t)kAsides<kForm, kSums> * kAsideFloats * 4;
  // the ring's place holds all vectors' sums at the end
  constexpr int kStages = kGradStages<kForm, kR, kB, kSums>;
  if (kSums > 0 && l.threads > l.plan.warps * 32)
    l.stage_bytes = std::max(l.stage_bytes, ((size_t)kNormParts * kAsideFloats * 4 + kStages - 1) / kStages);
  static std::atomic<bool> ready[kMaxDevices];
  return launch(norm_grad_kernel<kForm, kAligned, kCluster, kR, kB, kSums>, ready, g, l, kStages, s);
}

}  // namespace

cudaError_t launch_norm(NormArgs a, cudaStream_t s) {
  const int vectors = (a.w_post != nullptr) + (a.b_post != nullptr) + (a.w_pre != nullptr) + (a.b_pre != nullptr);
  NormLaunch l = plan_of(a, (a.r_bf16 ? 1 : 2) + (a.b_bf16 ? 1 : 2), vectors, 2);
  for (RowStep* step : {&a.residual_step, &a.branch_step, &a.out_step, &a.normed_step}) step->next = step->row * l.plan.stride;
  l.plan.margin = margin_of({a.residual_step, a.branch_step});
  return with_variant(a, form_of(a, a.normed && (a.out != nullptr) == (a.branch != nullptr)), l.plan.parts > 1,
                      [&](auto form, auto aligned, auto cluster, auto r, auto b) {
                        static std::atomic<bool> ready[kMaxDevices];
                        return launch(norm_kernel<form(), aligned(), cluster(), r(), b()>, ready, a, l, kForwardStages, s);
                      });
}

cudaError_t launch_norm_grad(NormGradArgs g, cudaStream_t s) {
  NormArgs& a = g.f;
  const bool biases = g.d_b_post || g.d_b_pre || (g.d_gate && a.b_post), weights = g.d_w_post || g.d_w_pre || g.d_gate;
  NormLaunch l = {};
  l.plan.parts = l.plan.units = 1;
  if (a.n > 0) {
    l = plan_of(a, 2 * (a.r_bf16 ? 1 : 2) + 2 * (a.b_bf16 ? 1 : 2), a.w_pre != nullptr, 1);
    for (RowStep* step : {&a.residual_step, &a.branch_step, &g.d_out_step, &g.d_normed_step, &g.d_residual_step,
                          &g.d_branch_step})
      step->next = step->row * l.plan.stride;
    l.plan.margin = margin_of({a.residual_step, a.branch_step, g.d_out_step, g.d_normed_step});
    g.gate_parts = g.parts + (size_t)(l.ctas / l.plan.parts) * kNormParts * (size_t)a.dim;
    // sums of a form: the weights' with RMS, all with LAYER; a call that wants others takes the mixed form
    const Form form = form_of(a, g.d_out && g.d_normed && g.d_residual && (g.d_branch != nullptr) == (a.branch != nullptr));
    const bool rms = form == kRms || form == kAddRms || form == kFirstRms, fits = rms ? weights && !biases : biases;
    const cudaError_t e = with_variant(a, fits ? form : kMixed, l.plan.parts > 1,
                                       [&](auto known, auto aligned, auto cluster, auto r, auto b) {
      if constexpr (known() != kMixed) {
        return run_grad<known(), aligned(), cluster(), r(), b(), Known<known()>::kBias ? 2 : 1>(g, l, s);
      } else {
        if (biases) return run_grad<known(), aligned(), cluster(), r(), b(), 2>(g, l, s);
        if (weights) return run_grad<known(), aligned(), cluster(), r(), b(), 1>(g, l, s);
        return run_grad<known(), aligned(), cluster(), r(), b(), 0>(g, l, s);
      }
    });
    if (e != cudaSuccess) return e;
  }
  if (!biases && !weights) return cudaSuccess;
  const int64_t groups = g.d_gate && a.n > a.gate_rows ? (a.n + a.gate_rows - 1) / a.gate_rows : 0;
  const int units = l.plan.units, jobs = groups <= units ? (int)groups : units - 1;
  return launch_overlapped(norm_join_kernel, dim3((unsigned)((a.dim + kJoinCols - 1) / kJoinCols), (unsigned)(kNormParts + jobs)),
                           dim3(jobs > 64 ? 256 : kJoinWarps * 32), 0, s, a.n > 0, g, l.ctas / l.plan.parts, units, jobs);
}

// The sums of each CTA's vectors, and two rows of a gate for each run.
size_t norm_grad_part_bytes(int64_t dim, int64_t n) {
  const NormDivision d = divide(dim, n, 1);
  return ((size_t)d.rows_at_once * kNormParts + (size_t)d.units * 2) * (size_t)dim * 4;
}

}  // namespace ops
}  // namespace mfsdp
