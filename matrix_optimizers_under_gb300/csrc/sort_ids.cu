// Stable sort of ids by value: the order that groups token positions by token
// (the embedding gradient's sums) or rows by expert (the grouped products).
//
// Least-significant-digit radix sort, 8 bits a pass, ceil(bits / 8) passes over
// (key, position) pairs.  The n ids are cut into tiles, one CTA each, whose
// warps take consecutive runs of it, so that "earlier" is (tile, warp, step,
// lane) order.  A pass counts every tile's digits, adds up the counts that
// come before a tile's -- all smaller digits of every tile, and its own digit
// in earlier tiles -- and moves the pairs.  A pair's place among its warp's
// equal digits comes from ballots, so the sort is stable and its result
// does not depend on timing.  An id outside [0, n_keys) sorts as n_keys, after
// all valid ones.
//
// Up to 65536 ids are sorted by one cluster of up to 8 CTAs in one launch: the
// pairs stay in shared memory, the counts and the moves go through distributed
// shared memory.  The work is latency, not bandwidth (32768 ids are 256 KB): two passes
// as separate launches took 36 us with cold caches, so 13.  More ids take two launches a
// pass, on up to kMaxTiles CTAs.
#include <atomic>

#include "ops_internal.h"
#include "ops_ptx.cuh"

namespace mfsdp {
namespace ops {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kDigits = 256;

// Lanes of the warp that hold the same 8-bit digit, among the lanes of `live`:
// one ballot a bit.  (A match instruction takes ~250 cycles of its scheduler: the
// counting loop of 32768 ids took 8200 cycles a pass with it, and 36 % of the sort.)
__device__ __forceinline__ unsigned same_digit(int digit, unsigned live) {
  unsigned same = live;
#pragma unroll
  for (int b = 0; b < 8; ++b) {
    const unsigned v = __ballot_sync(0xffffffffu, (digit >> b) & 1);
    same &= (digit >> b) & 1 ? v : ~v;
  }
  return same;
}

// ------------------------------------------------------------- one cluster
constexpr int kClusterThreads = 1024;
constexpr int kClusterWarps = kClusterThreads / 32;
constexpr int kClusterSteps = 8;                                // pairs of a thread
constexpr int kClusterTile = kClusterThreads * kClusterSteps;   // pairs of a CTA
constexpr int kMaxCluster = kSortSms;
constexpr int kQuarters = kClusterThreads / kDigits;             // threads that add up one digit's warps
constexpr size_t kClusterSmem = (size_t)kClusterTile * 16 + (size_t)kClusterWarps * kDigits * 4;

struct ClusterArgs {
  const void* ids;
  int32_t ids64, n_keys, n;
  int32_t steps;            // pairs a thread takes: the tile is 1024 steps
  int32_t passes;
  int32_t* keys_out;
  int32_t* order_out;
  int32_t* zero;
};

__global__ void __launch_bounds__(kClusterThreads, 1) sort_cluster_kernel(const __grid_constant__ ClusterArgs a) {
  extern __shared__ __align__(16) uint8_t smem[];
  uint64_t* pairs = reinterpret_cast<uint64_t*>(smem);                       // (position << 32) | key
  uint64_t* local = pairs + kClusterTile;                                    // this CTA's pairs by digit
  int (*cnt)[kDigits] = reinterpret_cast<int (*)[kDigits]>(smem + (size_t)kClusterTile * 16);
  __shared__ int hist[kDigits];                                              // this CTA's digits
  __shared__ int quarter[kQuarters][kDigits];
  __shared__ int start[kDigits], shift_to[kDigits];      // of a digit in `local`; from there to its place
  __shared__ int scan[2][kDigits / 32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = blockIdx.x, ctas = gridDim.x;                             // the grid is one cluster
  const int tile = a.steps * kClusterThreads;
  ptx::launch_dependents();
  if (rank == 0 && threadIdx.x == 0 && a.zero) *a.zero = 0;
  const int local0 = warp * a.steps * 32 + lane;                             // this thread's first pair in the tile
  uint64_t pr[kClusterSteps];
#pragma unroll
  for (int k = 0; k < kClusterSteps; ++k) {
    const int i = rank * tile + local0 + 32 * k;
    if (k < a.steps && i < a.n) {
      const int64_t v = a.ids64 ? static_cast<const int64_t*>(a.ids)[i] : static_cast<const int32_t*>(a.ids)[i];
      pr[k] = ((uint64_t)(uint32_t)i << 32) | (uint32_t)(v >= 0 && v < a.n_keys ? (int)v : a.n_keys);
    }
  }
  for (int pass = 0; pass < a.passes; ++pass) {
    const int shift = 8 * pass;
    if (pass > 0) {
#pragma unroll
      for (int k = 0; k < kClusterSteps; ++k)
        if (k < a.steps && rank * tile + local0 + 32 * k < a.n) pr[k] = pairs[local0 + 32 * k];
    }
    for (int d = threadIdx.x; d < kClusterWarps * kDigits; d += kClusterThreads) (&cnt[0][0])[d] = 0;
    __syncthreads();
    int place[kClusterSteps];            // among the warp's pairs of its digit
#pragma unroll
    for (int k = 0; k < kClusterSteps; ++k) {
      if (k >= a.steps) break;
      const bool in = rank * tile + local0 + 32 * k < a.n;
      const int digit = in ? (int)((uint32_t)pr[k] >> shift) & (kDigits - 1) : 0;
      const unsigned same = same_digit(digit, __ballot_sync(0xffffffffu, in));
      if (in) place[k] = cnt[warp][digit] + __popc(same & ((1u << lane) - 1));
      __syncwarp();
      if (in && (same >> lane) == 1u) cnt[warp][digit] = place[k] + 1;
      __syncwarp();
    }
    __syncthreads();
    // counts of a digit over the warps before each: four threads a digit
    const int d = threadIdx.x & (kDigits - 1), q = threadIdx.x / kDigits;
    constexpr int kPer = kClusterWarps / kQuarters;
    int own[kPer], sum = 0;
#pragma unroll
    for (int w = 0; w < kPer; ++w) own[w] = cnt[q * kPer + w][d];
#pragma unroll
    for (int w = 0; w < kPer; ++w) {
      const int c = own[w];
      own[w] = sum;
      sum += c;
    }
    quarter[q][d] = sum;
    __syncthreads();
    int ahead = 0, mine = 0;
#pragma unroll
    for (int k = 0; k < kQuarters; ++k) {
      if (k < q) ahead += quarter[k][d];
      mine += quarter[k][d];
    }
#pragma unroll
    for (int w = 0; w < kPer; ++w) cnt[q * kPer + w][d] = own[w] + ahead;
    if (q == 0) hist[d] = mine;
    ptx::cluster_sync();                 // every CTA's counts stand, and its pairs are in registers
    int total = 0, before = 0, run = mine, all = 0;
    if (q == 0) {
      const uint32_t at = ptx::smem_u32(&hist[d]);
      int h[kMaxCluster];                // all in flight together: a remote read takes ~0.5 us
#pragma unroll
      for (int c = 0; c < kMaxCluster; ++c)
        h[c] = c < ctas ? ptx::ld_shared_cluster_s32(ptx::mapa_shared(at, (uint32_t)c)) : 0;
#pragma unroll
      for (int c = 0; c < kMaxCluster; ++c) {
        total += h[c];
        if (c < rank) before += h[c];
      }
      all = total;                       // inclusive scans over the digits: here, and in the cluster
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, run, o), u = __shfl_up_sync(0xffffffffu, all, o);
        if (lane >= o) {
          run += v;
          all += u;
        }
      }
      if (lane == 31) {
        scan[0][warp] = run;
        scan[1][warp] = all;
      }
    }
    __syncthreads();
    if (q == 0) {
      for (int w = 0; w < warp; ++w) {
        run += scan[0][w];
        all += scan[1][w];
      }
      start[d] = run - mine;
      shift_to[d] = all - total + before - (run - mine);
    }
    __syncthreads();
    // By digit in this CTA first, so that neighbours then move to neighbouring places.
#pragma unroll
    for (int k = 0; k < kClusterSteps; ++k) {
      if (k >= a.steps || rank * tile + local0 + 32 * k >= a.n) break;
      const int digit = ((uint32_t)pr[k] >> shift) & (kDigits - 1);
      local[start[digit] + cnt[warp][digit] + place[k]] = pr[k];
    }
    __syncthreads();
    const bool last = pass == a.passes - 1;
    const int held = min(tile, a.n - rank * tile);
#pragma unroll
    for (int k = 0; k < kClusterSteps; ++k) {
      const int j = k * kClusterThreads + threadIdx.x;
      if (j >= held) break;
      const uint64_t v = local[j];
      const int to = j + shift_to[((uint32_t)v >> shift) & (kDigits - 1)];
      if (last) {
        a.keys_out[to] = (int32_t)(uint32_t)v;
        a.order_out[to] = (int32_t)(v >> 32);
      } else {
        const int c = to / tile;
        ptx::st_shared_cluster_u64(ptx::mapa_shared(ptx::smem_u32(&pairs[to - c * tile]), (uint32_t)c), v);
      }
    }
    if (!last) ptx::cluster_sync();      // every pair has arrived, and no CTA still reads these counts
  }
  ptx::cluster_sync();                   // no CTA leaves while another reads its counts
}

cudaError_t launch_cluster(const SortArgs& s, int passes, cudaStream_t stream) {
  static std::atomic<bool> ready[kMaxDevices];          // the kernel's shared memory is allowed, per device
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
  if (!ready[dev].load()) {
    e = cudaFuncSetAttribute(sort_cluster_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kClusterSmem);
    if (e != cudaSuccess) return e;
    ready[dev].store(true);
  }
  ClusterArgs a{};
  a.ids = s.ids;
  a.ids64 = s.ids64;
  a.n_keys = (int32_t)s.n_keys;
  a.n = (int32_t)s.n;
  a.passes = passes;
  a.keys_out = s.keys_out;
  a.order_out = s.order_out;
  a.zero = s.zero;
  int ctas = 1;
  // a CTA an SM, up to 8, before a thread takes a second pair
  while (ctas < kMaxCluster && s.n > (int64_t)ctas * kClusterThreads) ctas *= 2;
  a.steps = (int)((s.n + (int64_t)ctas * kClusterThreads - 1) / ((int64_t)ctas * kClusterThreads));
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = (unsigned)ctas;
  attr.val.clusterDim.y = 1;
  attr.val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)ctas);
  cfg.blockDim = dim3(kClusterThreads);
  cfg.dynamicSmemBytes = kClusterSmem;
  cfg.stream = stream;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, sort_cluster_kernel, a);
}

// ---------------------------------------------------------- two launches a pass
constexpr int kMaxTiles = 256;
constexpr int kMinSteps = 8;            // a warp's steps of 32 ids a tile, at least

struct SortPlan {
  int tiles;
  int steps;                            // steps of 32 ids a warp takes
  int passes;
};

SortPlan plan_sort(int64_t n, int64_t n_keys) {
  SortPlan p{};
  int bits = 0;
  while (bits < 32 && (n_keys >> bits) != 0) ++bits;     // keys are 0 .. n_keys
  p.passes = std::max(1, (bits + 7) / 8);
  const int64_t per_step = kWarps * 32;
  const int64_t steps_all = (n + per_step - 1) / per_step;
  const int64_t steps = std::max<int64_t>(kMinSteps, (steps_all + kMaxTiles - 1) / kMaxTiles);
  p.steps = (int)steps;
  p.tiles = (int)std::max<int64_t>(1, (steps_all + steps - 1) / steps);
  return p;
}

struct PassArgs {
  const void* ids;          // first pass: the ids; later ones: null
  int32_t ids64;
  int32_t n_keys;
  const int2* in;           // (key, position) pairs of the last pass
  int2* out;                // pairs, or in the last pass null:
  int32_t* keys_out;
  int32_t* order_out;
  int32_t* counts;          // [tile][digit]
  int64_t n;
  int32_t tiles, steps, shift;
  int32_t* zero;            // first pass
};

__device__ __forceinline__ int2 load_pair(const PassArgs& a, int64_t i) {
  if (!a.ids) return a.in[i];
  const int64_t v = a.ids64 ? static_cast<const int64_t*>(a.ids)[i] : static_cast<const int32_t*>(a.ids)[i];
  return make_int2(v >= 0 && v < a.n_keys ? (int)v : a.n_keys, (int)i);
}

// Counts of each digit, per warp, over the tile's run of each warp.
__device__ __forceinline__ void count_digits(const PassArgs& a, int (*cnt)[kDigits]) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int d = threadIdx.x; d < kWarps * kDigits; d += kThreads) (&cnt[0][0])[d] = 0;
  __syncthreads();
  const int64_t base = ((int64_t)blockIdx.x * kWarps + warp) * a.steps * 32;
  for (int k = 0; k < a.steps; ++k) {
    const int64_t i = base + k * 32 + lane;
    if (i < a.n) atomicAdd(&cnt[warp][(load_pair(a, i).x >> a.shift) & (kDigits - 1)], 1);
  }
  __syncthreads();
}

__global__ void __launch_bounds__(kThreads) sort_count_kernel(const __grid_constant__ PassArgs a) {
  __shared__ int cnt[kWarps][kDigits];
  if (a.zero && blockIdx.x == 0 && threadIdx.x == 0) *a.zero = 0;
  count_digits(a, cnt);
  int s = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) s += cnt[w][threadIdx.x];
  a.counts[(int64_t)blockIdx.x * kDigits + threadIdx.x] = s;
}

__global__ void __launch_bounds__(kThreads) sort_move_kernel(const __grid_constant__ PassArgs a) {
  __shared__ int cnt[kWarps][kDigits];       // counts, then the next place of each warp's digit
  __shared__ int scan[kDigits];
  count_digits(a, cnt);
  const int d = threadIdx.x;
  int before = 0, total = 0;
  for (int t = 0; t < a.tiles; ++t) {
    const int c = a.counts[(int64_t)t * kDigits + d];
    total += c;
    if (t < (int)blockIdx.x) before += c;
  }
  scan[d] = total;
  __syncthreads();
  for (int o = 1; o < kDigits; o <<= 1) {     // inclusive scan over the digits
    const int v = d >= o ? scan[d - o] : 0;
    __syncthreads();
    scan[d] += v;
    __syncthreads();
  }
  int at = scan[d] - total + before;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    const int c = cnt[w][d];
    cnt[w][d] = at;
    at += c;
  }
  __syncthreads();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t base = ((int64_t)blockIdx.x * kWarps + warp) * a.steps * 32;
  for (int k = 0; k < a.steps; ++k) {
    const int64_t i = base + k * 32 + lane;
    const bool in = i < a.n;
    const unsigned live = __ballot_sync(0xffffffffu, in);
    const int2 p = in ? load_pair(a, i) : make_int2(0, 0);
    const int digit = (p.x >> a.shift) & (kDigits - 1);
    const unsigned same = same_digit(digit, live);
    if (in) {
      const int place = cnt[warp][digit] + __popc(same & ((1u << lane) - 1));
      __syncwarp(live);
      if ((same >> lane) == 1u) cnt[warp][digit] = place + 1;     // the last of them moves the next place on
      if (a.out) {
        a.out[place] = p;
      } else {
        a.keys_out[place] = p.x;
        a.order_out[place] = p.y;
      }
    }
    __syncwarp();
  }
}

// starts[k] = the number of sorted keys below k, for k = 0 .. n_keys.
__global__ void __launch_bounds__(kThreads) key_starts_kernel(const int32_t* keys, int64_t n, int64_t n_keys,
                                                              int32_t* starts) {
  const int64_t k = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  if (k > n_keys) return;
  int64_t lo = 0, hi = n;
  while (lo < hi) {
    const int64_t mid = (lo + hi) >> 1;
    if (keys[mid] < k) lo = mid + 1; else hi = mid;
  }
  starts[k] = (int32_t)lo;
}

}  // namespace

size_t sort_scratch_bytes(int64_t n, int64_t n_keys) {
  if (n <= kMaxCluster * kClusterTile) return 0;
  const SortPlan p = plan_sort(n, n_keys);
  return round_up((size_t)p.tiles * kDigits * 4, 256) + 2 * round_up((size_t)n * 8, 256);
}

cudaError_t launch_sort(const SortArgs& s, cudaStream_t stream) {
  if (s.n <= 0) return cudaSuccess;
  const SortPlan p = plan_sort(s.n, s.n_keys);
  if (s.n <= kMaxCluster * kClusterTile) return launch_cluster(s, p.passes, stream);
  uint8_t* base = static_cast<uint8_t*>(s.scratch);
  int2* buf[2];
  buf[0] = reinterpret_cast<int2*>(base + round_up((size_t)p.tiles * kDigits * 4, 256));
  buf[1] = reinterpret_cast<int2*>(reinterpret_cast<uint8_t*>(buf[0]) + round_up((size_t)s.n * 8, 256));
  for (int k = 0; k < p.passes; ++k) {
    PassArgs a{};
    a.ids = k == 0 ? s.ids : nullptr;
    a.ids64 = s.ids64;
    a.n_keys = (int32_t)s.n_keys;
    a.in = k == 0 ? nullptr : buf[(k - 1) & 1];
    a.out = k == p.passes - 1 ? nullptr : buf[k & 1];
    a.keys_out = s.keys_out;
    a.order_out = s.order_out;
    a.counts = reinterpret_cast<int32_t*>(base);
    a.n = s.n;
    a.tiles = p.tiles;
    a.steps = p.steps;
    a.shift = 8 * k;
    a.zero = k == 0 ? s.zero : nullptr;
    sort_count_kernel<<<p.tiles, kThreads, 0, stream>>>(a);
    sort_move_kernel<<<p.tiles, kThreads, 0, stream>>>(a);
  }
  return cudaGetLastError();
}

cudaError_t launch_key_starts(const int32_t* keys, int64_t n, int64_t n_keys, int32_t* starts, cudaStream_t s) {
  key_starts_kernel<<<(unsigned)((n_keys + kThreads) / kThreads), kThreads, 0, s>>>(keys, n, n_keys, starts);
  return cudaGetLastError();
}

}  // namespace ops
}  // namespace mfsdp
