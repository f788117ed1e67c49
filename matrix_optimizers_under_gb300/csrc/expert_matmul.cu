// Matrix products grouped by expert, on 5th-generation tensor cores: rows
// [starts[e], starts[e + 1]) of the activations meet expert e's matrix W_e
// (rows x cols).
//   forward:          Y[t, :]  = W_e X[t, :]
//   input gradient:   dX[t, :] = W_e^T dY[t, :]
//   weight gradient:  dW_e (+)= dY_e^T X_e         (zero for an expert without rows)
//
// Groups are ragged, and a mixture-of-experts layer has many small ones, so
// the forward products put the matrix on the MMA's M side (always full: 256
// rows of W_e, or of W_e^T, a CTA pair) and the tokens on its N side, which goes in steps
// of 32: a group of 40 tokens costs 64 columns, not 256.  The weight gradient
// has the matrix on both sides and contracts over the tokens.  Operands, as
// the tensor copies find them in memory (K: the contraction):
//   forward          A = W_e    K-major       B = X     K-major
//   input gradient   A = W_e^T  MN-major      B = dY    K-major
//   weight gradient  A = dY^T   MN-major      B = X^T   MN-major
// No operand is transposed or copied first.  A matrix edge needs no code: the
// maps are bounded by the matrix (three dimensions, the expert the last) and
// fill with zeros.  A group's edge does: on the N side the extra tokens are
// computed and not stored; on the K side (weight gradient) a group's last
// tokens past a multiple of 16, the MMA's K, come from a copy padded to 16 rows with
// zeros, which a small kernel makes first: 16 rows of both operands an expert.
// (Zeroing the next group's rows in shared memory instead, in both CTAs of the pair,
// cost the issuer 1800-1950 cycles a tile of 5300; zeroing one operand
// would let a NaN of the other through.)
//
// CTA pairs (one CTA per SM, cta_group::2) take tiles of 256 x up to 256 round-robin
// from a list that every CTA works out from `starts`, expert by expert, so a wave's
// tiles share their operands in L2.  A CTA loads its 128 rows of A and its half of B,
// 32 KB per 64 of K: 64 bytes a clock at the full MMA rate, where a CTA alone on 128 x
// 256 would need 96.  Warp roles: 0 producer, 1 MMA issuer (even CTA), 4-11 epilogue;
// two accumulators in TMEM let the epilogue overlap the next tile.  The pipeline has as
// many stages of K = 64 as shared memory holds at the launch's widest tile: 6 of 32 KB
// for 256 tokens, 10 of 20 KB for a few tokens, where the product is bound by reading
// W.
//
// One expert, 32768 x 2048 x 2048: 156 us, 1757 TFLOP/s.  115 experts of 1408 x 2048 that
// share 32768 tokens: forward 162 us, input gradient of 16383 tokens 127, weight gradient
// of 128 in bf16 202, each kernel by itself; 180 to 184, 129 to 132 and 214 to 223 for calls back to
// back on inputs that L2 does not hold.  These are bound by operands on their way
// (a group of 285 tokens takes two tiles, which both read W: 115 of them 170 us, of 256
// tokens 150) and by HBM, at 4.9, 5.9 and 4.4 TB/s.
#include <cuda.h>
#include <cuda_bf16.h>

#include <climits>
#include <mutex>

#include "ops_internal.h"
#include "ops_ptx.cuh"

namespace mfsdp {
namespace ops {
namespace {

constexpr int kPairM = 256;               // rows of a pair's tile
constexpr int kCtaM = 128;                // rows of one CTA's half: its TMEM lanes
constexpr int kMaxN = 256;                // columns of a tile
constexpr int kStepN = 32;                // N granularity of the pair MMA
constexpr int kBlockK = 64;               // K of a stage: one 128-byte swizzle row of bf16
constexpr int kBytesA = kCtaM * kBlockK * 2;          // 16 KB
constexpr int kMnBlock = 64 * kBlockK * 2;            // 8 KB: 64 MN elements x 64 K rows (MN-major)
constexpr int kEnd = 16;                              // K of one MMA: rows of a group's padded end
constexpr int kMaxStages = 10;
// The producer and the issuer take two stages at a time: a turn of their loops
// (election, counters) costs ~300 cycles, and a stage's MMAs take 512.
constexpr int kTurn = 2;
// Shared memory of the stages (six of 32 KB, or ten of 20 KB), and of a part of an
// epilogue warp's staging, which has two.
constexpr int kRingBytes(int mode, bool accumulate) {
  return mode != kExpertWeightGrad ? 10 * 20480 : accumulate ? 4 * 32768 : 6 * 32768;
}
constexpr int kPartBytes(int mode) { return mode == kExpertWeightGrad ? 2048 : 1024; }
// Contraction of an fp32 output that one accumulator takes.  The tensor cores' additions
// cut off low bits, always towards zero: off by 1.0e-6 of the result (2-norms, normal
// operands) at K = 1024, 2.1e-6 at 2048, 1.9e-5 at 16384, 7.6e-5 at 65536, where a loop of
// fp32 additions is off by 3e-7.  So a longer one is taken in even turns, and the turns'
// sums are added, rounded to nearest, where the output lies.  Turns of up to 2048 would be
// faster (one expert, 32768 x 2048 x 2048: 163 us instead of 180; its weight gradient 180
// instead of 211) and twice as far off; of up to 960, three here, 228 and 219 us.
// A bf16 output is off by 1.7e-3 of its rounding alone, which the cut bits would reach near
// K = 2^20 (positive operands there: 6.1e-3 too small in the mean): it takes turns of up to
// 32768 (3.8e-5), whose sum stays in tensor memory.  (Weight gradient of one expert, 2048 x 2048
// and 131072 tokens: 603 us with turns and without.)
constexpr int kMaxK(bool bf16) { return bf16 ? 32768 : 1024; }
constexpr int kEpiWarps = 8;
constexpr int kFirstEpiWarp = 4;
constexpr int kThreads = 32 * (kFirstEpiWarp + kEpiWarps);
constexpr int kSplitPairs = kSms / 2;                 // pairs that a split contraction is cut for
constexpr int kFewTokens = 16;                         // forward: so many go without tensor cores
constexpr int kAccCols = 256;
constexpr int kTmemCols = 512;
constexpr uint64_t kDrainNs = 2000000000ull;          // limit of the waits that end a CTA

struct Maps {
  CUtensorMap a;      // box 64 x 128 (K-major A) or 64 x 64
  CUtensorMap b;      // box 64 x 32 (K-major B) or 64 x 64
  CUtensorMap c;      // box 64 x 128 (K-major B); weight gradient: the padded ends of A, box 64 x 16
  CUtensorMap d;      // box 64 x 64 (K-major B); weight gradient: the padded ends of B, box 64 x 16
  CUtensorMap out;    // dW, box 128 bytes x 16; or Y, box 32 elements x 1 KB
};

// What adds up a split weight gradient.
struct ChunkSumArgs {
  const float* parts;
  void* out;
  const int32_t* starts;
  int64_t n_rows, rows, cols, part_ld, out_ld, out_stride;
  int32_t experts, chunk, slots, accumulate;
};

// First failing wait of a launch (its role), and the waits' limit.
struct Abort {
  volatile int* flag;
  int32_t* status;
  uint64_t limit_ns;
};
enum Role : int32_t { kRoleStage = 1, kRoleOperands = 2, kRoleAccFree = 3, kRoleAccFull = 4 };

template <bool kCluster>
__device__ __forceinline__ bool wait_bar(uint32_t bar, uint32_t parity, const Abort& ab, int32_t role) {
  auto poll = [&] { return kCluster ? ptx::mbar_try_wait_cluster(bar, parity) : ptx::mbar_try_wait(bar, parity); };
  if (poll()) return true;
  const uint64_t t0 = ptx::globaltimer_ns();
  while (true) {
#pragma unroll 1
    for (int i = 0; i < 32; ++i)
      if (poll()) return true;
    if (*ab.flag) return false;
    if (ptx::globaltimer_ns() - t0 > ab.limit_ns) {
      *ab.flag = 1;
      atomicCAS(ab.status, 0, role);
      return false;
    }
  }
}

// One tile: `rows` [m0, m0 + 256) of the M side, columns [n0, n0 + n) of the N
// side (n_mma of them in the MMA), k_len of contraction.
struct Tile {
  int32_t e;
  int32_t z;          // matrix of the output stack
  int32_t group;      // first token of the group
  int32_t m0, n0;
  int32_t n, n_mma;
  int32_t k_from, k_len;     // of the contraction: where it starts, how long it is
};

struct Shape {
  int32_t m;          // M side of every tile: rows (forward, weight gradient) or cols
  int32_t tiles_m;
  int32_t n;          // weight gradient: N side (cols)
  int32_t tiles_n, width_n;
  int32_t chunk;      // weight gradient: tokens of a chunk of a split contraction
};

__device__ __forceinline__ int ceil_div(int a, int b) { return (a + b - 1) / b; }
// Stages of a contraction of length k: whole blocks of 64 (the last one may be
// short), and in the weight gradient the padded end of a length that is no multiple of 16.
template <bool kWgrad>
__device__ __forceinline__ int blocks_of(int k) {
  return kWgrad ? ceil_div(k & ~(kEnd - 1), kBlockK) + ((k & (kEnd - 1)) != 0) : ceil_div(k, kBlockK);
}
// n split over `parts` tiles, each a multiple of `step` wide.
__device__ __forceinline__ int even_width(int n, int parts, int step = kStepN) {
  return (ceil_div(n, parts) + step - 1) / step * step;
}

// Rows of shared memory that one CTA's nh columns of a K-major B take: the copies' boxes.
__device__ __forceinline__ uint32_t rows_b(int nh) { return nh > 96 ? 128 : ceil_div(nh, 32) * 32; }

// Chunks of a split contraction of length k (none: one, of zeros).
__host__ __device__ __forceinline__ int chunks_of(int k, int chunk) { return k <= chunk ? 1 : (k + chunk - 1) / chunk; }

// The chunk of a launch, and the chunks of the experts before `e` and of e: by a
// whole warp, with an expert or two a lane.  Groups whose starts fall overlap, and may make
// more chunks than there is workspace for; then every group is one.
struct Chunks {
  int chunk, before, mine;
};
__device__ __forceinline__ Chunks find_chunks(const int32_t* starts, int experts, int n_rows, int chunk, int slots,
                                              int e) {
  static_assert(kSplitPairs / 2 <= 64, "two experts a lane");
  const int lane = threadIdx.x & 31;
  int len[2];
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int i = min(lane + 32 * k, experts - 1);
    const int to = starts[i + 1], from = starts[i];
    len[k] = min(max(to, 0), n_rows) - (i == 0 ? 0 : min(max(from, 0), n_rows));
  }
  Chunks r{chunk, 0, 0};
  auto count = [&](auto want) {
    int sum = 0;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int i = lane + 32 * k;
      if (i < experts && want(i)) sum += chunks_of(len[k], r.chunk);
    }
    return (int)__reduce_add_sync(0xffffffffu, (unsigned)sum);
  };
  if (count([](int) { return true; }) > slots) r.chunk = INT_MAX;
  r.before = count([&](int i) { return i < e; });
  r.mine = count([&](int i) { return i == e; });
  return r;
}

// First token of expert e's group, kept inside the rows there are.
__device__ __forceinline__ int start_of(const ExpertArgs& p, int e) {
  return e == 0 ? 0 : min(max(p.starts[e], 0), (int)p.n_rows);
}

template <int kMode>
__device__ __forceinline__ Tile decode(const ExpertArgs& p, const Shape& sh, const int32_t* start,
                                       const int32_t* first, int t) {
  Tile r;
  // the expert whose tiles begin last at or before t
  auto expert_of = [&]() {
    int lo = 0, hi = p.n_experts - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (first[mid] <= t) lo = mid; else hi = mid - 1;
    }
    return lo;
  };
  if (kMode == kExpertWeightGrad) {
    const int per = sh.tiles_m * sh.tiles_n;
    int i, chunk = 0;
    if (p.chunk > 0) {
      r.e = expert_of();
      i = t - first[r.e];
      chunk = i / per;
      i -= chunk * per;
      r.z = first[r.e] / per + chunk;
    } else {
      r.e = r.z = t / per;
      i = t - r.e * per;
    }
    const int j = i / sh.tiles_m;
    r.m0 = (i - j * sh.tiles_m) * kPairM;
    r.n0 = j * sh.width_n;
    r.n = min(sh.width_n, sh.n - r.n0);
    r.group = start_of(p, r.e);
    r.k_len = max(0, start_of(p, r.e + 1) - r.group);
    if (p.chunk > 0) {
      r.group += chunk * sh.chunk;
      r.k_len = min(r.k_len - chunk * sh.chunk, sh.chunk);
    }
  } else {
    const int lo = expert_of();
    r.e = r.z = lo;
    const int len = start[lo + 1] - start[lo];
    const int width = even_width(len, ceil_div(len, kMaxN));
    const int i = t - first[lo], j = i / sh.tiles_m;
    r.m0 = (i - j * sh.tiles_m) * kPairM;
    r.n0 = j * width;
    r.n = min(width, len - r.n0);
    r.group = start[lo];
    r.k_len = (int)(kMode == kExpertForward ? p.cols : p.rows);
  }
  r.n_mma = (r.n + kStepN - 1) / kStepN * kStepN;
  return r;
}

// `rows` (32, 64, 96 or 128) rows of K-major B, K columns k0 on, from token t on.
__device__ __forceinline__ void load_tokens(const Maps& maps, uint32_t sb, uint32_t rows, int k0, int t, uint32_t bar) {
  if (rows == 128) {
    ptx::tma_load_3d_pair(sb, &maps.c, k0, t, 0, bar);
  } else if (rows >= 64) {
    ptx::tma_load_3d_pair(sb, &maps.d, k0, t, 0, bar);
    if (rows > 64) ptx::tma_load_3d_pair(sb + 8192, &maps.b, k0, t + 64, 0, bar);
  } else {
    ptx::tma_load_3d_pair(sb, &maps.b, k0, t, 0, bar);
  }
}

// A value that all lanes hold, as the compiler can see.
__device__ __forceinline__ uint32_t uniform(uint32_t v) { return __shfl_sync(0xffffffffu, v, 0); }

// The tiles a pair takes: pair0, pair0 + pairs, ...  Finding a tile's place
// takes divisions and a search, ~1000 cycles, of the ~3000 a small tile takes
// in all; so a warp finds 32 tiles at a time, one a lane, and hands them out.
template <int kMode, bool kBf16>
struct TileWalk {
  const ExpertArgs& p;
  const Shape& sh;
  const int32_t* start;
  const int32_t* first;
  int t, pairs, n_tiles;
  int held;               // tiles left in `mine`
  int rest, turn;         // what is left of the tile's contraction, and a turn's share
  Tile mine;

  __device__ __forceinline__ TileWalk(const ExpertArgs& p_, const Shape& sh_, const int32_t* start_,
                                      const int32_t* first_, int pair0, int pairs_, int n_tiles_)
      : p(p_), sh(sh_), start(start_), first(first_), t(pair0), pairs(pairs_), n_tiles(n_tiles_), held(0), rest(0), turn(0) {}
  // The next tile, or the next turn of the same one, the same in all lanes (kShape: only
  // its n_mma and k_len); false after the last.
  template <bool kShape = false>
  __device__ __forceinline__ bool next(Tile& r) {
    if (rest > 0) {
      r.k_from += r.k_len;
      r.k_len = min(rest, turn);
      rest -= r.k_len;
      return true;
    }
    if (t >= n_tiles) return false;
    if (held == 0) {
      const int64_t ahead = t + (int64_t)(threadIdx.x & 31) * pairs;
      if (ahead < n_tiles) mine = decode<kMode>(p, sh, start, first, (int)ahead);
      held = 32;
      __syncwarp();
    }
    const int lane = 32 - held;
    if (!kShape) {
      r.e = __shfl_sync(0xffffffffu, mine.e, lane);
      r.z = __shfl_sync(0xffffffffu, mine.z, lane);
      r.group = __shfl_sync(0xffffffffu, mine.group, lane);
      r.m0 = __shfl_sync(0xffffffffu, mine.m0, lane);
      r.n0 = __shfl_sync(0xffffffffu, mine.n0, lane);
      r.n = __shfl_sync(0xffffffffu, mine.n, lane);
    }
    r.n_mma = __shfl_sync(0xffffffffu, mine.n_mma, lane);
    r.k_len = __shfl_sync(0xffffffffu, mine.k_len, lane);
    r.k_from = 0;
    if (r.k_len > kMaxK(kBf16)) {
      turn = (ceil_div(r.k_len, ceil_div(r.k_len, kMaxK(kBf16))) + kBlockK - 1) / kBlockK * kBlockK;
      rest = r.k_len - turn;
      r.k_len = turn;
    }
    --held;
    t += pairs;
    return true;
  }
};

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// 32 columns (`cols` of them in the matrix) of each of a warp's 32 rows (`rows`
// of them), element by element, for rows that do not start on 16-byte
// boundaries: through shared memory, so that a store's lanes are neighbours in a row.
// out: the first row's first element.
template <bool kBf16, bool kAccumulate>
__device__ __forceinline__ void put_plain(const ExpertArgs& p, uint8_t* stage, const uint32_t (&v)[32], int64_t at,
                                          int rows, int cols, bool add = false) {
  const int lane = threadIdx.x & 31;
  float* const part = reinterpret_cast<float*>(stage);      // 16 rows of 33 floats
  // what is added to, all rows' loads in flight (one after the other: 27 us a tile)
  uint32_t old[32];                                         // as they are: a conversion here would wait for its load
  if ((kAccumulate || add) && lane < cols) {
#pragma unroll
    for (int r = 0; r < 32; ++r) {
      const int64_t i = at + min(r, rows - 1) * p.out_ld + lane;
      if constexpr (kBf16) old[r] = static_cast<const uint16_t*>(p.out)[i];
      else old[r] = static_cast<const uint32_t*>(p.out)[i];
    }
  }
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    __syncwarp();
    if ((lane >> 4) == h) {
#pragma unroll
      for (int c = 0; c < 32; ++c) part[(lane & 15) * 33 + c] = __uint_as_float(v[c]);
    }
    __syncwarp();
    if (lane >= cols) continue;
#pragma unroll
    for (int r = 0; r < 16; ++r) {
      if (16 * h + r >= rows) break;
      float x = part[r * 33 + lane];
      if (kAccumulate || add) x += __uint_as_float(kBf16 ? old[16 * h + r] << 16 : old[16 * h + r]);
      const int64_t i = at + (16 * h + r) * p.out_ld + lane;
      if constexpr (kBf16) static_cast<__nv_bfloat16*>(p.out)[i] = __float2bfloat16_rn(x);
      else static_cast<float*>(p.out)[i] = x;
    }
  }
}

// `bytes` of zeros (of elements of `esz`), by the epilogue's threads, in words of 16 bytes
// but for the ends.
__device__ __forceinline__ void put_zeros(uint8_t* to, int64_t bytes, int esz) {
  const int tid = threadIdx.x - 32 * kFirstEpiWarp;
  if (bytes <= 0) return;
  const int64_t head = min((int64_t)(16 - (reinterpret_cast<uintptr_t>(to) & 15)) & 15, bytes);
  const int64_t words = (bytes - head) / 16, tail = head + 16 * words;
  for (int64_t i = tid; i < words; i += 32 * kEpiWarps)
    __stcs(reinterpret_cast<uint4*>(to + head) + i, make_uint4(0, 0, 0, 0));
  // fewer than 16 bytes at each end: a thread an element
  const int64_t at = tid < 8 ? (int64_t)tid * esz : tail + (int64_t)(tid - 8) * esz;
  if (tid < 16 && at < (tid < 8 ? head : bytes)) {
    if (esz == 2) *reinterpret_cast<uint16_t*>(to + at) = 0;
    else *reinterpret_cast<uint32_t*>(to + at) = 0;
  }
}

// 128 bytes of each of a warp's 32 rows (64 bf16 or 32 fp32 columns, `x` on,
// of rows `y` on of matrix `z`), lane l holding row l's in `w`.  The rows go, 16 at a
// time, through the warp's two 2 KB of shared memory, out by tensor copies, which
// leave out what lies past the matrix (`rows` rows are left in it) and take the
// writes off the warp: with its own stores, of whole lines, the epilogue took
// 3800 cycles a tile of 2300 cycles of MMAs; with each lane's to its own row
// 5000.  Chunk c of row r sits at c ^ (r & 7), the copy's swizzle.
__device__ __forceinline__ void put_rows(uint8_t* stage, const uint32_t (&w)[32], const CUtensorMap* map, int x, int y,
                                         int z, int rows, uint32_t& parts, bool add = false) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    if (16 * h >= rows) break;
    uint8_t* const part = stage + (parts++ & 1) * kPartBytes(kExpertWeightGrad);
    if (lane == 0) ptx::bulk_wait_read<1>();           // the copy before the last has left this part
    __syncwarp();
    if ((lane >> 4) == h) {
#pragma unroll
      for (int c = 0; c < 8; ++c)
        *reinterpret_cast<uint4*>(part + (lane & 15) * 128 + ((c ^ (lane & 7)) << 4)) =
            make_uint4(w[4 * c], w[4 * c + 1], w[4 * c + 2], w[4 * c + 3]);
      ptx::fence_proxy_async_smem();
    }
    __syncwarp();
    if (lane == 0) {
      if (add) ptx::tma_add_3d(map, ptx::smem_u32(part), x, y + 16 * h, z);
      else ptx::tma_store_3d(map, ptx::smem_u32(part), x, y + 16 * h, z);
      ptx::bulk_commit();
    }
  }
}
// The way back, in two steps: 128 bytes of each of a warp's 32 rows (`rows` and
// `chunks` of 16 bytes of them in the matrix) on their way into `buf`, which nothing waits for
// here; and each lane's row from there.
constexpr int kFetchBytes = 32 * 128;
constexpr int kFetches = 2;                            // of a warp, ahead of the one it adds
__device__ __forceinline__ void fetch_rows(uint8_t* buf, const uint8_t* in, int64_t pitch, int rows, int chunks) {
  const int lane = threadIdx.x & 31, c = lane & 7;
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const int r = 4 * k + (lane >> 3);
    if (r < rows && c < chunks)
      ptx::copy_async_16(ptx::smem_u32(buf) + r * 128 + ((c ^ (r & 7)) << 4), in + r * pitch + 16 * c);
  }
}
__device__ __forceinline__ void fetched_row(const uint8_t* buf, uint32_t (&w)[32]) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int c = 0; c < 8; ++c) {
    const uint4 v = *reinterpret_cast<const uint4*>(buf + lane * 128 + ((c ^ (lane & 7)) << 4));
    w[4 * c] = v.x; w[4 * c + 1] = v.y; w[4 * c + 2] = v.z; w[4 * c + 3] = v.w;
  }
}

// Adds the columns at `before` of the other accumulator, the sum of a tile's earlier turns
// (16 at a time, for the registers).
template <int kN>
__device__ __forceinline__ void add_before(uint32_t before, uint32_t (&r)[kN]) {
#pragma unroll
  for (int h = 0; h < kN; h += 16) {
    uint32_t b[16];
    ptx::tmem_get_32x32b_x16(before + h, b);
#pragma unroll
    for (int k = 0; k < 16; ++k) r[h + k] = __float_as_uint(__uint_as_float(r[h + k]) + __uint_as_float(b[k]));
  }
}

// One chunk of a weight gradient's rows from the accumulator at `taddr`: 64
// columns to bf16 (`sum`: with those at `before` added), or 32 to fp32; kAccumulate: added to
// `w`, what is there.  `last`: then hands the accumulator back.
template <bool kBf16, bool kAccumulate, typename Release>
__device__ __forceinline__ void put_chunk(const CUtensorMap* map, uint8_t* stage, uint32_t (&w)[32], uint32_t taddr,
                                          uint32_t before, bool sum, int x, int y, int z, int rows, uint32_t& parts,
                                          bool add, bool last, Release release) {
  uint32_t acc[32];
#pragma unroll
  for (int h = 0; h < (kBf16 ? 2 : 1); ++h) {
    ptx::tmem_ld_32x32b_x32(taddr + 32 * h, acc);
    ptx::tmem_ld_wait();
    if (kBf16 && sum) add_before(before + 32 * h, acc);
    if (last && h == (kBf16 ? 1 : 0)) release();
#pragma unroll
    for (int k = 0; k < (kBf16 ? 16 : 32); ++k) {
      if constexpr (kBf16) {
        float a = __uint_as_float(acc[2 * k]), b = __uint_as_float(acc[2 * k + 1]);
        if constexpr (kAccumulate) {
          a += bf16_lo(w[16 * h + k]);
          b += bf16_hi(w[16 * h + k]);
        }
        const __nv_bfloat162 q = __floats2bfloat162_rn(a, b);
        w[16 * h + k] = *reinterpret_cast<const uint32_t*>(&q);
      } else {
        w[k] = kAccumulate && !add ? __float_as_uint(__uint_as_float(acc[k]) + __uint_as_float(w[k])) : acc[k];
      }
    }
  }
  put_rows(stage, w, map, x, y, z, rows, parts, !kBf16 && add);
}

// 32 tokens (`cnt` of them the group's) of a warp's 32 rows of M, lane l holding
// row l's in `r`: 64 or 128 bytes of each token's row of Y.  Whole pieces of 1 KB (16
// tokens, or 8 in fp32) go through shared memory and out by tensor copies, off
// the warp's path (2700 cycles a chunk with its own 2-byte stores); the last tokens
// of a group, whose neighbours are another's, and layouts whose rows do not start
// on 16-byte boundaries, by stores.
template <bool kBf16, bool kVec>
__device__ __forceinline__ void put_tokens(const ExpertArgs& p, const CUtensorMap* map, uint8_t* stage,
                                           const uint32_t (&r)[32], int row0, int rows, int token, int cnt,
                                           uint32_t& parts, bool add) {
  constexpr int kPiece = kBf16 ? 16 : 8;
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int q = 0; q < 32 / kPiece; ++q) {
    if (q * kPiece >= cnt) break;
    if (kVec && (q + 1) * kPiece <= cnt) {
      uint8_t* const part = stage + (parts++ & 1) * kPartBytes(kExpertForward);
      if (lane == 0) ptx::bulk_wait_read<1>();         // the copy before the last has left this part
      __syncwarp();
#pragma unroll
      for (int j = 0; j < kPiece; ++j) {
        const float x = __uint_as_float(r[q * kPiece + j]);
        if constexpr (kBf16) reinterpret_cast<__nv_bfloat16*>(part)[32 * j + lane] = __float2bfloat16_rn(x);
        else reinterpret_cast<float*>(part)[32 * j + lane] = x;
      }
      ptx::fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        if (!kBf16 && add) ptx::tma_add_3d(map, ptx::smem_u32(part), row0, token + q * kPiece, 0);
        else ptx::tma_store_3d(map, ptx::smem_u32(part), row0, token + q * kPiece, 0);
        ptx::bulk_commit();
      }
    } else if (lane < rows) {
      const int64_t at = (int64_t)(token + q * kPiece) * p.out_ld + row0 + lane;
#pragma unroll
      for (int j = 0; j < kPiece; ++j) {
        if (q * kPiece + j >= cnt) break;
        const float x = __uint_as_float(r[q * kPiece + j]);
        if constexpr (kBf16) static_cast<__nv_bfloat16*>(p.out)[at + j * p.out_ld] = __float2bfloat16_rn(x);
        else {
          float* const o = static_cast<float*>(p.out) + at + j * p.out_ld;
          *o = add ? x + *o : x;
        }
      }
    }
  }
}

// kBf16: the output's type.  kVec: its rows start on 16-byte boundaries.
// kAccumulate: a weight gradient that adds to what is there, fetched while the products
// run, at the price of two stages.  (128 x 1408 x 2048, 32768 tokens, us: bf16 300, fp32
// 463, floors 250 and 468; with loads where the sum is made 452 and 810; tensor copies that
// add in fp32 545.)
template <int kMode, bool kBf16, bool kAccumulate, bool kVec>
__global__ void __launch_bounds__(kThreads, 1) expert_kernel(const __grid_constant__ ExpertArgs p,
                                                             const __grid_constant__ Maps maps) {
  constexpr bool kWgrad = kMode == kExpertWeightGrad;
  constexpr bool kAmn = kMode != kExpertForward;
  extern __shared__ uint8_t smem_raw[];
  // first token (clamped) and first tile of each expert (weight gradient: of a split one)
  constexpr int kListed = kWgrad ? kSplitPairs / 2 : MFSDP_MAX_EXPERTS;
  __shared__ int32_t start[kListed + 1], first[kListed + 1];
  __shared__ int32_t widest;                            // columns of the launch's widest tile
  __shared__ __align__(8) uint64_t full_bar[kMaxStages];    // even CTA: both CTAs' operands have landed
  __shared__ __align__(8) uint64_t empty_bar[kMaxStages];
  __shared__ __align__(8) uint64_t tfull_bar[2], tempty_bar[2], drain_bar;
  __shared__ uint32_t tmem_slot;
  __shared__ int abort_flag;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = ptx::cluster_ctarank();
  const uint32_t smem_base = (ptx::smem_u32(smem_raw) + 1023u) & ~1023u;
  const int n_rows = (int)p.n_rows;

  Shape sh;
  sh.m = (int)(kMode == kExpertInputGrad ? p.cols : p.rows);
  sh.tiles_m = ceil_div(sh.m, kPairM);
  sh.n = (int)p.cols;
  sh.tiles_n = ceil_div(sh.n, kMaxN);
  sh.width_n = even_width(sh.n, sh.tiles_n, 64);       // whole chunks of the epilogue, which writes them whole

  const bool listed = !kWgrad || p.chunk > 0;
  sh.chunk = kWgrad && listed ? find_chunks(p.starts, p.n_experts, n_rows, p.chunk, p.slots, 0).chunk : 0;
  if (listed)
    for (int i = threadIdx.x; i <= p.n_experts; i += kThreads) start[i] = start_of(p, i);
  if (warp == 1) {
    ptx::tmem_alloc_pair(ptx::smem_u32(&tmem_slot), kTmemCols);
    ptx::tmem_relinquish_pair();
  }
  if (threadIdx.x == 0) {
    for (int s = 0; s < kMaxStages; ++s) {
      ptx::mbar_init(ptx::smem_u32(&full_bar[s]), 1);
      ptx::mbar_init(ptx::smem_u32(&empty_bar[s]), 1);
    }
    for (int a = 0; a < 2; ++a) {
      ptx::mbar_init(ptx::smem_u32(&tfull_bar[a]), 1);
      ptx::mbar_init(ptx::smem_u32(&tempty_bar[a]), 2 * kEpiWarps);
    }
    ptx::mbar_init(ptx::smem_u32(&drain_bar), 1);
    abort_flag = 0;
    // No wait of this launch can have run out yet (2 s at least), so nothing
    // recorded is lost here.
    if (blockIdx.x == 0) *p.status = 0;
    ptx::fence_barrier_init();
    ptx::fence_proxy_async_smem();
  }
  __syncthreads();
  if (warp == 0 && listed) {
    // tiles before each expert, and the widest tile
    int base = 0, wide = kStepN;
    for (int e0 = 0; e0 < p.n_experts; e0 += 32) {
      const int e = e0 + lane;
      const int len = e < p.n_experts ? max(0, start[e + 1] - start[e]) : 0;
      const int nt = ceil_div(len, kMaxN);
      if (nt) wide = max(wide, even_width(len, nt));
      int sum = kWgrad ? chunks_of(len, sh.chunk) * sh.tiles_m * sh.tiles_n : nt * sh.tiles_m;
      if (e >= p.n_experts) sum = 0;
      const int own = sum;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, sum, o);
        if (lane >= o) sum += v;
      }
      if (e < p.n_experts) first[e] = base + sum - own;
      base += __shfl_sync(0xffffffffu, sum, 31);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) wide = max(wide, __shfl_xor_sync(0xffffffffu, wide, o));
    if (lane == 0) {
      first[p.n_experts] = base;
      widest = wide;
    }
  }
  ptx::tc_fence_before();
  ptx::cluster_sync();
  ptx::tc_fence_after();
  const uint32_t tmem_base = tmem_slot;
  const Abort ab{&abort_flag, p.status, p.wait_limit_ns};
  // Packed operands come from the kernel before this one.  Padded ends too, but the
  // producers wait for those at the first one they meet (where there is none, that kernel
  // has nothing to do): 25.6 and 24.5 us for 8 groups of 285.
  if (!p.only_ends) {
    ptx::wait_dependencies();
    ptx::fence_proxy_async_global();
  }
  const int n_tiles = listed ? first[p.n_experts] : p.n_experts * sh.tiles_m * sh.tiles_n;
  TileWalk<kMode, kBf16> walk(p, sh, start, first, blockIdx.x >> 1, gridDim.x >> 1, n_tiles);
  Tile tl;
  // Shared memory of a stage: A, then this CTA's half of B.
  const int wide = kWgrad ? sh.width_n : widest;
  const uint32_t stage_bytes = kBytesA + (kWgrad ? ceil_div(wide / 2, 64) * kMnBlock : rows_b(wide / 2) * 128);
  const int stages = min(kMaxStages, kRingBytes(kMode, kAccumulate) / (int)stage_bytes);

  if (warp == 0) {
    // -------------------------------------------------------------- producer
    // The whole warp runs the loop on warp-uniform values and one elected lane
    // issues: with the loop inside one lane, every copy took 100-170 cycles to
    // issue and the issue bound the kernel.
    const uint32_t rank_u = uniform(rank), base_u = uniform(smem_base);
    const uint32_t full0 = uniform(ptx::smem_u32(&full_bar[0])), empty0 = uniform(ptx::smem_u32(&empty_bar[0]));
    const uint32_t pair_full0 = uniform(ptx::mapa_shared(full0, 0));
    if (n_rows > 0 && ptx::elect_one()) {
      ptx::prefetch_tensormap(&maps.a);
      ptx::prefetch_tensormap(&maps.b);
      ptx::prefetch_tensormap(&maps.c);
    }
    __syncwarp();
    uint32_t s = 0, use = 0;
    bool ok = true, ends_there = !kWgrad || !p.only_ends;
    while (walk.next(tl)) {
      const int blocks = blocks_of<kWgrad>(tl.k_len);
      if (!ends_there && (tl.k_len & (kEnd - 1)) != 0) {
        ptx::wait_dependencies();
        ptx::fence_proxy_async_global();
        ends_there = true;
      }
      const int nh = tl.n_mma >> 1;                         // this CTA's columns of B
      const int mc = tl.m0 + (int)rank_u * kCtaM;
      // rows wholly past the matrix are not loaded (their output is not stored)
      const bool a_in = mc < sh.m;
      const int copies_b = ceil_div(nh, 64);                // weight gradient
      const uint32_t rows = rows_b(nh), bytes_b = kWgrad ? copies_b * kMnBlock : rows * 128;
      const uint32_t pair_bytes = (tl.m0 + kCtaM < sh.m ? 2u : 1u) * kBytesA + 2u * bytes_b;
      const bool ragged = kWgrad && (tl.k_len & (kEnd - 1)) != 0;
      const int nc = tl.n0 + (int)rank_u * nh;
      for (int kb = 0; kb < blocks; kb += kTurn) {
        const int turn = min(kTurn, blocks - kb);
        const uint32_t s1 = s + 1 == (uint32_t)stages ? 0 : s + 1, use1 = s1 == 0 ? use + 1 : use;
        if (ptx::elect_one()) {
#pragma unroll
          for (int h = 0; h < kTurn; ++h) {
            if (h >= turn) break;
            const uint32_t slot = h == 0 ? s : s1, slot_use = h == 0 ? use : use1;
            // after a wait that gave up, the leader issues nothing more
            ok = ok && wait_bar<false>(empty0 + 8 * slot, (slot_use & 1) ^ 1, ab, kRoleStage);
            if (!ok) break;
            const uint32_t sa = base_u + slot * stage_bytes, sb = sa + kBytesA, bar = pair_full0 + 8 * slot;
            const int k0 = tl.k_from + (kb + h) * kBlockK;
            const bool last = ragged && kb + h == blocks - 1;       // 16 rows: a quarter of the bytes
            if (rank_u == 0)
              ptx::mbar_arrive_expect_tx(full0 + 8 * slot, last ? pair_bytes * kEnd / kBlockK : pair_bytes);
            if (a_in) {
              if (!kAmn) {
                ptx::tma_load_3d_pair(sa, &maps.a, k0, mc, tl.e, bar);
              } else {
                const CUtensorMap* map = last ? &maps.c : &maps.a;
                const int y = last ? tl.e * kEnd : (kWgrad ? tl.group + k0 : k0), z = kWgrad ? 0 : tl.e;
                ptx::tma_load_3d_pair(sa, map, mc, y, z, bar);
                ptx::tma_load_3d_pair(sa + kMnBlock, map, mc + 64, y, z, bar);
              }
            }
            if (kWgrad) {
              const CUtensorMap* map = last ? &maps.d : &maps.b;
              const int y = last ? tl.e * kEnd : tl.group + k0;
              ptx::tma_load_3d_pair(sb, map, nc, y, 0, bar);
              if (copies_b > 1) ptx::tma_load_3d_pair(sb + kMnBlock, map, nc + 64, y, 0, bar);
            } else {
              load_tokens(maps, sb, rows, k0, tl.group + nc, bar);
            }
          }
        }
        if (turn > 1) { s = s1; use = use1; }
        if (++s == (uint32_t)stages) { s = 0; ++use; }
      }
    }
    __syncwarp();
    // Drain: every stage this CTA filled has been read, so no copy into its
    // shared memory is in flight (bounded).
    for (int i = 0; i < stages; ++i) {
      if (use > 0 || s > 0) {
        const uint32_t last = s == 0 ? stages - 1 : s - 1, luse = s == 0 ? use - 1 : use;
        if (!__all_sync(0xffffffffu, ptx::mbar_wait(empty0 + 8 * last, luse & 1, kDrainNs))) break;
        s = last;
        use = luse;
      }
    }
  } else if (warp == 1) {
    if (rank == 0) {
      // ----------------------------------------------------------- MMA issuer
      const uint32_t base_u = uniform(smem_base), tmem_u = uniform(tmem_base);
      const uint32_t full0 = uniform(ptx::smem_u32(&full_bar[0])), empty0 = uniform(ptx::smem_u32(&empty_bar[0]));
      const uint32_t tfull0 = uniform(ptx::smem_u32(&tfull_bar[0])), tempty0 = uniform(ptx::smem_u32(&tempty_bar[0]));
      uint32_t s = 0, use = 0, acc_it = 0;
      bool ok = true;
      while (walk.template next<true>(tl)) {
        const int blocks = blocks_of<kWgrad>(tl.k_len);
        if (blocks == 0) continue;
        const bool ragged = kWgrad && (tl.k_len & (kEnd - 1)) != 0;
        const uint32_t a = acc_it & 1, acc_parity = ((acc_it >> 1) & 1) ^ 1;
        const uint32_t d_tmem = tmem_u + a * kAccCols;
        const uint32_t idesc = ptx::idesc_bf16_f32(kPairM, (uint32_t)tl.n_mma, kWgrad ? 1u : 0u, kAmn ? 1u : 0u);
        for (int kb = 0; kb < blocks; kb += kTurn) {
          const int turn = min(kTurn, blocks - kb);
          const uint32_t s1 = s + 1 == (uint32_t)stages ? 0 : s + 1, use1 = s1 == 0 ? use + 1 : use;
          if (ptx::elect_one()) {
            if (kb == 0) ok = ok && wait_bar<true>(tempty0 + 8 * a, acc_parity, ab, kRoleAccFree);
#pragma unroll
            for (int h = 0; h < kTurn; ++h) {
              if (h >= turn) break;
              const uint32_t slot = h == 0 ? s : s1, slot_use = h == 0 ? use : use1;
              ok = ok && wait_bar<true>(full0 + 8 * slot, slot_use & 1, ab, kRoleOperands);
              if (!ok) break;
              ptx::tc_fence_after();
              // K-major: 16 elements (32 bytes) along the swizzle row, 8-row groups
              // 1 KB apart.  MN-major: 16 K rows (2 KB), 64-element blocks 8 KB
              // apart (leading offset), 8-row K groups 1 KB apart (stride offset).
              const uint32_t sa = base_u + slot * stage_bytes;
              const uint64_t adesc = ptx::smem_desc_sw128(sa, kAmn ? kMnBlock : 16, 1024);
              const uint64_t bdesc = ptx::smem_desc_sw128(sa + kBytesA, kWgrad ? kMnBlock : 16, 1024);
              // K-major operands past the contraction's end are zeros of the copy's fill
              const int left = tl.k_len - (kb + h) * kBlockK;
              const int steps = ragged && kb + h == blocks - 1
                                    ? 1
                                    : min(kBlockK / 16, kWgrad ? left / 16 : ceil_div(left, 16));
#pragma unroll
              for (int k = 0; k < kBlockK / 16; ++k)
                if (k < steps)
                  ptx::umma_bf16_pair(d_tmem, adesc + k * (kAmn ? 2048 >> 4 : 32 >> 4),
                                      bdesc + k * (kWgrad ? 2048 >> 4 : 32 >> 4), idesc,
                                      kb + h > 0 || k > 0 ? 1u : 0u);
              ptx::umma_commit_pair_multicast(empty0 + 8 * slot, 0x3);
            }
            if (ok && kb + turn == blocks) ptx::umma_commit_pair_multicast(tfull0 + 8 * a, 0x3);
          }
          if (turn > 1) { s = s1; use = use1; }
          if (++s == (uint32_t)stages) { s = 0; ++use; }
        }
        ++acc_it;
      }
      // every MMA issued has completed before TMEM is released
      __syncwarp();
      if (ptx::elect_one()) ptx::umma_commit_pair_multicast(ptx::smem_u32(&drain_bar), 0x1);
      __syncwarp();
      ptx::mbar_wait(ptx::smem_u32(&drain_bar), 0, kDrainNs);
    }
  } else if (warp >= kFirstEpiWarp) {
    // -------------------------------------------------------------- epilogue
    // Warp w reads TMEM lane quadrant w % 4; the two warps of a quadrant take
    // alternate chunks of 32 columns.
    const int quad = warp & 3, half = (warp - kFirstEpiWarp) >> 2;
    uint8_t* const stage = smem_raw + (smem_base - ptx::smem_u32(smem_raw)) + kRingBytes(kMode, kAccumulate) +
                           (warp - kFirstEpiWarp) * 2 * kPartBytes(kMode);
    constexpr int kEsz = kBf16 ? 2 : 4;
    constexpr int kWidth = kWgrad && kVec ? 128 / kEsz : 32;     // columns of a chunk
    uint32_t acc_it = 0, parts = 0;
    // With kAccumulate what the output holds is fetched ahead, chunk by chunk in the order
    // in which they are added to, from the coming tiles too.
    struct Fetch {
      Tile tl;
      int c;
      bool more;
      uint32_t made, taken;
    } fetch{};
    uint8_t* const fetch_buf = smem_raw + (smem_base - ptx::smem_u32(smem_raw)) + kRingBytes(kMode, kAccumulate) +
                               kEpiWarps * 2 * kPartBytes(kMode) + (warp - kFirstEpiWarp) * kFetches * kFetchBytes;
    TileWalk<kMode, kBf16> ahead = walk;
    auto fetch_next = [&]() {
      fetch.c += 2 * kWidth;
      while (fetch.more && fetch.c >= fetch.tl.n_mma) {
        do fetch.more = ahead.next(fetch.tl);
        while (fetch.more && (fetch.tl.k_len == 0 || fetch.tl.k_from > 0));
        fetch.c = kWidth * half;
      }
      if (fetch.more) {
        const int y = fetch.tl.m0 + (int)rank * kCtaM + quad * 32, x = fetch.tl.n0 + fetch.c;
        fetch_rows(fetch_buf + (fetch.made & 1) * kFetchBytes,
                   static_cast<const uint8_t*>(p.out) + (fetch.tl.z * p.out_stride + y * p.out_ld + x) * kEsz,
                   p.out_ld * kEsz, sh.m - y, min(8, (fetch.tl.n - fetch.c) * kEsz / 16));
      }
      ptx::copy_async_commit();
      ++fetch.made;
    };
    if constexpr (kAccumulate && kVec) {
      fetch.tl.n_mma = 0;
      fetch.c = 0;
      fetch.more = true;
      fetch.made = fetch.taken = 0;
      for (int k = 0; k < kFetches; ++k) fetch_next();
    }
    while (walk.next(tl)) {
      const int row0 = tl.m0 + (int)rank * kCtaM + quad * 32;
      const int64_t at0 = kWgrad ? tl.z * p.out_stride + row0 * p.out_ld + tl.n0 : 0;      // the warp's first row
      if (kWgrad && tl.k_len == 0) {
        if (p.accumulate) continue;
        if constexpr (kVec) {
          uint32_t z[32];
#pragma unroll
          for (int j = 0; j < 32; ++j) z[j] = 0;
          for (int c = kWidth * half; c < tl.n; c += 2 * kWidth)
            put_rows(stage, z, &maps.out, tl.n0 + c, row0, tl.z, sh.m - row0, parts);
        } else if (tl.n0 == 0) {
          // this CTA's rows, all their columns: they lie in one piece
          const int first_row = tl.m0 + (int)rank * kCtaM;
          put_zeros(static_cast<uint8_t*>(p.out) + (tl.z * p.out_stride + first_row * p.out_ld) * kEsz,
                    (int64_t)min(kCtaM, sh.m - first_row) * p.out_ld * kEsz, kEsz);
        }
        continue;
      }
      const uint32_t a = acc_it & 1;
      if (!__all_sync(0xffffffffu, wait_bar<false>(ptx::smem_u32(&tfull_bar[a]), (acc_it >> 1) & 1, ab, kRoleAccFull)))
        break;
      ptx::tc_fence_after();
      const uint32_t t_lane = tmem_base + ((uint32_t)(quad * 32) << 16);
      const uint32_t t_row = t_lane + a * kAccCols, t_before = t_lane + (a ^ 1) * kAccCols;
      // A bf16 output's turns: the sum of the earlier ones stands in the other accumulator,
      // whose turn to be filled comes next, and moves to this one.
      const bool sum = kBf16 && tl.k_from > 0;
      // this warp's reads of the accumulators are done: hand them back
      auto hand_back = [&](bool this_one, bool before) {
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          if (before) ptx::mbar_arrive_signal(ptx::mapa_shared(ptx::smem_u32(&tempty_bar[a ^ 1]), 0));
          if (this_one) ptx::mbar_arrive_signal(ptx::mapa_shared(ptx::smem_u32(&tempty_bar[a]), 0));
        }
      };
      auto release = [&]() { hand_back(true, sum); };
      if (kWidth * half >= tl.n_mma) {                    // no chunk for this warp
        hand_back(true, false);
      } else if (kBf16 && walk.rest > 0) {
        if (sum) {
          for (int c = kWidth * half; c < tl.n_mma; c += 2 * kWidth)
#pragma unroll
            for (int h = 0; h < kWidth; h += 16) {
              uint32_t r[16];
              ptx::tmem_get_32x32b_x16(t_row + (uint32_t)(c + h), r);
              add_before(t_before + (uint32_t)(c + h), r);
              ptx::tmem_put_32x32b_x16(t_row + (uint32_t)(c + h), r);
            }
          hand_back(false, true);
        }
      }
      if (kBf16 && walk.rest > 0) {
        ++acc_it;
        continue;
      }
      const bool add = !kBf16 && tl.k_from > 0;
      if (kVec && !kBf16 && tl.k_from > 0) {               // what the last turn wrote is there
        if (lane == 0) ptx::bulk_wait_all();
        __syncwarp();
      }
      for (int c = kWidth * half; c < tl.n_mma; c += 2 * kWidth) {
        const bool last = c + 2 * kWidth >= tl.n_mma;
        __syncwarp();
        if constexpr (kWgrad && kVec) {
          uint32_t w[32];
          if (kAccumulate && !add) {
            ptx::copy_async_wait<kFetches - 1>();
            __syncwarp();
            fetched_row(fetch_buf + (fetch.taken++ & 1) * kFetchBytes, w);
            __syncwarp();
            fetch_next();
          }
          put_chunk<kBf16, kAccumulate>(&maps.out, stage, w, t_row + c, t_before + c, sum, tl.n0 + c, row0, tl.z,
                                        sh.m - row0, parts, add, last, release);
          continue;
        }
        uint32_t r[32];
        ptx::tmem_ld_32x32b_x32(t_row + (uint32_t)c, r);
        ptx::tmem_ld_wait();
        if (sum) add_before(t_before + (uint32_t)c, r);
        if (last) release();
        if constexpr (kWgrad) {
          put_plain<kBf16, kAccumulate>(p, stage, r, at0 + c, sh.m - row0, tl.n - c, add);
        } else {
          if (row0 < sh.m)
            put_tokens<kBf16, kVec>(p, &maps.out, stage, r, row0, sh.m - row0, tl.group + tl.n0 + c, tl.n - c,
                                    parts, add);
        }
      }
      ++acc_it;
    }
    if (kVec && lane == 0) ptx::bulk_wait_all();
    if (!kWgrad) {
      // rows of no expert
      const int64_t lo = start[p.n_experts], width = sh.m;
      const int64_t step = (int64_t)gridDim.x * (32 * kEpiWarps);
      for (int64_t i = (int64_t)blockIdx.x * (32 * kEpiWarps) + threadIdx.x - 32 * kFirstEpiWarp;
           i < (n_rows - lo) * width; i += step) {
        const int64_t at = (lo + i / width) * p.out_ld + i % width;
        if constexpr (kBf16) static_cast<uint16_t*>(p.out)[at] = 0;
        else static_cast<float*>(p.out)[at] = 0.f;
      }
    }
  }

  // No CTA of the pair leaves, or frees TMEM, while its peer may still arrive
  // on its barriers.
  __syncwarp();
  ptx::tc_fence_before();
  ptx::cluster_sync();
  if (warp == 1) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc_pair(tmem_base, kTmemCols);
  }
}

// Adds up a split weight gradient: dW_e (+)= the sum of its chunks, in their order.  An
// item is 128 elements of a matrix, four a lane.  A warp adds the chunks of an item; where
// there are many, the warps of a CTA take an eighth of them each.
constexpr int kSumWarps = 8;
constexpr int kFewChunks = 16;

template <bool kBf16>
__device__ __forceinline__ void put_sum(const ChunkSumArgs& a, int e, int64_t q, const float4& acc) {
  const int64_t quads = a.part_ld / 4, r = q / quads, c = (q - r * quads) * 4;
  const int64_t at = e * a.out_stride + r * a.out_ld + c;
  const float v[4] = {acc.x, acc.y, acc.z, acc.w};
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    if (c + k >= a.cols) break;
    if constexpr (kBf16) {
      __nv_bfloat16* o = static_cast<__nv_bfloat16*>(a.out) + at + k;
      *o = __float2bfloat16_rn(a.accumulate ? v[k] + __bfloat162float(*o) : v[k]);
    } else {
      float* o = static_cast<float*>(a.out) + at + k;
      *o = a.accumulate ? v[k] + *o : v[k];
    }
  }
}

template <bool kBf16>
__global__ void __launch_bounds__(32 * kSumWarps) sum_chunks_kernel(const __grid_constant__ ChunkSumArgs a) {
  __shared__ float4 sums[kSumWarps][32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, e = blockIdx.y;
  const Chunks my = find_chunks(a.starts, a.experts, (int)a.n_rows, a.chunk, a.slots, e);
  const int64_t size = a.rows * a.part_ld, quads = size / 4;
  const float* part = a.parts + my.before * size;
  auto add = [&](int64_t q, int lo, int hi) {
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
    for (int c = lo; c < hi; ++c) {
      const float4 x = *reinterpret_cast<const float4*>(part + c * size + 4 * q);
      acc.x += x.x; acc.y += x.y; acc.z += x.z; acc.w += x.w;
    }
    return acc;
  };
  ptx::wait_dependencies();
  if (my.mine <= kFewChunks) {
    for (int64_t q = ((int64_t)blockIdx.x * kSumWarps + warp) * 32 + lane; q < quads;
         q += (int64_t)gridDim.x * kSumWarps * 32)
      put_sum<kBf16>(a, e, q, add(q, 0, my.mine));
    return;
  }
  for (int64_t q0 = (int64_t)blockIdx.x * 32; q0 < quads; q0 += (int64_t)gridDim.x * 32) {
    const int64_t q = q0 + lane;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    if (q < quads) acc = add(q, my.mine * warp / kSumWarps, my.mine * (warp + 1) / kSumWarps);
    __syncthreads();
    sums[warp][lane] = acc;
    __syncthreads();
    if (warp != 0 || q >= quads) continue;
#pragma unroll
    for (int w = 1; w < kSumWarps; ++w) {
      const float4 x = sums[w][lane];
      acc.x += x.x; acc.y += x.y; acc.z += x.z; acc.w += x.w;
    }
    put_sum<kBf16>(a, e, q, acc);
  }
}

// What a call prepares for its tensor copies, in one launch: copies of operands whose
// rows do not start on 16-byte boundaries (`rows` rows of `width` elements, ld apart,
// of each of n matrices `stride` apart, into rows of width8 elements, zero-filled; a
// matrix without tokens is left out), and the padded ends of the groups (rows 16 e ..
// 16 e + 15: the last len % 16 rows of group e, then zeros; a length that is a multiple
// of 16 needs none).
struct PrepareJob {
  const uint16_t* src;
  uint16_t* dst;
  int64_t ld, stride, rows;
  int32_t width, width8, n;
  int32_t ends;            // 1: the groups' ends
  int32_t of_experts;      // 1: the n matrices are the experts'
  int32_t block0, per;     // first block of the job, blocks of a matrix
};
struct PrepareArgs {
  PrepareJob job[4];
  int32_t jobs;
  int32_t blocks;
  const int32_t* starts;
  int64_t n_rows;
};
constexpr int kPrepareThreads = 256;

// 8 elements from column c of a row of `width`, zero past it.  Inside a row that does not
// start on a 16-byte boundary (not `vec`) they come out of the two 16-byte words that hold
// them, which lie in the row; at its ends one by one.  (30776 x 1097 copied and multiplied:
// 48 us with single elements everywhere, 42 so.)
__device__ __forceinline__ uint4 load8(const uint16_t* row, int c, int width, bool vec) {
  if (vec) return *reinterpret_cast<const uint4*>(row + c);
  uint32_t w[8];
  if (c >= 8 && c + 16 <= width) {
    const uintptr_t at = reinterpret_cast<uintptr_t>(row + c);
    const uint4* const words = reinterpret_cast<const uint4*>(at & ~(uintptr_t)15);
    const uint4 a = words[0], b = words[1];
    w[0] = a.x; w[1] = a.y; w[2] = a.z; w[3] = a.w;
    w[4] = b.x; w[5] = b.y; w[6] = b.z; w[7] = b.w;
    const bool by1 = at & 4, by2 = at & 8;
#pragma unroll
    for (int k = 0; k < 7; ++k) w[k] = by1 ? w[k + 1] : w[k];
#pragma unroll
    for (int k = 0; k < 5; ++k) w[k] = by2 ? w[k + 2] : w[k];
    const uint32_t shift = at & 2 ? 16 : 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) w[k] = __funnelshift_r(w[k], w[k + 1], shift);
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const uint32_t x = c + 2 * k < width ? row[c + 2 * k] : 0, y = c + 2 * k + 1 < width ? row[c + 2 * k + 1] : 0;
    w[k] = x | (y << 16);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

__global__ void __launch_bounds__(kPrepareThreads) prepare_kernel(const __grid_constant__ PrepareArgs a) {
  ptx::launch_dependents();
  int k = 0;
  while (k + 1 < a.jobs && (int)blockIdx.x >= a.job[k + 1].block0) ++k;
  const PrepareJob& j = a.job[k];
  const int e = (blockIdx.x - j.block0) / j.per, part = (blockIdx.x - j.block0) - e * j.per;
  const int chunks = j.width8 >> 3, n = (int)a.n_rows;
  int lo = 0, hi = 0;
  if (j.of_experts) {
    lo = e == 0 ? 0 : min(max(a.starts[e], 0), n);
    hi = min(max(a.starts[e + 1], 0), n);
  }
  if (j.ends) {
    const int rest = max(0, hi - lo) & (kEnd - 1);
    if (rest == 0) return;
    const bool vec = j.ld % 8 == 0 && j.width % 8 == 0;
    for (int i = part * kPrepareThreads + threadIdx.x; i < kEnd * chunks; i += j.per * kPrepareThreads) {
      const int r = i / chunks, c = (i - r * chunks) * 8;
      uint4 v = make_uint4(0, 0, 0, 0);
      if (r < rest) v = load8(j.src + (int64_t)(hi - rest + r) * j.ld, c, j.width, vec);
      *reinterpret_cast<uint4*>(j.dst + ((int64_t)e * kEnd + r) * j.width8 + c) = v;
    }
    return;
  }
  if (j.of_experts && hi <= lo) return;
  const uint16_t* src = j.src + e * j.stride;
  uint16_t* dst = j.dst + (int64_t)e * j.rows * j.width8;
  const int64_t total = j.rows * chunks;
  for (int64_t i = (int64_t)part * kPrepareThreads + threadIdx.x; i < total; i += (int64_t)j.per * kPrepareThreads) {
    const int64_t r = i / chunks;
    const int c = (int)(i - r * chunks) * 8;
    *reinterpret_cast<uint4*>(dst + r * j.width8 + c) = load8(src + r * j.ld, c, j.width, false);
  }
}

// The forward product of few tokens, as serving has them: bound by reading the matrices of
// the experts that have any.  An item is one row of a matrix and up to four tokens of its
// expert: a warp's, 16 bytes of the row a lane, four such loads and the first token's in
// flight; the lanes' sums are added at the end.  No tensor memory, clusters or copies to set
// up.  Against the tensor kernel, us, of 1408 x 2048: 1 token 3.7 and 10.9; 8 of 8 experts
// 11.2 and 14.9; 8 of one 7.8 and 12.5; 16 of 16 17.8 and 24.5 (92 MB: 7 TB/s past the first
// 4 us); 16 of one 11.2 and 12.4; 32 of one would take longer.  8 loads in flight a warp and
// three CTAs an SM spill (15.2 for 8 of 8); a ring of bulk-copied rows for 8 warps took 23.6.
constexpr int kFewThreads = 256;
constexpr int kFewAhead = 4;                              // loads of 256 columns, in flight
constexpr int kFewAtOnce = 4;                             // tokens

template <bool kBf16, bool kVec>
__global__ void __launch_bounds__(kFewThreads, 4) few_tokens_kernel(const __grid_constant__ ExpertArgs p) {
  __shared__ int32_t experts[kFewTokens], tokens[kFewTokens];            // of the items, by token
  __shared__ int2 found[kFewTokens];                                     // as the threads come upon them
  __shared__ int count;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    count = 0;
    if (blockIdx.x == 0) *p.status = 0;
  }
  __syncthreads();
  for (int e = threadIdx.x; e < p.n_experts; e += kFewThreads) {
    const int hi = start_of(p, e + 1);
    for (int t = start_of(p, e); t < hi; t += kFewAtOnce) {
      const int at = atomicAdd(&count, 1);
      if (at < kFewTokens) found[at] = make_int2(e, t);
    }
  }
  __syncthreads();
  // every CTA needs them in the same order: its rows are a share of the whole list
  if ((int)threadIdx.x < min(count, kFewTokens)) {
    const int2 mine = found[threadIdx.x];
    int at = 0;
    for (int k = 0; k < min(count, kFewTokens); ++k)
      at += found[k].y < mine.y || (found[k].y == mine.y && found[k].x < mine.x);
    experts[at] = mine.x;
    tokens[at] = mine.y;
  }
  __syncthreads();
  const int rows = (int)p.rows, cols = (int)p.cols;
  const int items = min(count, kFewTokens) * rows;       // (at most 16 * 2^24)
  const uint16_t* const x = static_cast<const uint16_t*>(p.a);
  for (int it = blockIdx.x * (kFewThreads / 32) + warp; it < items; it += gridDim.x * (kFewThreads / 32)) {
    const int at = it / rows, r = it - at * rows, e = experts[at], t0 = tokens[at];
    const int len = min(start_of(p, e + 1) - t0, kFewAtOnce);
    const uint16_t* const w = static_cast<const uint16_t*>(p.b) + e * p.b_stride + (int64_t)r * cols;
    float acc[kFewAtOnce] = {};
    for (int c0 = 8 * lane; c0 < cols; c0 += 256 * kFewAhead) {
      uint4 q[kFewAhead];
#pragma unroll
      for (int k = 0; k < kFewAhead; ++k)
        if (c0 + 256 * k < cols) q[k] = load8(w, c0 + 256 * k, cols, kVec);
#pragma unroll
      for (int t = 0; t < kFewAtOnce; ++t) {
        if (t >= len) break;
        uint4 y[kFewAhead];                               // the first token's are in flight with the row
#pragma unroll
        for (int k = 0; k < kFewAhead; ++k)
          if (c0 + 256 * k < cols) y[k] = load8(x + (int64_t)(t0 + t) * p.a_ld, c0 + 256 * k, cols, kVec);
#pragma unroll
        for (int k = 0; k < kFewAhead; ++k) {
          if (c0 + 256 * k >= cols) break;
          const uint32_t a[4] = {q[k].x, q[k].y, q[k].z, q[k].w}, b[4] = {y[k].x, y[k].y, y[k].z, y[k].w};
#pragma unroll
          for (int i = 0; i < 4; ++i)
            acc[t] = fmaf(bf16_hi(a[i]), bf16_hi(b[i]), fmaf(bf16_lo(a[i]), bf16_lo(b[i]), acc[t]));
        }
      }
    }
#pragma unroll
    for (int t = 0; t < kFewAtOnce; ++t) {
      if (t >= len) break;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) acc[t] += __shfl_xor_sync(0xffffffffu, acc[t], o);
      if (lane != t) continue;
      const int64_t i = (int64_t)(t0 + t) * p.out_ld + r;
      if constexpr (kBf16) static_cast<__nv_bfloat16*>(p.out)[i] = __float2bfloat16_rn(acc[t]);
      else static_cast<float*>(p.out)[i] = acc[t];
    }
  }
  // rows of no expert
  const int64_t none = start_of(p, p.n_experts), total = (p.n_rows - none) * rows;
  for (int64_t i = (int64_t)blockIdx.x * kFewThreads + threadIdx.x; i < total; i += (int64_t)gridDim.x * kFewThreads) {
    const int64_t at = (none + i / rows) * p.out_ld + i % rows;
    if constexpr (kBf16) static_cast<uint16_t*>(p.out)[at] = 0;
    else static_cast<float*>(p.out)[at] = 0.f;
  }
}

cudaError_t launch_few_tokens(const ExpertArgs& a, cudaStream_t s) {
  const bool vec = a.cols % 8 == 0 && (a.n_experts == 1 || a.b_stride % 8 == 0) && (a.n_rows == 1 || a.a_ld % 8 == 0);
  const int64_t ctas = (a.n_rows * a.rows + kFewThreads / 32 - 1) / (kFewThreads / 32);       // at most
  const unsigned grid = (unsigned)std::min<int64_t>(ctas, 4 * (int64_t)std::max(1, sm_count()));
  const auto go = a.out_bf16 ? (vec ? few_tokens_kernel<true, true> : few_tokens_kernel<true, false>)
                             : (vec ? few_tokens_kernel<false, true> : few_tokens_kernel<false, false>);
  go<<<grid, kFewThreads, 0, s>>>(a);
  return cudaGetLastError();
}

using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                   const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                   CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
  static EncodeTiledFn fn = [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      f = nullptr;
    return reinterpret_cast<EncodeTiledFn>(f);
  }();
  return fn;
}

// A stack of n matrices (width x height, rows ld apart, matrices `stride`
// apart) in boxes of box_cols x box_rows x 1, swizzled where a row is 128 bytes.
bool encode(CUtensorMap* map, const void* base, int64_t width, int64_t height, int64_t ld, int64_t n, int64_t stride,
            int box_rows, int box_cols = 64, bool f32 = false, bool swizzle = true) {
  const EncodeTiledFn fn = encode_fn();
  if (!fn) return false;
  const int64_t esz = f32 ? 4 : 2;
  const cuuint64_t dims[3] = {(cuuint64_t)width, (cuuint64_t)height, (cuuint64_t)n};
  const cuuint64_t strides[2] = {(cuuint64_t)(ld * esz), (cuuint64_t)(stride * esz)};
  const cuuint32_t box[3] = {(cuuint32_t)box_cols, (cuuint32_t)box_rows, 1};
  const cuuint32_t one[3] = {1, 1, 1};
  return fn(map, f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base),
            dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
            swizzle ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int kMode, bool kBf16, bool kAccumulate, bool kVec>
cudaError_t launch_kernel(const ExpertArgs& a, const Maps& maps, int64_t max_tiles, cudaStream_t s) {
  constexpr size_t kSmemBytes = kRingBytes(kMode, kAccumulate) + kEpiWarps * 2 * kPartBytes(kMode) +
                                (kAccumulate ? kEpiWarps * kFetches * kFetchBytes : 0) + 1024;
  const auto kernel = expert_kernel<kMode, kBf16, kAccumulate, kVec>;
  static std::mutex mu;
  static int resident[kMaxDevices] = {};      // CTA pairs on the device at once
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = kSmemBytes;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  int pairs = 0;
  {
    std::lock_guard<std::mutex> lock(mu);
    if (resident[dev] == 0) {
      e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmemBytes);
      if (e != cudaSuccess) return e;
      cfg.gridDim = dim3((unsigned)(2 * (sm_count() / 2)), 1, 1);
      int n = 0;
      e = cudaOccupancyMaxActiveClusters(&n, kernel, &cfg);
      if (e != cudaSuccess) return e;
      if (n < 1) return cudaErrorInvalidConfiguration;
      resident[dev] = n;
    }
    pairs = resident[dev];
  }
  cfg.numAttrs = a.prepared ? 2 : 1;      // may start beside the kernels that prepare its operands
  cfg.stream = s;
  cfg.gridDim = dim3((unsigned)(2 * std::max<int64_t>(1, std::min<int64_t>(pairs, max_tiles))), 1, 1);
  e = cudaLaunchKernelEx(&cfg, kernel, a, maps);
  return e == cudaSuccess ? cudaGetLastError() : e;
}

template <int kMode>
cudaError_t launch_mode(const ExpertArgs& a, const Maps& maps, int64_t max_tiles, cudaStream_t s) {
  if constexpr (kMode == kExpertWeightGrad) {
    if (a.accumulate)
      return a.out_vec ? (a.out_bf16 ? launch_kernel<kMode, true, true, true>(a, maps, max_tiles, s)
                                     : launch_kernel<kMode, false, true, true>(a, maps, max_tiles, s))
                       : (a.out_bf16 ? launch_kernel<kMode, true, true, false>(a, maps, max_tiles, s)
                                     : launch_kernel<kMode, false, true, false>(a, maps, max_tiles, s));
  }
  return a.out_vec ? (a.out_bf16 ? launch_kernel<kMode, true, false, true>(a, maps, max_tiles, s)
                                 : launch_kernel<kMode, false, false, true>(a, maps, max_tiles, s))
                   : (a.out_bf16 ? launch_kernel<kMode, true, false, false>(a, maps, max_tiles, s)
                                 : launch_kernel<kMode, false, false, false>(a, maps, max_tiles, s));
}

int64_t up4(int64_t x) { return (x + 3) / 4 * 4; }
int64_t up8(int64_t x) { return (x + 7) / 8 * 8; }

// The jobs of one call and the workspace they fill.
struct Prepare {
  PrepareArgs a{};
  uint8_t* at;

  Prepare(const ExpertArgs& p) : at(p.packs) {
    a.starts = p.starts;
    a.n_rows = p.n_rows;
  }
  const void* add(const void* src, int64_t ld, int64_t stride, int64_t rows, int64_t width, int n, bool of_experts,
                  bool ends) {
    PrepareJob& j = a.job[a.jobs++];
    j.src = static_cast<const uint16_t*>(src);
    j.dst = reinterpret_cast<uint16_t*>(at);
    j.ld = ld;
    j.stride = stride;
    j.rows = rows;
    j.width = (int32_t)width;
    j.width8 = (int32_t)up8(width);
    j.n = n;
    j.of_experts = of_experts;
    j.ends = ends;
    j.block0 = a.blocks;
    const int64_t share = std::max<int64_t>(1, (int64_t)sm_count() * 8 / n);       // enough blocks to fill the GPU
    const int64_t blocks = (rows * (up8(width) / 8) + kPrepareThreads - 1) / kPrepareThreads;
    j.per = (int32_t)std::min<int64_t>(ends ? 1 : share, blocks);
    a.blocks += j.per * n;
    at += packed_bytes(n * rows, width);
    return j.dst;
  }
  // Activations n x width, ld apart: in place when every row starts on a 16-byte
  // boundary (a single row always does), else packed.
  void rows(const void** x, int64_t* ld, int64_t n, int64_t width) {
    if (n > 1 && *ld % 8 != 0) *x = add(*x, *ld, 0, n, width, 1, false, false);
    if (n <= 1 || *ld % 8 != 0) *ld = up8(width);
  }
  cudaError_t launch(cudaStream_t s) const {
    if (a.jobs == 0) return cudaSuccess;
    prepare_kernel<<<(unsigned)a.blocks, kPrepareThreads, 0, s>>>(a);
    return cudaGetLastError();
  }
};

// A weight gradient whose tiles leave half of the GPU idle may have its contraction cut: chunks
// of this many tokens (0: not cut), whose matrices go to the workspace in fp32 and are
// added by a second kernel.  As many as the pairs take in one turn, 512 tokens at least.
// A pair takes 4 (bf16) to 6 ns (fp32) for a token.  Whole, the longest group sets the time: taken as
// one and a half times the mean, which a cut has to make up for.  Cut, it is a chunk of fp32, the
// second launch (5 us, 833 tokens' time) and the parts' way out and in (0.42 us a MB, 70 tokens').
// Warm, GPU time in us, cut / whole, of bf16 gradients, groups even (and uneven, the longest about twice
// the mean), * where the rule cuts:
//    1 expert,   4096 tokens,  512 x  512   16.7 / 25.4 *
//    1           4096         1024 x 2048   29.5 / 25.4
//    1          16384         1024 x 1024   43.3 / 76.1 *
//    2           8192          512 x 1024   22.8 / 25.4 (23.6 / 30.5) *
//    4           4096          256 x 1024   18.5 / 13.1 (18.7 / 18.0)
//    4          16384          256 x  512   19.2 / 25.4 (21.3 / 44.1) *
//    8           8192          128 x  512   17.7 / 12.8 (17.7 / 18.2)
//    8          16384          256 x  256   18.7 / 17.2 (18.2 / 26.7) *
//   16          32768          256 x  512   29.0 / 18.5 (28.2 / 31.3)
// Of 1260 such pairs, fp32 gradients among them, the rule's choice is 1.8 % above the better one
// in the geometric mean; 1024 tokens an expert, whatever the matrices, 2.7 %, never cutting 68 %.
int64_t split_chunk(int64_t experts, int64_t n, int64_t rows, int64_t cols) {
  const int64_t tiles = ((rows + kPairM - 1) / kPairM) * ((cols + kMaxN - 1) / kMaxN);
  const int64_t most = kSplitPairs / tiles;          // chunks in all
  if (2 * experts > most || n < 4096) return 0;
  const int64_t parts = most - experts + 1;          // every expert's last chunk is short
  const int64_t chunk = std::max<int64_t>(512, ((n + parts - 1) / parts + kBlockK - 1) / kBlockK * kBlockK);
  const int64_t longest = experts == 1 ? n : 3 * n / (2 * experts);
  const int64_t part_bytes = (2 * n / chunk + experts) * rows * up4(cols) * 2;       // n / chunk + experts / 2 parts
  return longest > chunk + 833 + 70 * part_bytes / 1000000 ? chunk : 0;
}
// Chunks that there can be.
int64_t split_slots(int64_t experts, int64_t n, int64_t chunk) { return n / chunk + experts; }

}  // namespace

size_t expert_split_bytes(int64_t experts, int64_t n, int64_t rows, int64_t cols) {
  const int64_t chunk = split_chunk(experts, n, rows, cols);
  return chunk == 0 ? 0 : round_up((size_t)split_slots(experts, n, chunk) * rows * up4(cols) * sizeof(float), 256);
}

cudaError_t launch_expert(const ExpertArgs& in, cudaStream_t s) {
  ExpertArgs a = in;
  if (a.mode == kExpertForward && a.n_rows <= kFewTokens) return launch_few_tokens(a, s);
  const int64_t n = a.n_rows, mt = ((a.mode == kExpertInputGrad ? a.cols : a.rows) + kPairM - 1) / kPairM;
  Prepare prep(a);
  Maps maps{};
  ChunkSumArgs sum{};
  bool ok = true, sum_bf16 = false;
  // The longest wait is the epilogue's for a tile's whole contraction: 2 s, and
  // 64 ns for each of its K (8 clocks at the MMA's rate, at 1 GHz, 8 times over).
  const int64_t k_max = a.mode == kExpertWeightGrad ? n : (a.mode == kExpertForward ? a.cols : a.rows);
  a.wait_limit_ns = 2000000000ull + 64ull * (uint64_t)k_max;
  if (a.mode == kExpertWeightGrad) {
    if (n > 0) {                                   // without rows no tile has a contraction, and no copy is issued
      prep.rows(&a.a, &a.a_ld, n, a.rows);
      prep.rows(&a.b, &a.b_ld, n, a.cols);
      const void* end_a = prep.add(in.a, in.a_ld, 0, kEnd, a.rows, a.n_experts, true, true);
      const void* end_b = prep.add(in.b, in.b_ld, 0, kEnd, a.cols, a.n_experts, true, true);
      const int64_t m = (int64_t)a.n_experts * kEnd, ea = up8(a.rows), eb = up8(a.cols);
      ok = encode(&maps.a, a.a, a.rows, n, a.a_ld, 1, n * a.a_ld, 64) &&
           encode(&maps.b, a.b, a.cols, n, a.b_ld, 1, n * a.b_ld, 64) &&
           encode(&maps.c, end_a, a.rows, m, ea, 1, m * ea, kEnd) &&
           encode(&maps.d, end_b, a.cols, m, eb, 1, m * eb, kEnd);
    }
    const int64_t esz = a.out_bf16 ? 2 : 4;
    a.out_vec = a.cols * esz % 16 == 0 && (a.n_experts == 1 || a.out_stride * esz % 16 == 0);
    const int64_t stride = a.n_experts > 1 ? a.out_stride : a.rows * a.out_ld;
    a.chunk = (int32_t)split_chunk(a.n_experts, n, a.rows, a.cols);
    a.slots = a.chunk > 0 ? (int32_t)split_slots(a.n_experts, n, a.chunk) : 0;
    int64_t out_stride = stride;
    if (a.chunk > 0) {                             // the chunks' matrices, in fp32, in place of dW
      sum = {reinterpret_cast<const float*>(prep.at), a.out, a.starts, n, a.rows, a.cols, up4(a.cols), a.out_ld,
             a.out_stride, a.n_experts, a.chunk, a.slots, a.accumulate};
      sum_bf16 = a.out_bf16;
      a.out = prep.at;
      a.out_ld = up4(a.cols);
      a.out_stride = out_stride = a.rows * a.out_ld;
      a.out_bf16 = a.accumulate = 0;
      a.out_vec = 1;
    }
    if (a.out_vec)
      ok = ok && encode(&maps.out, a.out, a.cols, a.rows, a.out_ld, a.chunk > 0 ? a.slots : a.n_experts, out_stride, 16,
                        a.out_bf16 ? 64 : 32, !a.out_bf16);
  } else {
    const int64_t k = a.mode == kExpertForward ? a.cols : a.rows;
    if (a.cols % 8 != 0 || (a.n_experts > 1 && a.b_stride % 8 != 0)) {
      a.b = prep.add(a.b, a.b_ld, a.b_stride, a.rows, a.cols, a.n_experts, true, false);
      a.b_ld = up8(a.cols);
      a.b_stride = a.rows * a.b_ld;
    }
    prep.rows(&a.a, &a.a_ld, n, k);
    const int64_t w_stride = a.n_experts > 1 ? a.b_stride : a.rows * a.b_ld;
    ok = encode(&maps.a, a.b, a.cols, a.rows, a.b_ld, a.n_experts, w_stride, a.mode == kExpertForward ? 128 : 64) &&
         encode(&maps.b, a.a, k, n, a.a_ld, 1, n * a.a_ld, 32) &&
         encode(&maps.c, a.a, k, n, a.a_ld, 1, n * a.a_ld, 128) &&
         encode(&maps.d, a.a, k, n, a.a_ld, 1, n * a.a_ld, 64);
    // (a single row's leading dimension says nothing)
    const int64_t width = a.mode == kExpertForward ? a.rows : a.cols, y_ld = n > 1 ? a.out_ld : up8(width);
    // A tensor copy writes whole 16 bytes: where a row ends inside them, what lies
    // beside it would be lost.
    const int64_t esz = a.out_bf16 ? 2 : 4;
    a.out_vec = y_ld * esz % 16 == 0 && width * esz % 16 == 0;
    if (a.out_vec)
      ok = ok && encode(&maps.out, a.out, width, n, y_ld, 1, n * y_ld, a.out_bf16 ? 16 : 8, 32, !a.out_bf16, false);
  }
  if (!ok) return cudaErrorInvalidValue;
  a.prepared = prep.a.jobs > 0;
  a.only_ends = a.mode == kExpertWeightGrad && prep.a.jobs == 2;
  const cudaError_t e = prep.launch(s);
  if (e != cudaSuccess) return e;
  if (a.mode == kExpertWeightGrad) {
    const int64_t stack = a.chunk > 0 ? a.slots : a.n_experts;
    const cudaError_t err = launch_mode<kExpertWeightGrad>(a, maps, stack * mt * ((a.cols + kMaxN - 1) / kMaxN), s);
    if (err != cudaSuccess || a.chunk == 0) return err;
    const int64_t items = (a.rows * (a.out_ld / 4) + 31) / 32;
    const int64_t blocks = std::min<int64_t>(items, (8 * kSms + a.n_experts - 1) / a.n_experts);
    const dim3 grid((unsigned)blocks, (unsigned)a.n_experts);
    return launch_overlapped(sum_bf16 ? sum_chunks_kernel<true> : sum_chunks_kernel<false>, grid, dim3(32 * kSumWarps),
                             0, s, true, sum);
  }
  const int64_t tiles = mt * (n / kMaxN + std::min<int64_t>(a.n_experts, n));
  return a.mode == kExpertForward ? launch_mode<kExpertForward>(a, maps, tiles, s)
                                  : launch_mode<kExpertInputGrad>(a, maps, tiles, s);
}

}  // namespace ops
}  // namespace mfsdp
