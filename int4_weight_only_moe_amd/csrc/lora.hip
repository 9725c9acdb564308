// Low-rank adapters of many requests beside a shared projection.
//
// Row t of the batch belongs to a request with adapter a = ids[t] (A_a [r, K],
// B_a [N, r], scale s_a), or to one without (ids[t] outside [0, L)):
//   h_t  = A_a x_t                         out_t = base_t + s_a B_a h_t
//   dh_t = s_a B_a^T dout_t                dx_t  = dxbase_t + A_a^T dh_t
//   dA_a = sum_t dh_t x_t^T                dB_a  = s_a sum_t dout_t h_t^T
//
// The rows are grouped by adapter into tiles of up to 64 rows of one adapter
// (rows without one are the last group). The kernels:
//   group   the grouping, one workgroup; a forward of up to 256 rows has none:
//           there each workgroup finds its tile's rows from the ids;
//   down    contracts a wide side with a [r, W] operand (h, dh) in splits of W;
//   up      adds the splits, expands r values to a wide side and adds the base
//           (out, dx);
//   join    backward: dh, the sum of its splits, as it is and rank-major, and
//           s h rank-major (the transposed weights are made beside the grouping);
//   outer   sums rows' outer products (dA, dB), reduce joins what was cut.
// With r <= 128 each of them moves the wide side once, and that traffic is its
// floor (a copy reaches 5.2 TB/s read and written, a read 7); a small call is bound
// by its launches (one follows another every 3.6 us). The matrix cores have room,
// so the products are made exact: bf16 operands multiply exactly into fp32, and an
// fp32 factor (h, dh, an fp32 side) enters as three bf16 parts of 8 bits each, all
// 24 bits of fp32.
#include <type_traits>

#include "device_common.h"
#include "operators.h"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;
constexpr int kSub = 16;  // rows of a matrix-core tile

typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));

__device__ __forceinline__ uint32_t bf16_bits(float v) {
  return (uint32_t)__builtin_bit_cast(uint16_t, (__bf16)v);
}
__device__ __forceinline__ float bf16_value(uint32_t bits) { return __uint_as_float(bits << 16); }

// Two fp32 values rounded to bf16, the first in the low half.
__device__ __forceinline__ uint32_t bf16_pair(float lo, float hi) {
  typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
  return __builtin_bit_cast(uint32_t, bf16x2_t{(__bf16)lo, (__bf16)hi});
}

// Eight fp32 values as NP bf16 parts, v = parts[0] + parts[1] + ...: each part
// is the rounding of what the parts before it leave. Values are converted in pairs
// and taken apart again: one by one the compiler converts each of them twice.
template <int NP>
__device__ __forceinline__ void split_parts(const float (&v)[8], bf16x8_t (&parts)[NP]) {
  float rest[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) rest[i] = v[i];
#pragma unroll
  for (int p = 0; p < NP; ++p) {
    uint32_t d[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      d[i] = bf16_pair(rest[2 * i], rest[2 * i + 1]);
      rest[2 * i] -= bf16_value(d[i]);
      rest[2 * i + 1] -= __uint_as_float(d[i] & 0xffff0000u);
    }
    parts[p] = as_bf16x8(make_uint4(d[0], d[1], d[2], d[3]));
  }
}

// Whether every lane of `live` holds the same key as its first one.
__device__ __forceinline__ bool one_key(int key, uint64_t live) {
  const int first = __builtin_amdgcn_readfirstlane(__shfl(key, (int)__builtin_ctzll(live | (uint64_t(1) << 63)), 64));
  return (__ballot(key == first) & live) == live;
}

// Lanes of `live` whose key equals this lane's (keys below 2^nbits).
__device__ __forceinline__ uint64_t same_key(int key, int nbits, uint64_t live) {
  if (one_key(key, live)) return live;
  uint64_t m = live;
  for (int b = 0; b < nbits; ++b) {
    const bool bit = (key >> b) & 1;
    const uint64_t bal = __ballot(bit);
    m &= bit ? bal : ~bal;
  }
  return m;
}

__device__ __forceinline__ int bits_below(uint64_t m) {
  return __builtin_amdgcn_mbcnt_hi((uint32_t)(m >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)m, 0));
}

// ------------------------------------------------------------------ group
constexpr int kGroupThreads = 1024;
constexpr int kGroupWaves = kGroupThreads / 64;
constexpr int kMaxKeys = 1025;  // 1024 adapters and "none"

// Backward: the weights of the adapters that have rows, transposed. Workgroups
// 1.. of the grouping's launch do it, without waiting for the grouping.
struct TransposeArgs {
  const uint16_t* a;        // [L][r][K]
  const uint16_t* b;        // [L][N][r]
  int K, N, r;
  int64_t n_pad;
  uint16_t* at;             // [L][K][r]
  uint16_t* bt;             // [L][r][n_pad], zeros from N
  int a_blocks, b_blocks;   // workgroups per adapter
};

struct GroupArgs {
  const int32_t* ids;       // [M]
  int M, L;
  int32_t* sorted;          // rows by adapter, each list padded to 64 with M
  int4* tiles;              // a tile's adapter (L: rows without one), rows, and its list's range of positions
  int32_t* offsets;         // [L + 2]: each list's first position; [L] the first row without an adapter
  int all_tiles;            // room for: tiles past the last have no rows
};

// One 64 x 64 block of in [R][C] (C a multiple of 8) to out [C][pitch], rows
// from R on as zeros up to the pitch.
__device__ __forceinline__ void transpose_block(const uint16_t* __restrict__ in, int R, int C, int64_t pitch,
                                                uint16_t* __restrict__ out, int r0, int c0, uint16_t* lds) {
  constexpr int kPitch = 64 + 8;
  const int tid = threadIdx.x;
  if (tid < 64 * 8) {
    const int i = tid, row = i >> 3, col = (i & 7) * 8;
    uint4 v = make_uint4(0, 0, 0, 0);
    if (r0 + row < R && c0 + col < C) v = *(const uint4*)(in + (int64_t)(r0 + row) * C + c0 + col);
    *(uint4*)(lds + row * kPitch + col) = v;
  }
  __syncthreads();
  if (tid < 64 * 8) {
    const int i = tid, col = i >> 3, row = (i & 7) * 8;
    if (c0 + col >= C || r0 + row >= pitch) return;
    uint32_t d[4];
#pragma unroll
    for (int e = 0; e < 4; ++e)
      d[e] = lds[(row + 2 * e) * kPitch + col] | (uint32_t)lds[(row + 2 * e + 1) * kPitch + col] << 16;
    *(uint4*)(out + (int64_t)(c0 + col) * pitch + r0 + row) = make_uint4(d[0], d[1], d[2], d[3]);
  }
}

// Each of these workgroups lists the adapters that have rows, then takes every
// gridDim.x - 1'th block of their weights.
__device__ __forceinline__ void transpose_weights(const GroupArgs& g, const TransposeArgs& p, int* room) {
  int* used = room;                          // [1024]
  int* list = room + kGroupThreads;          // [1024]
  int* wave_n = list + kGroupThreads;        // [16]
  uint16_t* lds = (uint16_t*)(wave_n + 16);  // 64 x 72
  const int tid = threadIdx.x, wave = tid >> 6;
  used[tid] = 0;
  __syncthreads();
  constexpr int kAhead = 8;
  for (int f = tid; f < g.M; f += kAhead * kGroupThreads) {
    int id[kAhead];
#pragma unroll
    for (int q = 0; q < kAhead; ++q) id[q] = g.ids[f + q * kGroupThreads < g.M ? f + q * kGroupThreads : f];
#pragma unroll
    for (int q = 0; q < kAhead; ++q)
      if (id[q] >= 0 && id[q] < g.L) used[id[q]] = 1;
  }
  __syncthreads();
  const bool mine = used[tid] != 0;
  const uint64_t live = __ballot(mine);
  if ((tid & 63) == 0) wave_n[wave] = __builtin_popcountll(live);
  __syncthreads();
  int before = bits_below(live), n = 0;
#pragma unroll
  for (int w = 0; w < kGroupWaves; ++w) {
    before += w < wave ? wave_n[w] : 0;
    n += wave_n[w];
  }
  if (mine) list[before] = tid;
  __syncthreads();
  const int per = p.a_blocks + p.b_blocks;
  const int across = (p.K + 63) / 64, down = (int)((p.n_pad + 63) / 64);
  for (int64_t item = blockIdx.x - 1; item < (int64_t)n * per; item += gridDim.x - 1) {
    const int l = list[item / per];
    int i = (int)(item % per);
    if (i < p.a_blocks) {
      const int64_t at = (int64_t)l * p.r * p.K;
      transpose_block(p.a + at, p.r, p.K, p.r, p.at + at, i / across * 64, i % across * 64, lds);
    } else {
      i -= p.a_blocks;
      transpose_block(p.b + (int64_t)l * p.N * p.r, p.N, p.r, p.n_pad, p.bt + l * p.r * p.n_pad, i % down * 64,
                      i / down * 64, lds);
    }
    __syncthreads();
  }
}

// Stable grouping by one workgroup: each wave walks a contiguous range of the
// rows 64 at a time, counts its rows per adapter (one LDS update per distinct
// adapter of a step, so rows of one adapter in a run cost no more than mixed
// ones), the counts become each wave's first positions, and a second walk
// places the rows. Up to 8192 rows are read once. Bound by the latency of its
// passes: 6.5 us for 8192 rows, with the weights' transposition beside it (rank
// 64, [7168] both sides) too. One workgroup whatever the number of rows, so it
// grows with them: 23 us for 32768 rows in runs, 44 for 65536 (86 if the 64
// adapters are mixed), 1.3 ms for 2^20; the other workgroups' own reading of the ids
// does not show beside that.
__global__ __launch_bounds__(kGroupThreads, 8) void lora_group_kernel(GroupArgs p, TransposeArgs weights) {
  __shared__ __align__(16) int cnt[kGroupWaves][kMaxKeys];
  __shared__ int off[kMaxKeys + 1], rows_of[kMaxKeys];
  __shared__ int wave_tot[kGroupWaves];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  if (blockIdx.x > 0) {
    transpose_weights(p, weights, &cnt[0][0]);
    return;
  }
  const int keys = p.L + 1;
  const int nbits = 32 - __clz(p.L);
  for (int i = tid; i < keys; i += kGroupThreads)
#pragma unroll
    for (int w = 0; w < kGroupWaves; ++w) cnt[w][i] = 0;
  __syncthreads();
  const int seg = ((p.M + kGroupWaves - 1) / kGroupWaves + 63) / 64 * 64;
  const int f0 = wave * seg < p.M ? wave * seg : p.M;
  const int f1 = f0 + seg < p.M ? f0 + seg : p.M;
  // 512 rows of the wave's range: each lane's keys, and its rank among the equal
  // keys of its step (low half) with their number
  constexpr int kSteps = 8;
  int key[kSteps], place[kSteps];
  auto walk = [&](int fb) {
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
      const int f = fb + 64 * i + lane;
      const int id = p.ids[f < f1 ? f : f1 - 1];
      key[i] = id >= 0 && id < p.L ? id : p.L;
    }
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
      if (fb + 64 * i >= f1) break;
      const uint64_t same = same_key(key[i], nbits, __ballot(fb + 64 * i + lane < f1));
      place[i] = bits_below(same) | __builtin_popcountll(same) << 16;
    }
  };
  for (int fb = f0; fb < f1; fb += 64 * kSteps) {
    walk(fb);
#pragma unroll
    for (int i = 0; i < kSteps; ++i)
      if (fb + 64 * i + lane < f1 && (place[i] & 0xffff) == 0) cnt[wave][key[i]] += place[i] >> 16;
  }
  __syncthreads();
  // exclusive scan of the adapters' padded counts, one adapter a thread
  int total = 0;
  if (tid < p.L) {
#pragma unroll
    for (int w = 0; w < kGroupWaves; ++w) total += cnt[w][tid];
  }
  const int padded = (total + kLoraTile - 1) / kLoraTile * kLoraTile;
  int incl = padded;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int o = __shfl_up(incl, d, 64);
    if (lane >= d) incl += o;
  }
  if (lane == 63) wave_tot[wave] = incl;
  __syncthreads();
  int before = 0, all = 0;
#pragma unroll
  for (int w = 0; w < kGroupWaves; ++w) {
    before += w < wave ? wave_tot[w] : 0;
    all += wave_tot[w];
  }
  // a list's rows, then the padding; the waves' counts become first positions
  auto lay = [&](int key, int first, int count, int room) {
    off[key] = first;
    rows_of[key] = count;
    p.offsets[key] = first;
    for (int i = first + count; i < first + room; ++i) p.sorted[i] = p.M;
    int run = first;
#pragma unroll
    for (int w = 0; w < kGroupWaves; ++w) {
      const int c = cnt[w][key];
      cnt[w][key] = run;
      run += c;
    }
  };
  if (tid < p.L) lay(tid, before + incl - padded, total, padded);
  if (tid == kGroupThreads - 1) {  // rows without an adapter
    int none = 0;
    for (int w = 0; w < kGroupWaves; ++w) none += cnt[w][p.L];
    const int room = (none + kLoraTile - 1) / kLoraTile * kLoraTile;
    lay(p.L, all, none, room);
    off[p.L + 1] = all + room;
    p.offsets[p.L + 1] = all + room;
  }
  __syncthreads();
  const int tiles = off[p.L + 1] / kLoraTile;
  for (int b = tid; b < p.all_tiles; b += kGroupThreads) {
    if (b >= tiles) {
      p.tiles[b] = make_int4(p.L, 0, 0, 0);
      continue;
    }
    int lo = 0, hi = p.L;  // the last list that starts at or before the tile
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (off[mid] <= b * kLoraTile) lo = mid; else hi = mid - 1;
    }
    const int left = off[lo] + rows_of[lo] - b * kLoraTile;
    p.tiles[b] = make_int4(lo, left < kLoraTile ? left : kLoraTile, off[lo], off[lo + 1]);
  }
  for (int fb = f0; fb < f1; fb += 64 * kSteps) {
    if (seg > 64 * kSteps) walk(fb);  // else the one batch is still there
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
      if (fb + 64 * i + lane >= f1) continue;
      // every lane reads the running position before the first lane advances it
      // (one wave: its LDS operations complete in order)
      const int base = cnt[wave][key[i]];
      p.sorted[base + (place[i] & 0xffff)] = fb + 64 * i + lane;
      if ((place[i] & 0xffff) == 0) cnt[wave][key[i]] = base + (place[i] >> 16);
    }
  }
}

// ------------------------------------------------------------------ a workgroup's tile
struct TileArgs {
  const int32_t* ids;            // [M]
  const int32_t* sorted;         // the grouping, or null: a small batch
  const int4* tiles;
  int M, L;
};
struct Tile {
  int rows[kLoraTile];  // rows past the last repeat the first (their results are dropped)
  int key[kLoraSmallRows];
  int wave_leaders[kLoraSmallRows / 64];
  int count, adapter, first_rank;
};

// The tile's rows in LDS. Returns their number, 0 if there is no such tile.
// A small batch: row t leads a tile if it is the 64 i-th row of its adapter;
// the tiles count in the order of their leaders.
__device__ __forceinline__ int find_tile(const TileArgs& p, Tile& sh, int tile) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  if (p.sorted) {
    const int4 info = p.tiles[tile];
    const int first = p.sorted[tile * kLoraTile];
    const int row = p.sorted[tile * kLoraTile + lane];
    if (info.y == 0) return 0;
    if (tid < kLoraTile) sh.rows[tid] = row < p.M ? row : first;
    if (tid == 0) sh.adapter = info.x;
    __syncthreads();
    return info.y;
  }
  int key = -1;
  if (tid < p.M) {
    const int id = p.ids[tid];
    key = id >= 0 && id < p.L ? id : p.L;
  }
  if (tid < kLoraSmallRows) sh.key[tid] = key;
  if (tid == 0) sh.count = 0;
  __syncthreads();
  int rank = 0;
  for (int u = 0; u < p.M; u += 4) {
    const int4 k = *(const int4*)(sh.key + u);
    rank += (u < tid && k.x == key) + (u + 1 < tid && k.y == key) + (u + 2 < tid && k.z == key) +
            (u + 3 < tid && k.w == key);
  }
  const bool leads = key >= 0 && rank % kLoraTile == 0;
  const uint64_t leaders = __ballot(leads);
  if (lane == 0 && wave < kLoraSmallRows / 64) sh.wave_leaders[wave] = __builtin_popcountll(leaders);
  __syncthreads();
  int before = bits_below(leaders), all = 0;
#pragma unroll
  for (int w = 0; w < kLoraSmallRows / 64; ++w) {
    before += w < wave ? sh.wave_leaders[w] : 0;
    all += sh.wave_leaders[w];
  }
  if (tile >= all) return 0;
  if (leads && before == tile) {
    sh.adapter = key;
    sh.first_rank = rank;
  }
  __syncthreads();
  const int at = rank - sh.first_rank;
  if (key == sh.adapter && at >= 0 && at < kLoraTile) {
    sh.rows[at] = tid;
    atomicAdd(&sh.count, 1);
  }
  __syncthreads();
  const int n = sh.count;
  if (tid >= n && tid < kLoraTile) sh.rows[tid] = sh.rows[0];
  __syncthreads();
  return n;
}

// All ones or zeros, in a register whose value the compiler cannot trace: it
// turns a load whose value is dropped for some lanes into a branch around the
// load, and after one of those waits no longer for the loads that it needs but
// for all of them.
__device__ __forceinline__ uint32_t lane_mask(bool keep) {
  uint32_t m = keep ? 0xffffffffu : 0u;
  asm("" : "+v"(m));
  return m;
}

// 16 bytes of a row of W elements from element w. Past the row's end: zeros
// (Zero), or anything. Vec: the row is 16-byte aligned and W a multiple of 16
// bytes' elements.
template <typename T, bool Vec, bool Zero = true>
__device__ __forceinline__ uint4 load16(const T* __restrict__ row, int w, int W) {
  constexpr int kN = 16 / sizeof(T);
  if constexpr (Vec) {
    uint4 v = *(const uint4*)(row + (w < W ? w : 0));
    if constexpr (Zero) {
      const uint32_t m = lane_mask(w < W);
      v.x &= m; v.y &= m; v.z &= m; v.w &= m;
    }
    return v;
  } else {
    uint32_t d[4] = {0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      const T x = row[w + i < W ? w + i : 0];
      const uint32_t m = Zero ? lane_mask(w + i < W) : 0xffffffffu;
      if constexpr (sizeof(T) == 4) d[i] = __float_as_uint(x) & m;
      else d[i / 2] |= ((uint32_t)x & m) << (16 * (i & 1));
    }
    return make_uint4(d[0], d[1], d[2], d[3]);
  }
}

// Orders a wave's own LDS writes before its later reads (the hardware runs one
// wave's LDS operations in order; this keeps the compiler from moving them).
__device__ __forceinline__ void wave_lds_fence() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

// ------------------------------------------------------------------ down
struct DownArgs {
  TileArgs tile;
  const void* u;              // [M, W]
  int64_t ldu;
  int W;
  const uint16_t* v;          // [L][r][ldv], zeros from W to ldv
  int64_t v_stride, ldv;
  int r;
  int splits, split_steps;    // 128-byte steps per split
  float* part;                // [splits][M][r]
  float* h;                   // [M][r] or null: receives zeros for rows without an adapter
};

// A step is 128 bytes of the rows of u: 64 bf16 or 32 fp32 columns.
template <typename TU, int RT>
struct DownShape {
  static constexpr int kCols = 128 / sizeof(TU);
  static constexpr int kVChunks = kCols / 8;  // 16-byte chunks of a row of v
  static constexpr int kStage = kLoraTile * 128 + RT * 16 * kVChunks * 16;
  static constexpr int kSums = kLoraTile * RT * 16 * 4;
  static constexpr int kWaveBytes = kStage > kSums ? kStage : kSums;  // a wave's LDS
};

// A wave's sums over its steps of v[j][w] * u[row][w], left in its LDS as
// [row][rank] with the 16-byte chunks of a row exchanged by row.
// The matrix core wants lane (g, c) to hold 8 columns of row c, but a load
// instruction runs at full rate only where neighbouring lanes read neighbouring
// bytes (with 16 bytes a row and lane the kernel took 40 us instead of 32 for
// [8192, 7168], rank 64). So eight lanes read a row's 128 bytes, and the step
// goes through the wave's own part of LDS (no other wave takes part, so no
// barrier), chunks exchanged by row so that the 16 rows of a fragment lie in
// different banks. The next step's loads are in flight while this one is
// multiplied. Bound by the reading of u, beside which as many bytes of v come
// from L2: [8192, 7168] bf16, rank 64, 31.6 us (3.7 TB/s of u), six adapters'
// [4096, 7168] 25 us; one row 4.9 us, little more than a launch.
template <typename TU, int RT, bool VecU, int NSUB>
__device__ __forceinline__ void down_tile(const DownArgs& p, const Tile& sh, uint4* lds) {
  constexpr bool kF32 = std::is_same<TU, float>::value;
  using Shape = DownShape<TU, RT>;
  constexpr int kVC = Shape::kVChunks;
  constexpr int kLoadsU = NSUB * 2, kLoadsV = RT * kVC / 4;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, c = lane & 15, g = lane >> 4;
  const TU* urow[kLoadsU];
#pragma unroll
  for (int i = 0; i < kLoadsU; ++i) urow[i] = (const TU*)p.u + (int64_t)sh.rows[i * 8 + (lane >> 3)] * p.ldu;
  const uint16_t* vrow[kLoadsV];
#pragma unroll
  for (int i = 0; i < kLoadsV; ++i) {
    const int j = (i * 64 + lane) / kVC;
    vrow[i] = p.v + sh.adapter * p.v_stride + (j < p.r ? j : p.r - 1) * p.ldv;
  }
  uint4* vlds = lds + kLoraTile * 8;
  f32x4_t acc[RT][NSUB];
#pragma unroll
  for (int rt = 0; rt < RT; ++rt)
#pragma unroll
    for (int ts = 0; ts < NSUB; ++ts) acc[rt][ts] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
  const int steps = (p.W + Shape::kCols - 1) / Shape::kCols;
  const int s0 = blockIdx.y * p.split_steps;
  const int s1 = s0 + p.split_steps < steps ? s0 + p.split_steps : steps;
  uint4 u[kLoadsU], v[kLoadsV];
  auto load = [&](int s) {
#pragma unroll
    for (int i = 0; i < kLoadsU; ++i)
      u[i] = load16<TU, VecU>(urow[i], s * Shape::kCols + (lane & 7) * (16 / (int)sizeof(TU)), p.W);
#pragma unroll
    for (int i = 0; i < kLoadsV; ++i)
      v[i] = load16<uint16_t, true>(vrow[i], s * Shape::kCols + (lane % kVC) * 8, (int)p.ldv);
  };
  int s = s0 + wave;
  if (s < s1) load(s);
  for (; s < s1; s += kWaves) {
#pragma unroll
    for (int i = 0; i < kLoadsU; ++i) {
      const int row = i * 8 + (lane >> 3);
      lds[row * 8 + ((lane & 7) ^ (row & 7))] = u[i];
    }
#pragma unroll
    for (int i = 0; i < kLoadsV; ++i) {
      const int j = (i * 64 + lane) / kVC;
      vlds[j * kVC + ((lane % kVC) ^ (j & (kVC - 1)))] = v[i];
    }
    wave_lds_fence();
    if (s + kWaves < s1) load(s + kWaves);
#pragma unroll
    for (int ks = 0; ks < kVC / 4; ++ks) {
      bf16x8_t vf[RT];
#pragma unroll
      for (int rt = 0; rt < RT; ++rt)
        vf[rt] = as_bf16x8(vlds[(rt * 16 + c) * kVC + ((ks * 4 + g) ^ (c & (kVC - 1)))]);
#pragma unroll
      for (int ts = 0; ts < NSUB; ++ts) {
        const uint4* row = lds + (ts * kSub + c) * 8;
        if constexpr (kF32) {
          const uint4 lo = row[(2 * g) ^ (c & 7)], hi = row[(2 * g + 1) ^ (c & 7)];
          const float f[8] = {__uint_as_float(lo.x), __uint_as_float(lo.y), __uint_as_float(lo.z), __uint_as_float(lo.w),
                              __uint_as_float(hi.x), __uint_as_float(hi.y), __uint_as_float(hi.z), __uint_as_float(hi.w)};
          bf16x8_t q[3];
          split_parts<3>(f, q);
#pragma unroll
          for (int rt = 0; rt < RT; ++rt)
#pragma unroll
            for (int i = 0; i < 3; ++i) acc[rt][ts] = mfma16x16x32(vf[rt], q[i], acc[rt][ts]);
        } else {
          const bf16x8_t uf = as_bf16x8(row[(ks * 4 + g) ^ (c & 7)]);
#pragma unroll
          for (int rt = 0; rt < RT; ++rt) acc[rt][ts] = mfma16x16x32(vf[rt], uf, acc[rt][ts]);
        }
      }
    }
    wave_lds_fence();
  }
  // lane (g, c) holds ranks 16 rt + 4 g .. + 3 of row 16 ts + c
#pragma unroll
  for (int rt = 0; rt < RT; ++rt)
#pragma unroll
    for (int ts = 0; ts < NSUB; ++ts) {
      const int row = ts * kSub + c;
      *(f32x4_t*)(lds + row * RT * 4 + ((rt * 4 + g) ^ (row & (RT * 4 - 1)))) = acc[rt][ts];
    }
}

template <typename TU, int RT, bool VecU>
__global__ __launch_bounds__(kThreads) void lora_down_kernel(DownArgs p) {
  constexpr int kWaveChunks = DownShape<TU, RT>::kWaveBytes / 16;
  constexpr int kQuads = RT * 4;
  __shared__ __align__(16) Tile sh;
  __shared__ uint4 lds[kWaves * kWaveChunks];
  const int tid = threadIdx.x;
  const int n = find_tile(p.tile, sh, blockIdx.x);
  if (n == 0) return;
  if (sh.adapter == p.tile.L) {  // rows without an adapter
    if (p.h && blockIdx.y == 0)
      for (int i = tid; i < n * p.r; i += kThreads) p.h[(int64_t)sh.rows[i / p.r] * p.r + i % p.r] = 0.0f;
    return;
  }
  uint4* mine = lds + (tid >> 6) * kWaveChunks;
  if (n <= 16) down_tile<TU, RT, VecU, 1>(p, sh, mine);
  else if (n <= 32) down_tile<TU, RT, VecU, 2>(p, sh, mine);
  else down_tile<TU, RT, VecU, 4>(p, sh, mine);
  __syncthreads();
  float* part = p.part + (int64_t)blockIdx.y * p.tile.M * p.r;
  for (int i = tid; i < n * kQuads; i += kThreads) {
    const int t = i / kQuads, quad = i % kQuads;
    if (quad * 4 >= p.r) continue;
    const f32x4_t* at = (const f32x4_t*)(lds + t * kQuads + (quad ^ (t & (kQuads - 1))));
    *(f32x4_t*)(part + (int64_t)sh.rows[t] * p.r + quad * 4) =
        (at[0] + at[kWaveChunks]) + (at[2 * kWaveChunks] + at[3 * kWaveChunks]);
  }
}

// h: the sum of its splits; 0 for rows without an adapter. 5 us for 7 splits of
// [4096, 64].
__global__ __launch_bounds__(kThreads) void lora_sum_kernel(const float* __restrict__ part, int splits, int64_t size,
                                                            int r, const int32_t* __restrict__ ids, int L,
                                                            float* __restrict__ h) {
  const int64_t i = ((int64_t)blockIdx.x * kThreads + threadIdx.x) * 4;
  if (i >= size) return;
  const int id = ids[i / r];
  float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 8
  for (int s = 0; s < splits; ++s) {
    const float4 x = *(const float4*)(part + s * size + i);
    v.x += x.x; v.y += x.y; v.z += x.z; v.w += x.w;
  }
  if (id < 0 || id >= L) v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  *(float4*)(h + i) = v;
}

// ------------------------------------------------------------------ up
struct UpArgs {
  TileArgs tile;
  int r, N;
  const float* part;          // [splits][M][r]: the factor's partial sums
  int splits;
  const float* scales;        // [L] or null
  float* h;                   // [M, r] or null, receives the sums
  const uint16_t* b;          // [L][N][r]
  const void* base;           // [M, N] or null
  int64_t ld_base;
  void* out;                  // [M, N]
  int64_t ld_out;
  int n_block;                // columns per workgroup
  int across;                 // workgroups per tile
};

// Four consecutive columns from n of a row, as raw bits (fp32: one word each,
// bf16: two words in all); columns past the end hold anything. Vec: the row is
// 16-byte aligned and N % 4 == 0. Past: around the caches.
template <typename TO, bool Vec, bool Past>
__device__ __forceinline__ uint4 load4(const TO* row, int n, int N) {
  // columns past the end read the row's first ones: a load that is always made
  // keeps the count of loads in flight known
  if constexpr (Vec) {
    const TO* at = row + (n < N ? n : 0);
    if constexpr (sizeof(TO) == 4) return *(const uint4*)at;
    const u32x2_t v = Past ? __builtin_nontemporal_load((const u32x2_t*)at) : *(const u32x2_t*)at;
    return make_uint4(v[0], v[1], 0, 0);
  } else {
    uint32_t d[4] = {0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const TO x = row[n + i < N ? n + i : 0];
      if constexpr (sizeof(TO) == 4) d[i] = __float_as_uint(x);
      else d[i / 2] |= (uint32_t)x << (16 * (i & 1));
    }
    return make_uint4(d[0], d[1], d[2], d[3]);
  }
}
template <typename TO, bool Vec, bool Past>
__device__ __forceinline__ void store4(TO* row, int n, int N, uint4 v) {
  if constexpr (Vec) {
    if (n >= N) return;
    if constexpr (sizeof(TO) == 4) *(uint4*)(row + n) = v;
    else if constexpr (Past) __builtin_nontemporal_store(u32x2_t{v.x, v.y}, (u32x2_t*)(row + n));
    else *(u32x2_t*)(row + n) = u32x2_t{v.x, v.y};
  } else {
    const uint32_t d[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (n + i < N) {
        if constexpr (sizeof(TO) == 4) row[n + i] = __uint_as_float(d[i]);
        else row[n + i] = (uint16_t)(d[i / 2] >> (16 * (i & 1)));
      }
    }
  }
}

// LDS of a workgroup: the factor as three bf16 parts, and a wave's 64 rows of b.
// For bf16 results b goes through LDS in turns of 32 ranks each, so that a CU holds
// three workgroups up to rank 64 and two above: rank 64, [7168] columns of 8192
// rows 65 us and of 4096 rows 33.5, in one turn with two workgroups 72.5 and 32.4;
// rank 128 of 4096 rows 47.5, in one turn with one workgroup 57. With fp32 results
// the registers hold two and one (as two workgroups rank 128 of 2048 rows of [7165]
// takes 92 us instead of 67), for which one turn leaves room.
template <typename TO, int RC>
struct UpShape {
  static constexpr int kParts = 3;
  static constexpr int kPitch = RC + 8;                                        // of the factor's rows
  static constexpr int kTurns = sizeof(TO) == 2 && RC > 32 ? RC / 32 : 1;
  static constexpr int kSeg = RC / 8 / kTurns;                                 // 8-wide chunks of a row in a turn
  static constexpr int kWorkgroups = RC <= 64 ? 3 : (sizeof(TO) == 2 ? 2 : 1);  // a CU, aimed at
};

// The tile's factor: the sums of the partial sums, scaled.
template <typename TO, int RC>
__device__ __forceinline__ void up_factor(const UpArgs& p, const Tile& sh, int n, uint16_t* lds) {
  using Shape = UpShape<TO, RC>;
  const int tid = threadIdx.x;
  const int rows = (n + kSub - 1) / kSub * kSub;
  const float scale = p.scales ? p.scales[sh.adapter] : 1.0f;
  const int64_t split_size = (int64_t)p.tile.M * p.r;
  for (int i = tid; i < rows * (RC / 4); i += kThreads) {
    const int t = i / (RC / 4), j = i % (RC / 4) * 4;
    float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (t < n && j < p.r) {
      const int64_t at = (int64_t)sh.rows[t] * p.r + j;
#pragma unroll 8
      for (int s = 0; s < p.splits; ++s) {
        const float4 x = *(const float4*)(p.part + s * split_size + at);
        v.x += x.x; v.y += x.y; v.z += x.z; v.w += x.w;
      }
      if (p.h && blockIdx.x % p.across == 0) *(float4*)(p.h + at) = v;
    }
    float f[4] = {v.x * scale, v.y * scale, v.z * scale, v.w * scale};
#pragma unroll
    for (int q = 0; q < Shape::kParts; ++q) {
      uint32_t bits[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        bits[e] = bf16_bits(f[e]);
        f[e] -= bf16_value(bits[e]);
      }
      *(uint2*)(lds + (q * kLoraTile + t) * Shape::kPitch + j) = make_uint2(bits[0] | bits[1] << 16, bits[2] | bits[3] << 16);
    }
  }
}

constexpr int kUpCols = 64;  // columns of a wave

// out[row][n] = base[row][n] + sum_j b[n][j] * factor[row][j].
// The factor's bf16 parts are laid one after another along the contraction:
// 8-wide chunk number q of a lane's fragments is chunk q % (r / 8) of part
// q / (r / 8), so ranks 8 and 16 fill one 32-wide matrix-core step with their
// parts. A wave takes 64 columns: matrix-core tile i has the columns 4 c + i
// (c its column), so a lane ends with four consecutive columns of four rows, and
// 16 lanes read and write 128 (fp32: 256) consecutive bytes of a row. b's 64
// rows are consecutive in memory and go through the wave's own part of LDS, as
// in down. What does not depend on the factor is loaded before it is made.
// None: rows without an adapter, out = base.
// Bound by reading the base and writing out, beside which b comes from L2 and the
// matrix cores run: [8192, 7168] bf16 of rank 64 65 us (3.6 TB/s; 60.5 with a factor
// of two parts, 16 bits, whose loss shows in a bf16 result that cancels), [4096,
// 7168] 33.5 us, of rank 128 47.5, rank 16 [1999, 7168] 16 us.
template <typename TO, int RC, bool Vec, bool Past, int NSUB, bool None = false>
__device__ __forceinline__ void up_tile(const UpArgs& p, const Tile& sh, int n, uint16_t* lds, uint4* blds,
                                        int64_t (*offs)[kLoraTile]) {
  using Shape = UpShape<TO, RC>;
  constexpr int NP = Shape::kParts, kPitch = Shape::kPitch, kSeg = Shape::kSeg;
  constexpr int kChunks = RC / 8;                         // 8-wide chunks of a part
  constexpr int kSteps = (NP * kChunks + 3) / 4;          // 32-wide steps
  constexpr int kFrags = kChunks >= 4 ? kChunks / 4 : 1;  // different steps of b
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, c = lane & 15, g = lane >> 4;
  const uint16_t* b = p.b + (int64_t)sh.adapter * p.N * p.r;
  const int first = blockIdx.x % p.across * p.n_block;
  const int n_end = first + p.n_block < p.N ? first + p.n_block : p.N;
  int n0 = first + wave * kUpCols;
  uint4 braw[kChunks], base[NSUB][4];
  // without a base the loads read out, and their values are dropped
  const TO* from = p.base ? (const TO*)p.base : (const TO*)p.out;
  const uint32_t keep = p.base ? 0xffffffffu : 0u;
  // the rows' offsets once a tile: a 64-bit product for each load and store
  // took longer than the matrix cores
  if (threadIdx.x < kLoraTile) {
    offs[0][threadIdx.x] = sh.rows[threadIdx.x] * (p.base ? p.ld_base : p.ld_out);
    offs[1][threadIdx.x] = sh.rows[threadIdx.x] * p.ld_out;
  }
  __syncthreads();
  auto load_b = [&](int col0) {
    if constexpr (None) return;
#pragma unroll
    for (int i = 0; i < kChunks; ++i) {
      const int col = col0 + (i % kSeg * 64 + lane) / kSeg;
      braw[i] = load16<uint16_t, true>(b + (int64_t)(col < p.N ? col : p.N - 1) * p.r, (i / kSeg * kSeg + lane % kSeg) * 8,
                                       p.r);
    }
  };
  auto load_base = [&](int ts, int col) {
#pragma unroll
    for (int q = 0; q < 4; ++q)
      base[ts][q] = load4<TO, Vec, Past>(from + offs[0][ts * kSub + 4 * g + q], col, p.N);
  };
  if (n0 < n_end) {
    load_b(n0);
#pragma unroll
    for (int ts = 0; ts < NSUB; ++ts) load_base(ts, n0 + 4 * c);
  }
  if constexpr (!None) {
    up_factor<TO, RC>(p, sh, n, lds);
    __syncthreads();
  }
  auto columns = [&](auto more) {  // more: the wave has another group of columns, whose loads go out
    const int col = n0 + 4 * c;
    bf16x8_t bf[4][kFrags];
    if constexpr (!None) {
      // the 16 rows 4 c + i of a fragment in different banks: row m, chunk k at slot
      // k ^ (m / 4), or in several turns the rows of a fragment together, and chunks
      // exchanged by four rows of it
      auto at = [](int m, int k) {
        if constexpr (Shape::kTurns == 1) return m * kSeg + (k ^ ((m >> 2) & (kSeg - 1)));
        else return ((m & 3) * 16 + ((m >> 2) ^ (m & 3))) * kSeg + (k ^ (m >> 4));
      };
#pragma unroll
      for (int turn = 0; turn < Shape::kTurns; ++turn) {
#pragma unroll
        for (int i = 0; i < kSeg; ++i) blds[at((i * 64 + lane) / kSeg, lane % kSeg)] = braw[turn * kSeg + i];
        wave_lds_fence();
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int k = 0; k < kFrags / Shape::kTurns; ++k)
            bf[i][turn * kFrags / Shape::kTurns + k] = as_bf16x8(blds[at(4 * c + i, (k * 4 + g) % kSeg)]);
        wave_lds_fence();
      }
    }
    const int next = n0 + kWaves * kUpCols;
    if constexpr (decltype(more)::value) load_b(next);
#pragma unroll
    for (int ts = 0; ts < NSUB; ++ts) {
      f32x4_t acc[4];
      uint4 in[4];
#pragma unroll
      for (int q = 0; q < 4; ++q)
        in[q] = make_uint4(base[ts][q].x & keep, base[ts][q].y & keep, base[ts][q].z & keep, base[ts][q].w & keep);
      if constexpr (decltype(more)::value) load_base(ts, next + 4 * c);
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[i] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int k = 0; k < (None ? 0 : kSteps); ++k) {
        const int chunk = k * 4 + g;
        const int q = chunk / kChunks;
        bf16x8_t hf = as_bf16x8(
            *(const uint4*)(lds + ((q < NP ? q : 0) * kLoraTile + ts * kSub + c) * kPitch + (chunk % kChunks) * 8));
        if (kSteps * 4 > NP * kChunks && q >= NP) hf = as_bf16x8(make_uint4(0, 0, 0, 0));
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[i] = mfma16x16x32(hf, bf[i][k % kFrags], acc[i]);
      }
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int t = ts * kSub + 4 * g + q;
        uint4 d = in[q];
        if constexpr (None) {
        } else if constexpr (sizeof(TO) == 4) {
          d = make_uint4(__float_as_uint(__uint_as_float(in[q].x) + acc[0][q]),
                         __float_as_uint(__uint_as_float(in[q].y) + acc[1][q]),
                         __float_as_uint(__uint_as_float(in[q].z) + acc[2][q]),
                         __float_as_uint(__uint_as_float(in[q].w) + acc[3][q]));
        } else {
          d.x = bf16_pair(__uint_as_float(in[q].x << 16) + acc[0][q], __uint_as_float(in[q].x & 0xffff0000u) + acc[1][q]);
          d.y = bf16_pair(__uint_as_float(in[q].y << 16) + acc[2][q], __uint_as_float(in[q].y & 0xffff0000u) + acc[3][q]);
        }
        if (t < n) store4<TO, Vec, Past>((TO*)p.out + offs[1][t], col, p.N, d);
      }
    }
    n0 = next;
  };
  while (n0 + kWaves * kUpCols < n_end) columns(std::true_type{});
  if (n0 < n_end) columns(std::false_type{});
}

template <typename TO, int RC, bool Vec, bool Past>
__global__ __launch_bounds__(kThreads, (UpShape<TO, RC>::kWorkgroups)) void lora_up_kernel(UpArgs p) {
  __shared__ __align__(16) Tile sh;
  __shared__ __align__(16) uint16_t lds[UpShape<TO, RC>::kParts * kLoraTile * UpShape<TO, RC>::kPitch];
  __shared__ uint4 blds[kWaves][kUpCols * UpShape<TO, RC>::kSeg];
  const int n = find_tile(p.tile, sh, blockIdx.x / p.across);
  if (n == 0) return;
  const bool none = sh.adapter == p.tile.L;
  if (none && p.base == p.out) return;  // in place
  __shared__ __align__(16) int64_t offs[2][kLoraTile];
  uint4* mine = blds[threadIdx.x >> 6];
  if (none) up_tile<TO, RC, Vec, Past, 4, true>(p, sh, n, lds, mine, offs);
  else if (n <= 16) up_tile<TO, RC, Vec, Past, 1>(p, sh, n, lds, mine, offs);
  else if (n <= 32) up_tile<TO, RC, Vec, Past, 2>(p, sh, n, lds, mine, offs);
  else up_tile<TO, RC, Vec, Past, 4>(p, sh, n, lds, mine, offs);
}

// ------------------------------------------------------------------ join
// Of 16 ranks from j0: the three bf16 parts of scale * (sum of the splits of
// part) as outer's fragments, [32 positions of the grouping][part][16 ranks]
// [lane], lane (g, c) holding positions 8 g .. + 7 of rank c; zeros at the tile's
// padding. dh, if asked for, receives the scaled sums.
__device__ __forceinline__ void rank_major(const TileArgs& tile, const Tile& sh, int n, int index, int r, int j0,
                                           const float* part, int splits, const float* scales, float* dh, uint16_t* vt,
                                           float (*lds)[20]) {
  const int tid = threadIdx.x;
  const float scale = scales ? scales[sh.adapter] : 1.0f;
  {
    const int t = tid / 4, j = j0 + tid % 4 * 4;
    float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (t < n && j < r) {
      const int64_t at = (int64_t)sh.rows[t] * r + j;
#pragma unroll 8
      for (int s = 0; s < splits; ++s) {
        const float4 x = *(const float4*)(part + (int64_t)s * tile.M * r + at);
        v.x += x.x; v.y += x.y; v.z += x.z; v.w += x.w;
      }
      v = make_float4(v.x * scale, v.y * scale, v.z * scale, v.w * scale);
      if (dh) *(float4*)(dh + at) = v;
    }
    *(float4*)&lds[t][tid % 4 * 4] = v;
  }
  __syncthreads();
  if (tid >= 128) return;
  const int lane = tid & 63, half = tid >> 6;
  const int t = half * 32 + (lane >> 4) * 8;
  float f[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) f[e] = lds[t + e][lane & 15];
  bf16x8_t q[3];
  split_parts<3>(f, q);
  const int ranks = (r + 15) / 16;
#pragma unroll
  for (int e = 0; e < 3; ++e)
    *(uint4*)(vt + ((((int64_t)index * 2 + half) * 3 + e) * ranks + j0 / 16) * 512 + lane * 8) =
        __builtin_bit_cast(uint4, q[e]);
}

// dh: the sum of its splits, scaled, as it is and rank-major (even blockIdx.y);
// s h rank-major (odd). blockIdx.y / 2: 16 ranks. outer would otherwise make the
// parts once for each 128 columns. Bound by latency: 7.1 us for 8192 rows of
// rank 64, 3.5 to 4 for 1000 to 2000 of ranks up to 32 (with all ranks in one
// workgroup 8.4 and 4.9).
struct JoinArgs {
  TileArgs tile;
  int r, splits;
  const float* part;          // [splits][M][r]
  const float* scales;
  float* dh;                  // [M][r]
  uint16_t* dht;
  const float* h;             // [M][r]
  uint16_t* ht;
};
__global__ __launch_bounds__(kThreads) void lora_join_kernel(JoinArgs p) {
  __shared__ __align__(16) Tile sh;
  __shared__ __align__(16) float lds[kLoraTile][20];
  const int n = find_tile(p.tile, sh, blockIdx.x);
  if (n == 0 || sh.adapter == p.tile.L) return;
  const int j0 = blockIdx.y / 2 * 16;
  if (blockIdx.y % 2 == 0) rank_major(p.tile, sh, n, blockIdx.x, p.r, j0, p.part, p.splits, p.scales, p.dh, p.dht, lds);
  else rank_major(p.tile, sh, n, blockIdx.x, p.r, j0, p.h, 1, p.scales, nullptr, p.ht, lds);
}

// ------------------------------------------------------------------ outer
struct OuterSide {
  const void* u;              // [M, W]
  int64_t ldu;
  int W;
  const uint16_t* vt;         // fragments, as rank_major writes them
  float* out;                 // [L][r][W], or [L][W][r] (rank_minor)
  float* slots;               // [2 * chunks] of the same shape
  int chunk;                  // positions per workgroup, a multiple of 64
  int chunks;
};
struct OuterArgs {
  int r, M, L;
  int64_t cap;
  const int32_t* sorted;
  const int4* tiles;
  OuterSide a, b;             // dA (x, bf16), dB (the output side, either type)
  int b_blocks;               // workgroups of dB, before those of dA
};

constexpr int kPiece = 1024;  // positions whose rows are in LDS at a time

// sum over an adapter's rows of u[row][w] * v[row][j], for 128 columns and up
// to 64 ranks a workgroup. A step takes 32 positions: lane (g, c) loads 8
// columns from 8 c of its 8 rows and transposes that 8 x 8 block in registers
// (the contraction runs over rows); the four waves take an adapter's steps in
// turn and join their sums in LDS. The positions are cut into chunks whatever
// the adapters' lengths, so the work is even; sums of an adapter within one
// chunk go to the output, those of one that crosses the chunk's start or end to
// slots 2 c or 2 c + 1, which the reduce kernel adds in order. Ranks above 64
// are further workgroups, eight apart: on the same XCD, whose L2 has the columns.
// x and grad_out of [8192, 7168], rank 64, 68 us: their 235 MB at 3.5 TB/s, where a
// read reaches 7. Beside them come 12 KB of factor parts from L2 for each 8 KB of a
// side (rank 64: 352 MB), and the two waves of a rank pair load the same side; one
// wave or two a SIMD, loads one to three steps ahead and 32 ranks a wave or 64 leave
// that as it is and were within 15 % of each other. [1999, 7168] and [1999, 2048]
// of rank 16 13 us. An fp32 side enters as three parts, of whose products with the
// factor's three all are taken but the last with the last (2^-32 of the whole; a
// part is up to 2^-8 of the one before it, and fp32 rounds a product by 2^-24).
template <typename TU, int JT, int H, bool VecU, bool RankMinor>
__device__ __forceinline__ void outer_block(const OuterArgs& p, const OuterSide& side, int block,
                                            f32x4_t (*joined)[8 * JT][64], int64_t* offs) {
  constexpr bool kF32 = std::is_same<TU, float>::value;
  constexpr int kVecs = 8 * JT;                         // accumulators of a wave
  constexpr int kTurns = kWaves / H;                    // waves that take turns at the positions
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, c = lane & 15, g = lane >> 4;
  // XCD x (workgroups x, x + 8, ...) takes an eighth of the column blocks, those
  // of a chunk one after another: together the XCDs read whole rows
  const int across = (side.W + 127) / 128, part = (across + 7) / 8;
  const int zs = (p.r + 16 * JT * H - 1) / (16 * JT * H);
  const int at = block / 8 / zs;
  const int w0 = (block % 8 * part + at % part) * 128;
  const int chunk = at / part;
  if (w0 >= side.W) return;
  const int turn = wave / H;
  const int j0 = (block / 8 % zs * H + wave % H) * 16 * JT;
  const int ranks = (p.r + 15) / 16;
  const int p0 = chunk * side.chunk;
  const int p1 = p0 + side.chunk < p.cap ? p0 + side.chunk : (int)p.cap;
  f32x4_t acc[8][JT];

  struct Frags {
    uint32_t d[kF32 ? 1 : 8][4];
    float f[kF32 ? 8 : 1][8];
    bf16x8_t v[JT][3];
  };
  auto load = [&](int pos, int piece, Frags& x) {
#pragma unroll
    for (int t = 0; t < 8; ++t) {
      const TU* row = (const TU*)side.u + offs[pos - piece + 8 * g + t];
      if constexpr (kF32) {
        const uint4 lo = load16<float, VecU, false>((const float*)row, w0 + 8 * c, side.W);
        const uint4 hi = load16<float, VecU, false>((const float*)row, w0 + 8 * c + 4, side.W);
        x.f[t][0] = __uint_as_float(lo.x); x.f[t][1] = __uint_as_float(lo.y);
        x.f[t][2] = __uint_as_float(lo.z); x.f[t][3] = __uint_as_float(lo.w);
        x.f[t][4] = __uint_as_float(hi.x); x.f[t][5] = __uint_as_float(hi.y);
        x.f[t][6] = __uint_as_float(hi.z); x.f[t][7] = __uint_as_float(hi.w);
      } else {
        const uint4 v = load16<uint16_t, VecU, false>((const uint16_t*)row, w0 + 8 * c, side.W);
        x.d[t][0] = v.x; x.d[t][1] = v.y; x.d[t][2] = v.z; x.d[t][3] = v.w;
      }
    }
#pragma unroll
    for (int jt = 0; jt < JT; ++jt) {
      const int at = j0 / 16 + jt < ranks ? j0 / 16 + jt : ranks - 1;
#pragma unroll
      for (int q = 0; q < 3; ++q)
        x.v[jt][q] = as_bf16x8(*(const uint4*)(side.vt + (((int64_t)(pos / 32) * 3 + q) * ranks + at) * 512 + lane * 8));
    }
  };
  auto multiply = [&](const Frags& x) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      auto mac = [&](bf16x8_t uf, int q) {
#pragma unroll
        for (int jt = 0; jt < JT; ++jt) acc[i][jt] = mfma16x16x32(x.v[jt][q], uf, acc[i][jt]);
      };
      if constexpr (kF32) {
        const float col[8] = {x.f[0][i], x.f[1][i], x.f[2][i], x.f[3][i], x.f[4][i], x.f[5][i], x.f[6][i], x.f[7][i]};
        bf16x8_t uf[3];
        split_parts<3>(col, uf);
        mac(uf[0], 0);
        mac(uf[0], 1);
        mac(uf[0], 2);
        mac(uf[1], 0);
        mac(uf[1], 1);
        mac(uf[1], 2);
        mac(uf[2], 0);
        mac(uf[2], 1);
      } else {
        // 16-bit element i of rows 2m and 2m + 1
        const uint32_t sel = (i & 1) ? 0x07060302u : 0x05040100u;
        const bf16x8_t uf = as_bf16x8(make_uint4(__builtin_amdgcn_perm(x.d[1][i / 2], x.d[0][i / 2], sel),
                                                 __builtin_amdgcn_perm(x.d[3][i / 2], x.d[2][i / 2], sel),
                                                 __builtin_amdgcn_perm(x.d[5][i / 2], x.d[4][i / 2], sel),
                                                 __builtin_amdgcn_perm(x.d[7][i / 2], x.d[6][i / 2], sel)));
        mac(uf, 0);
        mac(uf, 1);
        mac(uf, 2);
      }
    }
  };

  for (int s0 = p0; s0 < p1;) {
    // an adapter's positions in the chunk; the last list (rows without an
    // adapter) and the room behind it have nothing
    const int4 info = p.tiles[s0 / kLoraTile];
    if (info.y == 0 || info.x == p.L) return;
    const int adapter = info.x, o0 = info.z, o1 = info.w;
    const int s1 = o1 < p1 ? o1 : p1;
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int jt = 0; jt < JT; ++jt) acc[i][jt] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
    for (int piece = s0; piece < s1; piece += kPiece) {
      const int end = piece + kPiece < s1 ? piece + kPiece : s1;
      __syncthreads();
      // padding repeats its tile's first row, whose factors there are 0: what
      // is not finite in that row is in this adapter's sums anyway
      for (int i = threadIdx.x; i < end - piece; i += kThreads) {
        const int row = p.sorted[piece + i], first = p.sorted[(piece + i) / kLoraTile * kLoraTile];
        offs[i] = (row < p.M ? row : first) * side.ldu;
      }
      __syncthreads();
      int pos = piece + 32 * turn;
      if (pos < end) {
        constexpr int kStep = 32 * kTurns;
        if constexpr (!kF32) {
          // The next step's loads are in flight during this one's products. No
          // load of the loop hangs on a condition, so each wait is for its own
          // step, and the barriers keep the compiler from mixing the steps.
          Frags f0, f1;
          load(pos, piece, f0);
          for (; pos + 2 * kStep < end; pos += 2 * kStep) {
            load(pos + kStep, piece, f1);
            __builtin_amdgcn_sched_barrier(0);
            multiply(f0);
            __builtin_amdgcn_sched_barrier(0);
            load(pos + 2 * kStep, piece, f0);
            __builtin_amdgcn_sched_barrier(0);
            multiply(f1);
            __builtin_amdgcn_sched_barrier(0);
          }
          if (pos + kStep < end) load(pos + kStep, piece, f1);
          multiply(f0);
          if (pos + kStep < end) multiply(f1);
        } else {
          for (; pos < end; pos += kStep) {
            Frags f;
            load(pos, piece, f);
            multiply(f);
          }
        }
      }
    }
    // join: lane (g, c) has columns 8 c + i, ranks 16 jt + 4 g + q. Four
    // accumulators (half of i, one jt) go to one wave.
    const int64_t size = (int64_t)p.r * side.W;
    float* out = (o0 >= p0 && o1 <= p0 + side.chunk) ? side.out + adapter * size
                                                     : side.slots + (2 * (int64_t)chunk + (o0 < p0 ? 0 : 1)) * size;
#pragma unroll
    for (int v = 0; v < kVecs; ++v) joined[wave][v][lane] = acc[v % 8][v / 8];
    __syncthreads();
    for (int v = turn * 4; v < kVecs; v += kTurns * 4) {
      f32x4_t sum[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        sum[i] = joined[wave % H][v + i][lane];
#pragma unroll
        for (int w = 1; w < kTurns; ++w) sum[i] += joined[w * H + wave % H][v + i][lane];
      }
      const int w = w0 + 8 * c + v % 8, j = j0 + 16 * (v / 8) + 4 * g;
      if (j < p.r) {
        if constexpr (RankMinor) {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (w + i < side.W) *(f32x4_t*)(out + (int64_t)(w + i) * p.r + j) = sum[i];
        } else {
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            float* to = out + (int64_t)(j + q) * side.W + w;
            if (w < side.W) *(f32x4_t*)to = f32x4_t{sum[0][q], sum[1][q], sum[2][q], sum[3][q]};
          }
        }
      }
    }
    __syncthreads();
    s0 = s1;
  }
}

template <typename TU, int JT, int H, bool VecU>
__global__ __launch_bounds__(kThreads, 2) void lora_outer_kernel(OuterArgs p) {
  __shared__ f32x4_t joined[kWaves][8 * JT][64];
  __shared__ __align__(16) int64_t offs[kPiece];
  if ((int)blockIdx.x < p.b_blocks) outer_block<TU, JT, H, VecU, true>(p, p.b, blockIdx.x, joined, offs);
  else outer_block<uint16_t, JT, H, true, false>(p, p.a, blockIdx.x - p.b_blocks, joined, offs);
}

// Adapters that cross chunks: their slots, in order; adapters without rows:
// zeros. blockIdx.z: dA, dB. 8 us for one adapter of rank 64 and [7168] both
// sides in 9 chunks (33 MB of partial sums, which the caches still hold).
struct ReduceArgs {
  const int32_t* offsets;
  int64_t size[2];
  int chunk[2];
  const float* slots[2];
  float* out[2];
};
__global__ __launch_bounds__(kThreads) void lora_reduce_kernel(ReduceArgs p) {
  const int a = blockIdx.y, z = blockIdx.z;
  const int o0 = p.offsets[a], o1 = p.offsets[a + 1];
  const int chunk = p.chunk[z];
  const int c0 = o0 / chunk, c1 = o1 > o0 ? (o1 - 1) / chunk : c0;
  if (o1 > o0 && c0 == c1) return;
  const int64_t size = p.size[z];
  const float* slots = p.slots[z];
  for (int64_t i = ((int64_t)blockIdx.x * kThreads + threadIdx.x) * 4; i < size;
       i += (int64_t)gridDim.x * kThreads * 4) {
    float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (o1 > o0) {
      v = *(const float4*)(slots + (2 * (int64_t)c0 + 1) * size + i);
#pragma unroll 4
      for (int c = c0 + 1; c <= c1; ++c) {
        const float4 x = *(const float4*)(slots + 2 * (int64_t)c * size + i);
        v.x += x.x; v.y += x.y; v.z += x.z; v.w += x.w;
      }
    }
    *(float4*)(p.out[z] + a * size + i) = v;
  }
}

// ------------------------------------------------------------------ launches
bool vec_ok(const void* p, int64_t ld, bool f32) {
  return !p || ((reinterpret_cast<uintptr_t>(p) & 15) == 0 && ld % (f32 ? 4 : 8) == 0);
}

hipError_t launch_down(DownArgs p, bool u_f32, int tiles, hipStream_t stream) {
  const bool vec = vec_ok(p.u, p.ldu, u_f32) && p.W % (u_f32 ? 4 : 8) == 0;
  p.split_steps = (int)ceil_div(ceil_div(p.W, u_f32 ? 32 : 64), p.splits);
  const dim3 grid(tiles, p.splits);
  auto go = [&](auto rt) {
    constexpr int RT = decltype(rt)::value;
    if (u_f32) {
      if (vec) lora_down_kernel<float, RT, true><<<grid, kThreads, 0, stream>>>(p);
      else lora_down_kernel<float, RT, false><<<grid, kThreads, 0, stream>>>(p);
    } else {
      if (vec) lora_down_kernel<uint16_t, RT, true><<<grid, kThreads, 0, stream>>>(p);
      else lora_down_kernel<uint16_t, RT, false><<<grid, kThreads, 0, stream>>>(p);
    }
  };
  if (p.r <= 16) go(std::integral_constant<int, 1>{});
  else if (p.r <= 32) go(std::integral_constant<int, 2>{});
  else if (p.r <= 64) go(std::integral_constant<int, 4>{});
  else go(std::integral_constant<int, 8>{});
  return hipGetLastError();
}

// past: base and out need not stay in the caches (bf16).
hipError_t launch_up(UpArgs p, bool out_f32, bool past, int tiles, hipStream_t stream) {
  const bool vec = vec_ok(p.base, p.ld_base, out_f32) && vec_ok(p.out, p.ld_out, out_f32) &&
                   p.N % (out_f32 ? 4 : 8) == 0;
  // as many workgroups as the chip holds at once (by their registers and LDS),
  // each going on to further columns with its next loads in flight; the column
  // blocks of a tile are neighbours, so that together they read whole rows
  // (rank 16, [1999, 7168]: 24 us with the tiles as neighbours, 15 so)
  const int64_t cols = ceil_div(p.N, kWaves * kUpCols);
  int64_t across = 256 * (p.r <= 64 ? 3 : (out_f32 ? 1 : 2)) / tiles;
  across = across < 1 ? 1 : (across > cols ? cols : across);
  p.n_block = (int)(ceil_div(cols, across) * kWaves * kUpCols);
  p.across = (int)ceil_div(p.N, p.n_block);
  const unsigned grid = (unsigned)(p.across * (int64_t)tiles);
  auto go = [&](auto rc) {
    constexpr int RC = decltype(rc)::value;
    if (out_f32) {
      if (vec) lora_up_kernel<float, RC, true, false><<<grid, kThreads, 0, stream>>>(p);
      else lora_up_kernel<float, RC, false, false><<<grid, kThreads, 0, stream>>>(p);
    } else {
      if (vec && past) lora_up_kernel<uint16_t, RC, true, true><<<grid, kThreads, 0, stream>>>(p);
      else if (vec) lora_up_kernel<uint16_t, RC, true, false><<<grid, kThreads, 0, stream>>>(p);
      else lora_up_kernel<uint16_t, RC, false, false><<<grid, kThreads, 0, stream>>>(p);
    }
  };
  if (p.r <= 8) go(std::integral_constant<int, 8>{});
  else if (p.r <= 16) go(std::integral_constant<int, 16>{});
  else if (p.r <= 32) go(std::integral_constant<int, 32>{});
  else if (p.r <= 64) go(std::integral_constant<int, 64>{});
  else go(std::integral_constant<int, 128>{});
  return hipGetLastError();
}

hipError_t launch_outer(OuterArgs p, bool b_f32, hipStream_t stream) {
  const bool vec = vec_ok(p.b.u, p.b.ldu, b_f32) && p.b.W % (b_f32 ? 4 : 8) == 0;
  const int64_t zs = ceil_div(p.r, 64);
  p.a.chunks = (int)ceil_div(p.cap, p.a.chunk);
  p.b.chunks = (int)ceil_div(p.cap, p.b.chunk);
  const int64_t b_blocks = ceil_div(ceil_div(p.b.W, 128), 8) * 8 * p.b.chunks * zs;
  const int64_t blocks = b_blocks + ceil_div(ceil_div(p.a.W, 128), 8) * 8 * p.a.chunks * zs;
  p.b_blocks = (int)b_blocks;
  auto go = [&](auto jt, auto h) {
    constexpr int JT = decltype(jt)::value, H = decltype(h)::value;
    if (b_f32 && vec) lora_outer_kernel<float, JT, H, true><<<(unsigned)blocks, kThreads, 0, stream>>>(p);
    else if (b_f32) lora_outer_kernel<float, JT, H, false><<<(unsigned)blocks, kThreads, 0, stream>>>(p);
    else if (vec) lora_outer_kernel<uint16_t, JT, H, true><<<(unsigned)blocks, kThreads, 0, stream>>>(p);
    else lora_outer_kernel<uint16_t, JT, H, false><<<(unsigned)blocks, kThreads, 0, stream>>>(p);
  };
  using One = std::integral_constant<int, 1>;
  using Two = std::integral_constant<int, 2>;
  if (p.r <= 16) go(One{}, One{});
  else if (p.r <= 32) go(Two{}, One{});
  else go(Two{}, Two{});
  return hipGetLastError();
}

int64_t align256(int64_t v) { return (v + 255) & ~int64_t(255); }

}  // namespace

LoraLayout lora_layout(int64_t M, int64_t L, int64_t K, int64_t N, int64_t r, bool backward) {
  LoraLayout o{};
  o.small = !backward && M <= kLoraSmallRows;
  const int64_t lists = M < L + 1 ? M : L + 1;  // adapters with rows, and the rows without one
  o.cap = ceil_div(M + lists * (kLoraTile - 1), kLoraTile) * kLoraTile;
  // a small batch has no padded lists: at most one tile per list and 64 rows
  o.tiles = (int)(o.small ? (M < M / kLoraTile + lists ? M : M / kLoraTile + lists) : o.cap / kLoraTile);
  // splits of the contraction: as many workgroups as the chip holds at once, two
  // a CU (8192 rows of rank 64: 256 workgroups 43 us, 384 35, 512 31, 700 40, 1024
  // 37), each wave at least one step, and no more than 8 partial sums to add (16:
  // 64 rows of rank 16 11 us instead of 8)
  const int64_t steps = ceil_div(backward ? N : K, 64);
  // (the tiles of a batch are M / 64 and part of one for each adapter with rows)
  const int64_t full = ceil_div(M, kLoraTile);
  int64_t splits = M > 0 ? 512 / (full + (L - 1 < full ? L - 1 : full) / 4) : 1;
  if (splits < 1) splits = 1;
  if (splits > 8) splits = 8;
  if (splits > ceil_div(steps, kWaves)) splits = ceil_div(steps, kWaves);
  o.splits = (int)ceil_div(steps, ceil_div(steps, splits));
  int64_t at = 0;
  auto take = [&](int64_t bytes) {
    const int64_t off = at;
    at += align256(bytes);
    return off;
  };
  // room for what any smaller batch takes too: splits * M <= 512 * 64 unless splits = 1
  const int64_t part_rows = 8 * M < 512 * kLoraTile ? 8 * M : 512 * kLoraTile;
  o.part_off = take((M > part_rows ? M : part_rows) * r * 4);
  if (!o.small) {
    o.sorted_off = take(o.cap * 4);
    o.block_off = take(o.cap / kLoraTile * 16);
    o.offs_off = take((L + 2) * 4);
    if (!backward) o.h_off = take(M * r * 4);
  }
  if (backward) {
    o.n_pad = ceil_div(N, 8) * 8;
    o.at_off = take(L * K * r * 2);
    o.bt_off = take(L * r * o.n_pad * 2);
    o.dh_off = take(M * r * 4);
    o.dht_off = take(3 * ceil_div(r, 16) * 16 * o.cap * 2);
    o.ht_off = take(3 * ceil_div(r, 16) * 16 * o.cap * 2);
    // positions per workgroup of the weight gradients: as many workgroups as
    // the chip holds at once, two a CU, so that partial sums are few; at least
    // one step for each wave
    auto slots = [&](int64_t W, int& chunk) {
      const int64_t across = ceil_div(W, 128) * ceil_div(r, 64);
      int64_t cuts = 512 / across;
      cuts = cuts < 1 ? 1 : cuts;
      const int64_t c = ceil_div(o.cap, cuts);
      chunk = (int)(ceil_div(c > 128 ? c : 128, kLoraTile) * kLoraTile);
      const int64_t most = ceil_div(o.cap, 128);
      return take(2 * (most < cuts ? most : cuts) * r * W * 4);
    };
    o.a_slots_off = slots(K, o.a_chunk);
    o.b_slots_off = slots(N, o.b_chunk);
  }
  o.total = at;
  return o;
}

namespace {

// The grouping (none for a small batch) and the arguments that name it.
hipError_t group_rows(const LoraArgs& a, const LoraLayout& o, const TransposeArgs& weights, TileArgs& t,
                      hipStream_t stream) {
  t = TileArgs{};
  t.ids = a.ids; t.M = a.M; t.L = a.L;
  if (o.small) return hipSuccess;
  GroupArgs g{};
  g.ids = a.ids; g.M = a.M; g.L = a.L;
  g.sorted = (int32_t*)(a.ws + o.sorted_off);
  g.tiles = (int4*)(a.ws + o.block_off);
  g.offsets = (int32_t*)(a.ws + o.offs_off);
  g.all_tiles = o.tiles;
  t.sorted = g.sorted; t.tiles = g.tiles;
  int64_t more = a.M > 0 ? (a.M < a.L ? a.M : a.L) * (int64_t)(weights.a_blocks + weights.b_blocks) : 0;
  if (more > 511) more = 511;  // with the grouping, two workgroups a CU
  lora_group_kernel<<<(unsigned)(1 + more), kGroupThreads, 0, stream>>>(g, weights);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_lora_forward(const LoraArgs& a, hipStream_t stream) {
  const LoraLayout o = lora_layout(a.M, a.L, a.K, a.N, a.r, false);
  TileArgs t;
  hipError_t err = group_rows(a, o, TransposeArgs{}, t, stream);
  if (err != hipSuccess) return err;
  DownArgs d{};
  d.tile = t;
  d.u = a.x; d.ldu = a.ldx; d.W = a.K;
  d.v = a.a; d.v_stride = (int64_t)a.r * a.K; d.ldv = a.K; d.r = a.r;
  d.splits = o.splits;
  d.part = (float*)(a.ws + o.part_off); d.h = a.h;
  UpArgs u{};
  u.tile = t; u.r = a.r; u.N = a.N;
  u.b = a.b; u.base = a.base; u.ld_base = a.ld_base; u.out = a.out; u.ld_out = a.ld_out;
  u.part = d.part; u.splits = o.splits; u.scales = a.scales; u.h = a.h;
  err = launch_down(d, false, o.tiles, stream);
  if (err != hipSuccess) return err;
  // up's workgroups each add their tile's splits again; where that is more than
  // the rest of what they read (64 rows of a few hundred columns), a launch of
  // its own does it once (4096 rows of rank 64: 5 + 33 us instead of more than 60)
  if (o.splits * a.r > 128 && !o.small) {
    float* h = a.h ? a.h : (float*)(a.ws + o.h_off);
    const int64_t size = (int64_t)a.M * a.r;
    lora_sum_kernel<<<(unsigned)ceil_div(size, 4 * kThreads), kThreads, 0, stream>>>(d.part, o.splits, size, a.r, a.ids,
                                                                                    a.L, h);
    if ((err = hipGetLastError()) != hipSuccess) return err;
    u.part = h; u.splits = 1; u.h = nullptr;
  }
  return launch_up(u, a.y_f32, false, o.tiles, stream);
}

hipError_t launch_lora_backward(const LoraArgs& a, hipStream_t stream) {
  const LoraLayout o = lora_layout(a.M, a.L, a.K, a.N, a.r, true);
  TransposeArgs f{};
  f.a = a.a; f.b = a.b; f.K = a.K; f.N = a.N; f.r = a.r; f.n_pad = o.n_pad;
  f.at = (uint16_t*)(a.ws + o.at_off); f.bt = (uint16_t*)(a.ws + o.bt_off);
  const int64_t ranks = ceil_div(a.r, 64);
  f.a_blocks = a.dx ? (int)(ranks * ceil_div(a.K, 64)) : 0;
  f.b_blocks = (int)(ranks * ceil_div(o.n_pad, 64));
  TileArgs t;
  hipError_t err = group_rows(a, o, f, t, stream);
  if (err != hipSuccess) return err;
  ReduceArgs red{};
  red.offsets = (const int32_t*)(a.ws + o.offs_off);
  red.size[0] = (int64_t)a.r * a.K; red.size[1] = (int64_t)a.r * a.N;
  red.chunk[0] = o.a_chunk; red.chunk[1] = o.b_chunk;
  red.slots[0] = (float*)(a.ws + o.a_slots_off); red.slots[1] = (float*)(a.ws + o.b_slots_off);
  red.out[0] = a.da; red.out[1] = a.db;
  if (a.M > 0) {
    DownArgs d{};
    d.tile = t;
    d.u = a.dout; d.ldu = a.ld_dout; d.W = a.N;
    d.v = f.bt; d.v_stride = a.r * o.n_pad; d.ldv = o.n_pad; d.r = a.r;
    d.splits = o.splits;
    d.part = (float*)(a.ws + o.part_off);
    if ((err = launch_down(d, a.y_f32, o.tiles, stream)) != hipSuccess) return err;
    JoinArgs j{};
    j.tile = t; j.r = a.r; j.splits = o.splits; j.part = d.part; j.scales = a.scales;
    j.dh = (float*)(a.ws + o.dh_off); j.dht = (uint16_t*)(a.ws + o.dht_off);
    j.h = a.h; j.ht = (uint16_t*)(a.ws + o.ht_off);
    lora_join_kernel<<<dim3(o.tiles, 2 * (unsigned)ceil_div(a.r, 16)), kThreads, 0, stream>>>(j);
    if ((err = hipGetLastError()) != hipSuccess) return err;
    OuterArgs w{};
    w.r = a.r; w.M = a.M; w.L = a.L; w.cap = o.cap; w.sorted = t.sorted; w.tiles = t.tiles;
    w.a.u = a.x; w.a.ldu = a.ldx; w.a.W = a.K; w.a.vt = j.dht; w.a.out = a.da;
    w.a.slots = (float*)(a.ws + o.a_slots_off); w.a.chunk = o.a_chunk;
    w.b.u = a.dout; w.b.ldu = a.ld_dout; w.b.W = a.N; w.b.vt = j.ht; w.b.out = a.db;
    w.b.slots = (float*)(a.ws + o.b_slots_off); w.b.chunk = o.b_chunk;
    if ((err = launch_outer(w, a.y_f32, stream)) != hipSuccess) return err;
    if (a.dx) {
      // last, so that outer finds grad_out where down left it, in the 256 MB cache
      // (8192 rows of [7168] twice, rank 64: outer 81 us after dx, 71 before it).
      // A call that moves more than the cache holds keeps dx and its base out of
      // it: their write-back fell into the next kernels (193 us in all, 185 so).
      const bool past = 6 * (int64_t)a.M * a.K + (a.y_f32 ? 4 : 2) * (int64_t)a.M * a.N > (int64_t(256) << 20);
      UpArgs u{};
      u.tile = t; u.r = a.r; u.N = a.K; u.part = j.dh; u.splits = 1;
      u.b = f.at; u.base = a.dx_base; u.ld_base = a.ld_dx_base; u.out = a.dx; u.ld_out = a.ld_dx;
      if ((err = launch_up(u, false, past, o.tiles, stream)) != hipSuccess) return err;
    }
  }
  const int64_t widest = red.size[0] > red.size[1] ? red.size[0] : red.size[1];
  int64_t blocks = ceil_div(widest, 4 * kThreads);
  if (blocks > 1024) blocks = 1024;
  lora_reduce_kernel<<<dim3((unsigned)blocks, (unsigned)a.L, 2), kThreads, 0, stream>>>(red);
  return hipGetLastError();
}

}  // namespace moe
