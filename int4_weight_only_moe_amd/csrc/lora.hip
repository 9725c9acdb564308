// Low-rank adapters of many requests beside a shared projection.
//
// Row t of the batch belongs to a request with adapter a = ids[t] (A_a [r, K],
// B_a [N, r], scale s_a), or to one without (ids[t] outside [0, L)):
//   h_t  = A_a x_t                         out_t = base_t + s_a B_a h_t
//   dh_t = s_a B_a^T dout_t                dx_t  = dxbase_t + A_a^T dh_t
//   dA_a = sum_t dh_t x_t^T                dB_a  = s_a sum_t dout_t h_t^T
//
// The rows are grouped by adapter as the layer groups its assignments by
// expert: lists padded to 64 rows, so a workgroup's tile holds rows of one
// adapter. Four kernels do the products on the matrix cores:
//   down    contracts a wide side with a [r, W] operand (h, dh): fp32 partial
//           sums of each split of W;
//   up      expands r values to a wide side and adds the base (out, dx);
//   finish  adds dh's partial sums and lays dh and s h out rank-major;
//   outer   sums rows' outer products (dA, dB).
// With r <= 128 every one of them moves the wide side once and is bound by
// that traffic, so the products are made exact where that is free: bf16
// operands multiply exactly into fp32, and an fp32 factor (h, dh, an fp32
// side) enters as bf16 parts of 8 bits each, three (24 bits: all of fp32)
// where the result is fp32, two (16 bits, 2^-17 relative: 2^-8 of what the
// result's rounding costs) where it is bf16.
#include <type_traits>

#include "device_common.h"
#include "operators.h"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;
constexpr int kSub = 16;  // rows of a matrix-core tile

__device__ __forceinline__ uint32_t bf16_bits(float v) {
  return (uint32_t)__builtin_bit_cast(uint16_t, (__bf16)v);
}
__device__ __forceinline__ float bf16_value(uint32_t bits) { return __uint_as_float(bits << 16); }

// Eight fp32 values as NP bf16 parts, v = parts[0] + parts[1] + ...: each part
// is the rounding of what the parts before it leave.
template <int NP>
__device__ __forceinline__ void split_parts(const float (&v)[8], bf16x8_t (&parts)[NP]) {
  float rest[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) rest[i] = v[i];
#pragma unroll
  for (int p = 0; p < NP; ++p) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      parts[p][i] = (__bf16)rest[i];
      rest[i] -= (float)parts[p][i];
    }
  }
}

// Eight consecutive elements from column w of a row of W elements, zeros past
// the row's end. Vec: the row is 16-byte aligned and W % 8 == 0 (bf16) or
// W % 4 == 0 (fp32).
template <bool Vec>
__device__ __forceinline__ bf16x8_t load8(const uint16_t* __restrict__ row, int w, int W) {
  if constexpr (Vec) {
    uint4 v = *(const uint4*)(row + (w < W ? w : 0));
    if (w >= W) v = make_uint4(0, 0, 0, 0);
    return as_bf16x8(v);
  } else {
    uint32_t e[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t x = row[w + i < W ? w + i : 0];
      e[i] = w + i < W ? x : 0u;
    }
    return as_bf16x8(make_uint4(e[0] | e[1] << 16, e[2] | e[3] << 16, e[4] | e[5] << 16, e[6] | e[7] << 16));
  }
}
template <bool Vec>
__device__ __forceinline__ void load8(const float* __restrict__ row, int w, int W, float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 8; i += 4) {
    if constexpr (Vec) {
      const float4 x = *(const float4*)(row + (w + i < W ? w + i : 0));
      v[i] = w + i < W ? x.x : 0.0f;
      v[i + 1] = w + i < W ? x.y : 0.0f;
      v[i + 2] = w + i < W ? x.z : 0.0f;
      v[i + 3] = w + i < W ? x.w : 0.0f;
    } else {
#pragma unroll
      for (int q = i; q < i + 4; ++q) {
        const float x = row[w + q < W ? w + q : 0];
        v[q] = w + q < W ? x : 0.0f;
      }
    }
  }
}

// The rows of tile `tile` of the grouping, in LDS: rows past the adapter's
// last repeat the first (their results are dropped). Returns the row count.
__device__ __forceinline__ int load_tile_rows(const int32_t* __restrict__ sorted, int tile, int M, int* rows,
                                              int* count) {
  if (threadIdx.x < 64) {
    const int first = sorted[tile * kLoraTile];
    const int row = sorted[tile * kLoraTile + threadIdx.x];
    rows[threadIdx.x] = row < M ? row : first;
    const uint64_t live = __ballot(row < M);
    if (threadIdx.x == 0) *count = __builtin_popcountll(live);
  }
  __syncthreads();
  return *count;
}

// ------------------------------------------------------------------ down
struct DownArgs {
  const void* u;              // [M, W]
  int64_t ldu;
  int W;
  const uint16_t* v;          // [L][r][ldv], zeros from W to ldv
  int64_t v_stride, ldv;
  int r, M;
  const int32_t* sorted;
  const int32_t* block_adapter;
  const int32_t* npp;
  float* part;                // [splits][M][r]
  int split_steps;            // 64-column steps per split
};

// part[split][row][j] = sum over the split's columns of v[j][w] * u[row][w].
// A step is 64 columns: lane (g, c) takes the 16 columns from 16 g of row c of
// either operand, as two 8-column fragments, so four lanes read 128
// consecutive bytes of a bf16 row. The waves take the split's steps in turn.
template <typename TU, int RT, bool VecU, int NSUB>
__device__ __forceinline__ void down_tile(const DownArgs& p, const int* rows, int adapter, float* red) {
  constexpr int kRed = RT * 16 + 4;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, c = lane & 15, g = lane >> 4;
  const TU* urow[NSUB];
#pragma unroll
  for (int ts = 0; ts < NSUB; ++ts) urow[ts] = (const TU*)p.u + (int64_t)rows[ts * kSub + c] * p.ldu;
  const uint16_t* vrow[RT];
#pragma unroll
  for (int rt = 0; rt < RT; ++rt) {
    const int j = rt * 16 + c < p.r ? rt * 16 + c : p.r - 1;
    vrow[rt] = p.v + adapter * p.v_stride + j * p.ldv;
  }
  f32x4_t acc[RT][NSUB];
#pragma unroll
  for (int rt = 0; rt < RT; ++rt)
#pragma unroll
    for (int ts = 0; ts < NSUB; ++ts) acc[rt][ts] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
  const int steps = (p.W + 63) / 64;
  const int s0 = blockIdx.y * p.split_steps;
  const int s1 = s0 + p.split_steps < steps ? s0 + p.split_steps : steps;
  for (int s = s0 + wave; s < s1; s += kWaves) {
    const int w = s * 64 + g * 16;
    bf16x8_t vf[RT][2];
#pragma unroll
    for (int rt = 0; rt < RT; ++rt)
#pragma unroll
      for (int hh = 0; hh < 2; ++hh) vf[rt][hh] = load8<true>(vrow[rt], w + 8 * hh, (int)p.ldv);
    if constexpr (std::is_same<TU, float>::value) {
#pragma unroll
      for (int ts = 0; ts < NSUB; ++ts)
#pragma unroll
        for (int hh = 0; hh < 2; ++hh) {
          float f[8];
          load8<VecU>(urow[ts], w + 8 * hh, p.W, f);
          bf16x8_t parts[3];
          split_parts<3>(f, parts);
#pragma unroll
          for (int rt = 0; rt < RT; ++rt)
#pragma unroll
            for (int q = 0; q < 3; ++q) acc[rt][ts] = mfma16x16x32(vf[rt][hh], parts[q], acc[rt][ts]);
        }
    } else {
      bf16x8_t uf[NSUB][2];
#pragma unroll
      for (int ts = 0; ts < NSUB; ++ts)
#pragma unroll
        for (int hh = 0; hh < 2; ++hh) uf[ts][hh] = load8<VecU>(urow[ts], w + 8 * hh, p.W);
#pragma unroll
      for (int hh = 0; hh < 2; ++hh)
#pragma unroll
        for (int ts = 0; ts < NSUB; ++ts)
#pragma unroll
          for (int rt = 0; rt < RT; ++rt) acc[rt][ts] = mfma16x16x32(vf[rt][hh], uf[ts][hh], acc[rt][ts]);
    }
  }
  // the waves' sums, in order; lane (g, c) holds ranks 16 rt + 4 g .. + 3 of row 16 ts + c
  for (int w = 0; w < kWaves; ++w) {
    if (wave == w) {
#pragma unroll
      for (int rt = 0; rt < RT; ++rt)
#pragma unroll
        for (int ts = 0; ts < NSUB; ++ts) {
          f32x4_t* at = (f32x4_t*)(red + (ts * kSub + c) * kRed + rt * 16 + 4 * g);
          *at = w == 0 ? acc[rt][ts] : *at + acc[rt][ts];
        }
    }
    __syncthreads();
  }
}

template <typename TU, int RT, bool VecU>
__global__ __launch_bounds__(kThreads) void lora_down_kernel(DownArgs p) {
  constexpr int kRed = RT * 16 + 4;
  __shared__ int rows[kLoraTile];
  __shared__ int count;
  __shared__ __align__(16) float red[kLoraTile * kRed];
  const int tile = blockIdx.x;
  if (tile * kLoraTile >= *p.npp) return;
  const int n = load_tile_rows(p.sorted, tile, p.M, rows, &count);
  const int adapter = p.block_adapter[tile];
  if (n <= 16) down_tile<TU, RT, VecU, 1>(p, rows, adapter, red);
  else if (n <= 32) down_tile<TU, RT, VecU, 2>(p, rows, adapter, red);
  else down_tile<TU, RT, VecU, 4>(p, rows, adapter, red);
  const int quads = p.r / 4;
  for (int i = threadIdx.x; i < n * quads; i += kThreads) {
    const int t = i / quads, j = (i % quads) * 4;
    *(float4*)(p.part + ((int64_t)blockIdx.y * p.M + rows[t]) * p.r + j) = *(const float4*)(red + t * kRed + j);
  }
}

// ------------------------------------------------------------------ up
struct UpArgs {
  const float* part;          // [splits][M][r]
  int splits, M, r, N, L;
  const int32_t* ids;         // [M]
  const int32_t* sorted;
  const int32_t* block_adapter;
  const int32_t* npp;
  int tiles;                  // grouping tiles; workgroups past them copy rows without an adapter
  const float* scales;        // [L] or null
  const uint16_t* b;          // [L][N][r]
  const void* base;           // [M, N] or null
  int64_t ld_base;
  void* out;                  // [M, N]
  int64_t ld_out;
  float* h;                   // [M, r] or null: receives the sums of the parts
  int n_block;                // columns per workgroup, a multiple of 256
};

template <typename TO, bool Vec>
__device__ __forceinline__ void load_base(const TO* base, int n, int N, float (&v)[16]) {
  if constexpr (std::is_same<TO, float>::value) {
#pragma unroll
    for (int i = 0; i < 16; i += 4) {
      if constexpr (Vec) {
        if (n + i < N) {
          const float4 x = *(const float4*)(base + n + i);
          v[i] = x.x; v[i + 1] = x.y; v[i + 2] = x.z; v[i + 3] = x.w;
        }
      } else {
#pragma unroll
        for (int q = i; q < i + 4; ++q)
          if (n + q < N) v[q] = base[n + q];
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < 16; i += 8) {
      if constexpr (Vec) {
        if (n + i < N) {
          const uint4 x = *(const uint4*)(base + n + i);
          const uint32_t d[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            v[i + 2 * q] = __uint_as_float(d[q] << 16);
            v[i + 2 * q + 1] = __uint_as_float(d[q] & 0xffff0000u);
          }
        }
      } else {
#pragma unroll
        for (int q = i; q < i + 8; ++q)
          if (n + q < N) v[q] = bf16_value(base[n + q]);
      }
    }
  }
}
template <typename TO, bool Vec>
__device__ __forceinline__ void store_out(TO* out, int n, int N, const float (&v)[16]) {
  if constexpr (std::is_same<TO, float>::value) {
#pragma unroll
    for (int i = 0; i < 16; i += 4) {
      if constexpr (Vec) {
        if (n + i < N) *(float4*)(out + n + i) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
      } else {
#pragma unroll
        for (int q = i; q < i + 4; ++q)
          if (n + q < N) out[n + q] = v[q];
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < 16; i += 8) {
      if constexpr (Vec) {
        uint32_t d[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) d[q] = bf16_bits(v[i + 2 * q]) | bf16_bits(v[i + 2 * q + 1]) << 16;
        if (n + i < N) *(uint4*)(out + n + i) = make_uint4(d[0], d[1], d[2], d[3]);
      } else {
#pragma unroll
        for (int q = i; q < i + 8; ++q)
          if (n + q < N) out[n + q] = (uint16_t)bf16_bits(v[q]);
      }
    }
  }
}

// Rows without an adapter: out = base (nothing to do in place), or zeros; h = 0.
template <typename TO>
__device__ void copy_rows(const UpArgs& p) {
  const int t0 = (blockIdx.x - p.tiles) * kLoraTile;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int n0 = blockIdx.y * p.n_block;
  const int n1 = n0 + p.n_block < p.N ? n0 + p.n_block : p.N;
  const bool in_place = p.base == p.out;
  for (int i = wave; i < kLoraTile && t0 + i < p.M; i += kWaves) {
    const int row = t0 + i;
    const int a = p.ids[row];
    if (a >= 0 && a < p.L) continue;
    if (!in_place) {
      TO* out = (TO*)p.out + (int64_t)row * p.ld_out;
      const TO* base = p.base ? (const TO*)p.base + (int64_t)row * p.ld_base : nullptr;
      for (int n = n0 + lane; n < n1; n += 64) out[n] = base ? base[n] : TO(0);
    }
    if (p.h && blockIdx.y == 0)
      for (int j = lane; j < p.r; j += 64) p.h[(int64_t)row * p.r + j] = 0.0f;
  }
}

// out[row][n] = base[row][n] + sum_j b[n][j] * (scale * h[row][j]).
// The factor's bf16 parts are laid one after another along the contraction:
// 8-wide chunk number q of a lane's fragments is chunk q % (r / 8) of part
// q / (r / 8), so ranks 8 and 16 fill one 32-wide matrix-core step with their
// parts. A wave's group is 64 columns: matrix-core tile i takes columns 4 m + i
// (m its row), so that a lane ends with 16 consecutive columns of one row.
template <typename TO, int RC, bool Vec>
__global__ __launch_bounds__(kThreads) void lora_up_kernel(UpArgs p) {
  constexpr int NP = std::is_same<TO, float>::value ? 3 : 2;
  constexpr int kChunks = RC / 8;                       // 8-wide chunks of a part
  constexpr int kSteps = (NP * kChunks + 3) / 4;        // 32-wide steps
  constexpr int kFrags = kChunks >= 4 ? kChunks / 4 : 1;  // different steps of b
  constexpr int kPitch = RC + 8;                        // elements, 16-byte multiple
  __shared__ int rows[kLoraTile];
  __shared__ int count;
  __shared__ __align__(16) uint16_t parts[NP][kLoraTile][kPitch];
  if ((int)blockIdx.x >= p.tiles) {
    copy_rows<TO>(p);
    return;
  }
  const int tile = blockIdx.x;
  if (tile * kLoraTile >= *p.npp) return;
  const int n = load_tile_rows(p.sorted, tile, p.M, rows, &count);
  const int adapter = p.block_adapter[tile];
  const int nsub = (n + kSub - 1) / kSub;
  const float scale = p.scales ? p.scales[adapter] : 1.0f;
  for (int i = threadIdx.x; i < nsub * kSub * (RC / 4); i += kThreads) {
    const int t = i / (RC / 4), j = (i % (RC / 4)) * 4;
    float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (t < n && j < p.r) {
      const float* at = p.part + (int64_t)rows[t] * p.r + j;
      for (int s = 0; s < p.splits; ++s) {
        const float4 x = *(const float4*)(at + (int64_t)s * p.M * p.r);
        v.x += x.x; v.y += x.y; v.z += x.z; v.w += x.w;
      }
      if (p.h && blockIdx.y == 0) *(float4*)(p.h + (int64_t)rows[t] * p.r + j) = v;
    }
    float f[4] = {v.x * scale, v.y * scale, v.z * scale, v.w * scale};
#pragma unroll
    for (int q = 0; q < NP; ++q) {
      uint32_t bits[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        bits[e] = bf16_bits(f[e]);
        f[e] -= bf16_value(bits[e]);
      }
      *(uint2*)&parts[q][t][j] = make_uint2(bits[0] | bits[1] << 16, bits[2] | bits[3] << 16);
    }
  }
  __syncthreads();

  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, c = lane & 15, g = lane >> 4;
  const uint16_t* b = p.b + (int64_t)adapter * p.N * p.r;
  const int n_end = (int)(blockIdx.y + 1) * p.n_block < p.N ? (int)(blockIdx.y + 1) * p.n_block : p.N;
  for (int n0 = blockIdx.y * p.n_block + wave * 64; n0 < n_end; n0 += kWaves * 64) {
    bf16x8_t bf[4][kFrags];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int col = n0 + 4 * c + i < p.N ? n0 + 4 * c + i : p.N - 1;
#pragma unroll
      for (int k = 0; k < kFrags; ++k) bf[i][k] = load8<true>(b + (int64_t)col * p.r, ((k * 4 + g) % kChunks) * 8, p.r);
    }
#pragma unroll
    for (int ts = 0; ts < 4; ++ts) {
      if (ts >= nsub) break;
      f32x4_t acc[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[i] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int k = 0; k < kSteps; ++k) {
        const int chunk = k * 4 + g;
        const int q = chunk / kChunks;
        bf16x8_t hf = as_bf16x8(*(const uint4*)&parts[q < NP ? q : 0][ts * kSub + c][(chunk % kChunks) * 8]);
        if (kSteps * 4 > NP * kChunks && q >= NP) hf = as_bf16x8(make_uint4(0, 0, 0, 0));
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[i] = mfma16x16x32(bf[i][k % kFrags], hf, acc[i]);
      }
      const int t = ts * kSub + c;
      if (t < n) {
        const int col = n0 + 16 * g;
        float v[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) v[e] = 0.0f;
        if (p.base) load_base<TO, Vec>((const TO*)p.base + (int64_t)rows[t] * p.ld_base, col, p.N, v);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int q = 0; q < 4; ++q) v[4 * q + i] += acc[i][q];
        store_out<TO, Vec>((TO*)p.out + (int64_t)rows[t] * p.ld_out, col, p.N, v);
      }
    }
  }
}

// ------------------------------------------------------------------ transpose
// in [L][R][C] -> out [L][C][pitch], columns R .. pitch zero, for the adapters
// that have rows in the batch.
__global__ __launch_bounds__(kThreads) void lora_transpose_kernel(const uint16_t* __restrict__ in, int R, int C,
                                                                  int64_t pitch, const int32_t* __restrict__ offsets,
                                                                  uint16_t* __restrict__ out) {
  __shared__ uint16_t tile[64][66];
  const int l = blockIdx.z;
  if (offsets[l] == offsets[l + 1]) return;
  const int64_t src = (int64_t)l * R * C, dst = (int64_t)l * C * pitch;
  const int c0 = blockIdx.x * 64, r0 = blockIdx.y * 64;
  const int x = threadIdx.x & 63, y = threadIdx.x >> 6;
  for (int i = y; i < 64; i += kWaves)
    tile[i][x] = (r0 + i < R && c0 + x < C) ? in[src + (int64_t)(r0 + i) * C + c0 + x] : (uint16_t)0;
  __syncthreads();
  for (int i = y; i < 64; i += kWaves)
    if (c0 + i < C && r0 + x < pitch) out[dst + (int64_t)(c0 + i) * pitch + r0 + x] = tile[x][i];
}

// ------------------------------------------------------------------ finish
struct FinishArgs {
  const float* part;          // [splits][M][r]
  int splits, M, r;
  const float* h;             // [M][r]
  const float* scales;        // [L] or null
  const int32_t* sorted;
  const int32_t* block_adapter;
  const int32_t* npp;
  int64_t cap;
  float* dh;                  // [M][r]
  uint16_t* dht;              // [3][r][cap]
  uint16_t* ht;               // [3][r][cap]
};

// dh = scale * (sum of its parts), and the three bf16 parts of dh and of
// scale * h at [part][rank][position in the grouping], zeros at the padding.
__global__ __launch_bounds__(kThreads) void lora_finish_kernel(FinishArgs p) {
  __shared__ int rows[kLoraTile];
  __shared__ int count;
  __shared__ float val[kLoraTile][kLoraMaxRank + 1];
  const int tile = blockIdx.x;
  if (tile * kLoraTile >= *p.npp) return;
  const int n = load_tile_rows(p.sorted, tile, p.M, rows, &count);
  const float scale = p.scales ? p.scales[p.block_adapter[tile]] : 1.0f;
  for (int side = 0; side < 2; ++side) {
    for (int i = threadIdx.x; i < kLoraTile * p.r; i += kThreads) {
      const int t = i / p.r, j = i % p.r;
      float v = 0.0f;
      if (t < n) {
        const int64_t at = (int64_t)rows[t] * p.r + j;
        if (side == 0) {
          for (int s = 0; s < p.splits; ++s) v += p.part[(int64_t)s * p.M * p.r + at];
          v *= scale;
          p.dh[at] = v;
        } else {
          v = p.h[at] * scale;
        }
      }
      val[t][j] = v;
    }
    __syncthreads();
    uint16_t* out = side == 0 ? p.dht : p.ht;
    for (int i = threadIdx.x; i < kLoraTile * p.r; i += kThreads) {
      const int t = i & 63, j = i >> 6;
      float v = val[t][j];
#pragma unroll
      for (int q = 0; q < 3; ++q) {
        const uint32_t bits = bf16_bits(v);
        v -= bf16_value(bits);
        out[((int64_t)q * p.r + j) * p.cap + (int64_t)tile * kLoraTile + t] = (uint16_t)bits;
      }
    }
    __syncthreads();
  }
}

// ------------------------------------------------------------------ outer
struct OuterArgs {
  const void* u;              // [M, W]
  int64_t ldu;
  int W, r, M;
  const uint16_t* vt;         // [3][r][cap]
  int64_t cap;
  const int32_t* sorted;
  const int32_t* block_adapter;
  const int32_t* offsets;     // [L + 1]
  const int32_t* npp;
  float* out;                 // [L][r][W], or [L][W][r] (RankMinor)
  float* slots;               // [2 * chunks] of the same shape
  int chunk;                  // positions per workgroup, a multiple of 64
};

// sum over an adapter's rows of u[row][w] * v[row][j], for 128 columns and up
// to 64 ranks a wave. A step takes 32 positions: lane (g, c) loads 8 columns
// from 8 c of its 8 rows and transposes that 8 x 8 block in registers (the
// contraction runs over rows). The positions are cut into chunks whatever the
// adapters' lengths, so the work is even; sums of an adapter within one chunk
// go to the output, those of one that crosses the chunk's start or end to
// slots 2 c or 2 c + 1, which the reduce kernel adds in order.
template <typename TU, int JT, bool VecU, bool RankMinor>
__global__ __launch_bounds__(kThreads) void lora_outer_kernel(OuterArgs p) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, c = lane & 15, g = lane >> 4;
  const int w0 = (blockIdx.x * kWaves + wave) * 128;
  const int j0 = blockIdx.z * 64;
  const int npp = *p.npp;
  const int p0 = blockIdx.y * p.chunk;
  if (w0 >= p.W || p0 >= npp) return;
  const int p1 = p0 + p.chunk < npp ? p0 + p.chunk : npp;
  f32x4_t acc[8][JT];
#pragma unroll
  for (int i = 0; i < 8; ++i)
#pragma unroll
    for (int jt = 0; jt < JT; ++jt) acc[i][jt] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};

  auto flush = [&](int adapter) {
    const int o0 = p.offsets[adapter], o1 = p.offsets[adapter + 1];
    const int64_t size = (int64_t)p.r * p.W;
    float* out = (o0 >= p0 && o1 <= p0 + p.chunk) ? p.out + adapter * size
                                                  : p.slots + (2 * (int64_t)blockIdx.y + (o0 < p0 ? 0 : 1)) * size;
#pragma unroll
    for (int jt = 0; jt < JT; ++jt) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if constexpr (RankMinor) {
          const int w = w0 + 8 * c + i, j = j0 + 16 * jt + 4 * g;
          if (w < p.W && j < p.r) *(f32x4_t*)(out + (int64_t)w * p.r + j) = acc[i][jt];
        } else {
          const int j = j0 + 16 * jt + c;
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const int w = w0 + 32 * g + 8 * q + i;
            if (w < p.W && j < p.r) out[(int64_t)j * p.W + w] = acc[i][jt][q];
          }
        }
        acc[i][jt] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
      }
    }
  };

  int adapter = p.block_adapter[p0 / kLoraTile];
  for (int pos = p0; pos < p1; pos += 32) {
    const int a = p.block_adapter[pos / kLoraTile];
    if (a != adapter) {
      flush(adapter);
      adapter = a;
    }
    const int4 ra = *(const int4*)(p.sorted + pos + 8 * g), rb = *(const int4*)(p.sorted + pos + 8 * g + 4);
    const int rows[8] = {ra.x, ra.y, ra.z, ra.w, rb.x, rb.y, rb.z, rb.w};
    bf16x8_t vf[JT][3];
#pragma unroll
    for (int jt = 0; jt < JT; ++jt) {
      const int j = j0 + 16 * jt + c < p.r ? j0 + 16 * jt + c : p.r - 1;
#pragma unroll
      for (int q = 0; q < 3; ++q)
        vf[jt][q] = as_bf16x8(*(const uint4*)(p.vt + ((int64_t)q * p.r + j) * p.cap + pos + 8 * g));
    }
    auto mac = [&](int i, bf16x8_t uf, int q) {
#pragma unroll
      for (int jt = 0; jt < JT; ++jt)
        acc[i][jt] = RankMinor ? mfma16x16x32(vf[jt][q], uf, acc[i][jt]) : mfma16x16x32(uf, vf[jt][q], acc[i][jt]);
    };
    if constexpr (std::is_same<TU, float>::value) {
      float f[8][8];
#pragma unroll
      for (int t = 0; t < 8; ++t) {
        load8<VecU>((const float*)p.u + (int64_t)(rows[t] < p.M ? rows[t] : 0) * p.ldu, w0 + 8 * c, p.W, f[t]);
#pragma unroll
        for (int i = 0; i < 8; ++i) f[t][i] = rows[t] < p.M ? f[t][i] : 0.0f;
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float col[8] = {f[0][i], f[1][i], f[2][i], f[3][i], f[4][i], f[5][i], f[6][i], f[7][i]};
        bf16x8_t uf[3];
        split_parts<3>(col, uf);
        mac(i, uf[0], 0);
        mac(i, uf[0], 1);
        mac(i, uf[0], 2);
        mac(i, uf[1], 0);
        mac(i, uf[1], 1);
        mac(i, uf[2], 0);
      }
    } else {
      uint32_t d[8][4];
#pragma unroll
      for (int t = 0; t < 8; ++t) {
        uint4 x = __builtin_bit_cast(
            uint4, load8<VecU>((const uint16_t*)p.u + (int64_t)(rows[t] < p.M ? rows[t] : 0) * p.ldu, w0 + 8 * c, p.W));
        if (rows[t] >= p.M) x = make_uint4(0, 0, 0, 0);
        d[t][0] = x.x; d[t][1] = x.y; d[t][2] = x.z; d[t][3] = x.w;
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        // 16-bit element i of rows 2m and 2m + 1
        const uint32_t sel = (i & 1) ? 0x07060302u : 0x05040100u;
        const bf16x8_t uf = as_bf16x8(make_uint4(__builtin_amdgcn_perm(d[1][i / 2], d[0][i / 2], sel),
                                                 __builtin_amdgcn_perm(d[3][i / 2], d[2][i / 2], sel),
                                                 __builtin_amdgcn_perm(d[5][i / 2], d[4][i / 2], sel),
                                                 __builtin_amdgcn_perm(d[7][i / 2], d[6][i / 2], sel)));
        mac(i, uf, 0);
        mac(i, uf, 1);
        mac(i, uf, 2);
      }
    }
  }
  flush(adapter);
}

// Adapters that cross chunks: their slots, in order; adapters without rows: zeros.
__global__ __launch_bounds__(kThreads) void lora_reduce_kernel(const int32_t* __restrict__ offsets, int64_t size,
                                                               int chunk, const float* __restrict__ slots,
                                                               float* __restrict__ out) {
  const int a = blockIdx.y;
  const int o0 = offsets[a], o1 = offsets[a + 1];
  const int c0 = o0 / chunk, c1 = o1 > o0 ? (o1 - 1) / chunk : c0;
  if (o1 > o0 && c0 == c1) return;
  for (int64_t i = ((int64_t)blockIdx.x * kThreads + threadIdx.x) * 4; i < size;
       i += (int64_t)gridDim.x * kThreads * 4) {
    float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (o1 > o0) {
      v = *(const float4*)(slots + (2 * (int64_t)c0 + 1) * size + i);
      for (int c = c0 + 1; c <= c1; ++c) {
        const float4 x = *(const float4*)(slots + 2 * (int64_t)c * size + i);
        v.x += x.x; v.y += x.y; v.z += x.z; v.w += x.w;
      }
    }
    *(float4*)(out + a * size + i) = v;
  }
}

// ------------------------------------------------------------------ launches
bool vec_ok(const void* p, int64_t ld, bool f32) {
  return !p || ((reinterpret_cast<uintptr_t>(p) & 15) == 0 && ld % (f32 ? 4 : 8) == 0);
}

hipError_t launch_down(const DownArgs& p, bool u_f32, int tiles, int splits, hipStream_t stream) {
  const bool vec = vec_ok(p.u, p.ldu, u_f32) && p.W % (u_f32 ? 4 : 8) == 0;
  const dim3 grid(tiles, splits);
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

hipError_t launch_up(UpArgs p, bool out_f32, hipStream_t stream) {
  const bool vec = vec_ok(p.base, p.ld_base, out_f32) && vec_ok(p.out, p.ld_out, out_f32) &&
                   p.N % (out_f32 ? 4 : 8) == 0;
  const int64_t rows64 = ceil_div(p.M, kLoraTile);
  // several column groups a workgroup once the batch fills the chip without
  int64_t groups = rows64 * ceil_div(p.N, 256) / 1024;
  groups = groups < 1 ? 1 : (groups > 8 ? 8 : groups);
  p.n_block = (int)groups * 256;
  const dim3 grid((unsigned)(p.tiles + rows64), (unsigned)ceil_div(p.N, p.n_block));
  auto go = [&](auto rc) {
    constexpr int RC = decltype(rc)::value;
    if (out_f32) {
      if (vec) lora_up_kernel<float, RC, true><<<grid, kThreads, 0, stream>>>(p);
      else lora_up_kernel<float, RC, false><<<grid, kThreads, 0, stream>>>(p);
    } else {
      if (vec) lora_up_kernel<uint16_t, RC, true><<<grid, kThreads, 0, stream>>>(p);
      else lora_up_kernel<uint16_t, RC, false><<<grid, kThreads, 0, stream>>>(p);
    }
  };
  if (p.r <= 8) go(std::integral_constant<int, 8>{});
  else if (p.r <= 16) go(std::integral_constant<int, 16>{});
  else if (p.r <= 32) go(std::integral_constant<int, 32>{});
  else if (p.r <= 64) go(std::integral_constant<int, 64>{});
  else go(std::integral_constant<int, 128>{});
  return hipGetLastError();
}

template <bool RankMinor>
hipError_t launch_outer(const OuterArgs& p, bool u_f32, int L, hipStream_t stream) {
  const bool vec = vec_ok(p.u, p.ldu, u_f32) && p.W % (u_f32 ? 4 : 8) == 0;
  if (p.M > 0) {
    const dim3 grid((unsigned)ceil_div(p.W, 128 * kWaves), (unsigned)ceil_div(p.cap, p.chunk),
                    (unsigned)ceil_div(p.r, 64));
    auto go = [&](auto jt) {
      constexpr int JT = decltype(jt)::value;
      if constexpr (RankMinor) {  // dB: the output side, either type
        if (u_f32 && vec) lora_outer_kernel<float, JT, true, true><<<grid, kThreads, 0, stream>>>(p);
        else if (u_f32) lora_outer_kernel<float, JT, false, true><<<grid, kThreads, 0, stream>>>(p);
        else if (vec) lora_outer_kernel<uint16_t, JT, true, true><<<grid, kThreads, 0, stream>>>(p);
        else lora_outer_kernel<uint16_t, JT, false, true><<<grid, kThreads, 0, stream>>>(p);
      } else {  // dA: x, bf16 with aligned rows
        lora_outer_kernel<uint16_t, JT, true, false><<<grid, kThreads, 0, stream>>>(p);
      }
    };
    if (p.r <= 16) go(std::integral_constant<int, 1>{});
    else if (p.r <= 32) go(std::integral_constant<int, 2>{});
    else go(std::integral_constant<int, 4>{});
    const hipError_t err = hipGetLastError();
    if (err != hipSuccess) return err;
  }
  const int64_t size = (int64_t)p.r * p.W;
  int64_t blocks = ceil_div(size, 4 * kThreads);
  if (blocks > 1024) blocks = 1024;
  lora_reduce_kernel<<<dim3((unsigned)blocks, (unsigned)L), kThreads, 0, stream>>>(p.offsets, size, p.chunk, p.slots,
                                                                                   p.out);
  return hipGetLastError();
}

int64_t align256(int64_t v) { return (v + 255) & ~int64_t(255); }

}  // namespace

LoraLayout lora_layout(int64_t M, int64_t L, int64_t K, int64_t N, int64_t r, bool backward) {
  LoraLayout o{};
  const int64_t touched = M < L ? M : L;
  o.cap = ceil_div(M + touched * (kLoraTile - 1), kLoraTile) * kLoraTile;
  // splits of the contraction: enough workgroups for the chip, each wave at
  // least one 64-column step, and no more than 16 partial sums to add
  const int64_t steps = ceil_div(backward ? N : K, 64);
  const int64_t tiles = ceil_div(M, kLoraTile) + touched / 2;
  int64_t splits = tiles > 0 ? ceil_div(512, tiles) : 1;
  if (splits > ceil_div(steps, kWaves)) splits = ceil_div(steps, kWaves);
  if (splits > 16) splits = 16;
  const int64_t split_steps = ceil_div(steps, splits);
  o.splits = (int)ceil_div(steps, split_steps);
  int64_t at = 0;
  auto take = [&](int64_t bytes) {
    const int64_t off = at;
    at += align256(bytes);
    return off;
  };
  o.sorted_off = take(o.cap * 4);
  o.block_off = take(o.cap / kLoraTile * 4);
  o.offs_off = take((L + 1) * 4);
  o.npp_off = take(4);
  o.part_off = take(o.splits * M * r * 4);
  if (backward) {
    o.n_pad = ceil_div(N, 8) * 8;
    o.at_off = take(L * K * r * 2);
    o.bt_off = take(L * r * o.n_pad * 2);
    o.dh_off = take(M * r * 4);
    o.dht_off = take(3 * r * o.cap * 2);
    o.ht_off = take(3 * r * o.cap * 2);
    // rows per partial gradient: at least 8 r, so that the partial sums are at
    // most a quarter of the rows' bytes, and at most about 2048 waves
    auto chunk = [&](int64_t W) {
      int64_t c = 8 * r;
      const int64_t even = M * ceil_div(W, 128) / 2048;
      c = c > even ? c : even;
      return ceil_div(c, kLoraTile) * kLoraTile;
    };
    o.a_chunk = (int)chunk(K);
    o.b_chunk = (int)chunk(N);
    o.a_slots_off = take(2 * ceil_div(o.cap, o.a_chunk) * r * K * 4);
    o.b_slots_off = take(2 * ceil_div(o.cap, o.b_chunk) * r * N * 4);
  }
  o.total = at;
  return o;
}

hipError_t launch_lora_forward(const LoraArgs& a, hipStream_t stream) {
  const LoraLayout o = lora_layout(a.M, a.L, a.K, a.N, a.r, false);
  int32_t* sorted = (int32_t*)(a.ws + o.sorted_off);
  int32_t* block = (int32_t*)(a.ws + o.block_off);
  int32_t* offsets = (int32_t*)(a.ws + o.offs_off);
  int32_t* npp = (int32_t*)(a.ws + o.npp_off);
  float* part = (float*)(a.ws + o.part_off);
  const int tiles = (int)(o.cap / kLoraTile);
  hipError_t err = launch_align(a.ids, a.M, a.L, kLoraTile, sorted, block, offsets, npp, stream);
  if (err != hipSuccess) return err;
  DownArgs d{};
  d.u = a.x; d.ldu = a.ldx; d.W = a.K;
  d.v = a.a; d.v_stride = (int64_t)a.r * a.K; d.ldv = a.K;
  d.r = a.r; d.M = a.M; d.sorted = sorted; d.block_adapter = block; d.npp = npp; d.part = part;
  d.split_steps = (int)ceil_div(ceil_div(a.K, 64), o.splits);
  err = launch_down(d, false, tiles, o.splits, stream);
  if (err != hipSuccess) return err;
  UpArgs u{};
  u.part = part; u.splits = o.splits; u.M = a.M; u.r = a.r; u.N = a.N; u.L = a.L;
  u.ids = a.ids; u.sorted = sorted; u.block_adapter = block; u.npp = npp; u.tiles = tiles;
  u.scales = a.scales; u.b = a.b; u.base = a.base; u.ld_base = a.ld_base; u.out = a.out; u.ld_out = a.ld_out;
  u.h = a.h;
  return launch_up(u, a.y_f32, stream);
}

hipError_t launch_lora_backward(const LoraArgs& a, hipStream_t stream) {
  const LoraLayout o = lora_layout(a.M, a.L, a.K, a.N, a.r, true);
  int32_t* sorted = (int32_t*)(a.ws + o.sorted_off);
  int32_t* block = (int32_t*)(a.ws + o.block_off);
  int32_t* offsets = (int32_t*)(a.ws + o.offs_off);
  int32_t* npp = (int32_t*)(a.ws + o.npp_off);
  float* part = (float*)(a.ws + o.part_off);
  uint16_t* at = (uint16_t*)(a.ws + o.at_off);
  uint16_t* bt = (uint16_t*)(a.ws + o.bt_off);
  float* dh = (float*)(a.ws + o.dh_off);
  uint16_t* dht = (uint16_t*)(a.ws + o.dht_off);
  uint16_t* ht = (uint16_t*)(a.ws + o.ht_off);
  const int tiles = (int)(o.cap / kLoraTile);
  hipError_t err = launch_align(a.ids, a.M, a.L, kLoraTile, sorted, block, offsets, npp, stream);
  if (err != hipSuccess) return err;
  if (a.M > 0) {
    if (a.dx) {
      lora_transpose_kernel<<<dim3((unsigned)ceil_div(a.K, 64), (unsigned)ceil_div(a.r, 64), a.L), kThreads, 0, stream>>>(
          a.a, a.r, a.K, a.r, offsets, at);
      if ((err = hipGetLastError()) != hipSuccess) return err;
    }
    lora_transpose_kernel<<<dim3((unsigned)ceil_div(a.r, 64), (unsigned)ceil_div(o.n_pad, 64), a.L), kThreads, 0, stream>>>(
        a.b, a.N, a.r, o.n_pad, offsets, bt);
    if ((err = hipGetLastError()) != hipSuccess) return err;
    DownArgs d{};
    d.u = a.dout; d.ldu = a.ld_dout; d.W = a.N;
    d.v = bt; d.v_stride = a.r * o.n_pad; d.ldv = o.n_pad;
    d.r = a.r; d.M = a.M; d.sorted = sorted; d.block_adapter = block; d.npp = npp; d.part = part;
    d.split_steps = (int)ceil_div(ceil_div(a.N, 64), o.splits);
    if ((err = launch_down(d, a.y_f32, tiles, o.splits, stream)) != hipSuccess) return err;
    FinishArgs f{};
    f.part = part; f.splits = o.splits; f.M = a.M; f.r = a.r; f.h = a.h; f.scales = a.scales;
    f.sorted = sorted; f.block_adapter = block; f.npp = npp; f.cap = o.cap; f.dh = dh; f.dht = dht; f.ht = ht;
    lora_finish_kernel<<<tiles, kThreads, 0, stream>>>(f);
    if ((err = hipGetLastError()) != hipSuccess) return err;
    if (a.dx) {
      UpArgs u{};
      u.part = dh; u.splits = 1; u.M = a.M; u.r = a.r; u.N = a.K; u.L = a.L;
      u.ids = a.ids; u.sorted = sorted; u.block_adapter = block; u.npp = npp; u.tiles = tiles;
      u.b = at; u.base = a.dx_base; u.ld_base = a.ld_dx_base; u.out = a.dx; u.ld_out = a.ld_dx;
      if ((err = launch_up(u, false, stream)) != hipSuccess) return err;
    }
  }
  OuterArgs w{};
  w.r = a.r; w.M = a.M; w.cap = o.cap; w.sorted = sorted; w.block_adapter = block; w.offsets = offsets; w.npp = npp;
  w.u = a.x; w.ldu = a.ldx; w.W = a.K; w.vt = dht; w.out = a.da;
  w.slots = (float*)(a.ws + o.a_slots_off); w.chunk = o.a_chunk;
  if ((err = launch_outer<false>(w, false, a.L, stream)) != hipSuccess) return err;
  w.u = a.dout; w.ldu = a.ld_dout; w.W = a.N; w.vt = ht; w.out = a.db;
  w.slots = (float*)(a.ws + o.b_slots_off); w.chunk = o.b_chunk;
  return launch_outer<true>(w, a.y_f32, a.L, stream);
}

}  // namespace moe
