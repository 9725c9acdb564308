// Root-mean-square norm with the residual's addition, and its backward pass.
//
//   h = x + residual (rounded to the stream's type), r = 1 / sqrt(mean(h^2) + eps)
//   out = bf16(h r w); out8 = e4m3(h r w / s), s = max |h r w| / 448 of some columns
//   backward, n = h r, u = w g:  dh = dres + r (u - n mean(u n)),  dw = sum_t g n
//
// Both are bound by HBM traffic: a row is read once and stays in registers
// between its sum and its outputs. Rows of up to 1024 columns take one wave,
// wider ones a workgroup; a lane holds 1, 2 or (from 16385 columns on) 4 chunks
// of 8 columns. Outputs go through the cache, where what reads them next finds
// them: with non-temporal stores [4096, 4096] took 20 us instead of 25, but with a
// reader of both outputs behind it 53 instead of 50.
#include <type_traits>

#include "device_common.h"
#include "operators.h"
#include "route_common.h"

namespace moe {
namespace {

constexpr double kE4m3Max = 448.0;

// Sum over a wave, every lane gets the same bits (wave_sum for fp32).
template <int kCtrl>
__device__ __forceinline__ double add_dpp(double v) {
  const uint64_t u = __builtin_bit_cast(uint64_t, v);
  const uint64_t o = (uint64_t)dpp<kCtrl>((uint32_t)(u >> 32)) << 32 | dpp<kCtrl>((uint32_t)u);
  return v + __builtin_bit_cast(double, o);
}
__device__ __forceinline__ double wave_sum64(double v) {
  v = add_dpp<kQuadSwap1>(v);
  v = add_dpp<kQuadSwap2>(v);
  v = add_dpp<kRowHalfMirror>(v);
  v = add_dpp<kRowMirror>(v);
  {
    const uint64_t u = __builtin_bit_cast(uint64_t, v);
    const auto lo = __builtin_amdgcn_permlane16_swap((uint32_t)u, (uint32_t)u, false, false);
    const auto hi = __builtin_amdgcn_permlane16_swap((uint32_t)(u >> 32), (uint32_t)(u >> 32), false, false);
    v = __builtin_bit_cast(double, (uint64_t)hi[0] << 32 | lo[0]) + __builtin_bit_cast(double, (uint64_t)hi[1] << 32 | lo[1]);
  }
  const uint64_t u = __builtin_bit_cast(uint64_t, v);
  const auto lo = __builtin_amdgcn_permlane32_swap((uint32_t)u, (uint32_t)u, false, false);
  const auto hi = __builtin_amdgcn_permlane32_swap((uint32_t)(u >> 32), (uint32_t)(u >> 32), false, false);
  return __builtin_bit_cast(double, (uint64_t)hi[0] << 32 | lo[0]) + __builtin_bit_cast(double, (uint64_t)hi[1] << 32 | lo[1]);
}

// The lanes that share a row: a wave (4 rows a workgroup), or with Wide all
// waves of the workgroup, which exchange through LDS.
constexpr int kMaxWaves = 16;
template <bool Wide>
struct Team {
  static constexpr int kRows = Wide ? 1 : 4;
  static __device__ __forceinline__ int lanes() { return Wide ? (int)blockDim.x : 64; }
  static __device__ __forceinline__ int lane() { return Wide ? threadIdx.x : threadIdx.x & 63; }
  static __device__ __forceinline__ int row() { return Wide ? 0 : __builtin_amdgcn_readfirstlane(threadIdx.x >> 6); }
  // (two barriers, so that `room` may be used again)
  template <typename T>
  static __device__ __forceinline__ T sum(T v, T* room) {
    if constexpr (sizeof(T) == 8) v = wave_sum64(v);
    else v = wave_sum(v);
    if constexpr (Wide) {
      const int waves = blockDim.x >> 6;
      if ((threadIdx.x & 63) == 0) room[threadIdx.x >> 6] = v;
      __syncthreads();
      v = room[0];
      for (int i = 1; i < waves; ++i) v += room[i];
      __syncthreads();
    }
    return v;
  }
};

// Element q of a lane's chunk i. Vec: chunks of 8 neighbours (16-byte loads);
// else neighbours lie in neighbouring lanes.
template <bool Vec>
__device__ __forceinline__ int column(int i, int q, int lane, int lanes) {
  return Vec ? (i * lanes + lane) * 8 + q : (i * 8 + q) * lanes + lane;
}

__device__ __forceinline__ float from_bf16(uint32_t bits) { return __uint_as_float(bits << 16); }
__device__ __forceinline__ uint16_t to_bf16(float v) { return __builtin_bit_cast(uint16_t, (__bf16)v); }

__device__ __forceinline__ void unpack8(uint4 p, float (&v)[8]) {
  const uint32_t u[4] = {p.x, p.y, p.z, p.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(u[i] << 16);
    v[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ uint4 pack8(const float (&v)[8]) {
  uint32_t u[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) u[i] = (uint32_t)to_bf16(v[2 * i]) | ((uint32_t)to_bf16(v[2 * i + 1]) << 16);
  return make_uint4(u[0], u[1], u[2], u[3]);
}

// `columns` further in a row: the row's address is the same in all lanes, and a
// 32-bit byte offset beside it takes half the registers of whole addresses.
template <typename T>
__device__ __forceinline__ T* beside(T* row, int columns) {
  using Byte = std::conditional_t<std::is_const_v<T>, const char, char>;
  return (T*)((Byte*)row + (uint32_t)(columns * (int)sizeof(T)));
}

// Chunk i of a row of bf16 or fp32 values (columns past N: what column 0
// holds; the caller drops them). Loads are unconditional, so that those of
// all chunks go out together.
template <bool Vec, typename T>
__device__ __forceinline__ void load_chunk(const T* row, int i, int lane, int lanes, int N, float (&v)[8]) {
  if constexpr (Vec) {
    const int c = column<true>(i, 0, lane, lanes);
    const T* p = beside(row, c < N ? c : 0);
    if constexpr (sizeof(T) == 2) {
      unpack8(*(const uint4*)p, v);
    } else {
      const float4 a = ((const float4*)p)[0], b = ((const float4*)p)[1];
      v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
      v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
    }
  } else {
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      const int c = column<false>(i, q, lane, lanes);
      const T x = *beside(row, c < N ? c : 0);
      if constexpr (sizeof(T) == 2) v[q] = from_bf16(x);
      else v[q] = x;
    }
  }
}

template <bool Vec, typename T>
__device__ __forceinline__ void store_chunk(T* row, int i, int lane, int lanes, int N, const float (&v)[8]) {
  if constexpr (Vec) {
    const int c = column<true>(i, 0, lane, lanes);
    if (c >= N) return;
    if constexpr (sizeof(T) == 2) {
      *(uint4*)beside(row, c) = pack8(v);
    } else {
      ((float4*)beside(row, c))[0] = make_float4(v[0], v[1], v[2], v[3]);
      ((float4*)beside(row, c))[1] = make_float4(v[4], v[5], v[6], v[7]);
    }
  } else {
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      const int c = column<false>(i, q, lane, lanes);
      if (c < N) {
        if constexpr (sizeof(T) == 2) *beside(row, c) = to_bf16(v[q]);
        else *beside(row, c) = v[q];
      }
    }
  }
}

// fp64 -> fp32 rounded to odd (towards zero, the last bit set if anything was
// lost): rounding that to e4m3 rounds the fp64 value once.
__device__ __forceinline__ float to_odd(double t) {
  const float f = (float)t;
  uint32_t u = __float_as_uint(f);
  const double back = f;
  u -= fabs(back) > fabs(t);
  u |= back != t;
  return __uint_as_float(u);
}

// Ordered like |v|, NaN the highest.
template <typename F>
using Bits = std::conditional_t<sizeof(F) == 4, uint32_t, unsigned long long>;
template <typename F>
__device__ __forceinline__ Bits<F> magnitude(F v) {
  return __builtin_bit_cast(Bits<F>, v) & (~(Bits<F>)0 >> 1);
}
template <typename B>
__device__ __forceinline__ B larger(B a, B b) { return a > b ? a : b; }

// The largest over `lanes` neighbouring lanes: 4, 8 or 16.
template <int kCtrl>
__device__ __forceinline__ uint32_t larger_dpp(uint32_t m) { return larger(m, dpp<kCtrl>(m)); }
template <int kCtrl>
__device__ __forceinline__ unsigned long long larger_dpp(unsigned long long m) {
  return larger(m, (unsigned long long)dpp<kCtrl>((uint32_t)(m >> 32)) << 32 | dpp<kCtrl>((uint32_t)m));
}
template <typename B>
__device__ __forceinline__ B largest_of(B m, int lanes) {
  m = larger_dpp<kQuadSwap1>(m);
  m = larger_dpp<kQuadSwap2>(m);
  if (lanes > 4) m = larger_dpp<kRowHalfMirror>(m);
  if (lanes > 8) m = larger_dpp<kRowMirror>(m);
  return m;
}

// The largest |h w| of a chunk. F = float: exact for bf16 h and w unless it over-
// or underflows, which fp32_top finds.
template <typename F>
__device__ __forceinline__ Bits<F> top_of(const float (&h)[8], const float (&w)[8]) {
  Bits<F> m = 0;
#pragma unroll
  for (int q = 0; q < 8; ++q) m = larger(m, magnitude((F)h[q] * (F)w[q]));
  return m;
}
__device__ __forceinline__ bool fp32_top(uint32_t m) {
  const float v = __uint_as_float(m);
  return v >= 0x1p-100f && v < 0x1p120f;
}

// e4m3 of h w rr / s, as 4 bytes a word. In fp32 that is off by at most 6
// roundings: where it is nowhere near the middle between two e4m3 values (bits 0 to
// 19 of a normal one) it rounds like the exact value. A wave with another value takes
// fp64 for its whole chunk of 512: with 128 columns a scale 6 of 100 chunks of normal
// values and 21 of those with a hundredth of the columns 20 times as large, with a
// scale a row 8 and 55, nearly all for values below 2^-6.
__device__ __forceinline__ void to_e4m3(const float (&h)[8], const float (&w)[8], double rr, float s, uint32_t (&out)[2]) {
  const float f = (float)rr * __builtin_amdgcn_rcpf(s);
  float y[8];
  bool close = !(f >= 0x1p-100f && f < 0x1p100f && s < 0x1p100f);
#pragma unroll
  for (int q = 0; q < 8; ++q) {
    y[q] = h[q] * w[q] * f;
    const uint32_t u = __float_as_uint(y[q]);
    close |= ((u & 0xFFFFFu) - (0x80000u - 16u) <= 32u) | !(fabsf(y[q]) >= 0x1p-6f && fabsf(y[q]) < 449.0f);
  }
  if (__any(close)) {
    const double f64 = rr / (double)s;
#pragma unroll
    for (int q = 0; q < 8; ++q) y[q] = to_odd((double)h[q] * (double)w[q] * f64);
  }
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int u = __builtin_amdgcn_cvt_pk_fp8_f32(y[4 * k], y[4 * k + 1], 0, false);
    out[k] = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(y[4 * k + 2], y[4 * k + 3], u, true);
  }
}

// One row a team. Profiled: [16384, 7168] bf16 161 us for 940 MB (5.8 TB/s; a copy of
// as much takes 181), [2048, 7168] of an fp32 stream with bf16 and 8-bit results of
// 128 columns a scale 45 us for 191 MB (4.3 TB/s; back to back in a graph, from the
// cache, 35.8, and 39 with a scale a row): there 46 vector instructions a column of a lane, 17 us of issue,
// run beside the loads of only two workgroups a CU (93 registers).
template <bool Wide, int C, bool Vec, typename S, bool Quant>
__global__ __launch_bounds__(Wide ? 64 * kMaxWaves : 256) void norm_kernel(NormArgs a) {
  using T = Team<Wide>;
  __shared__ double room[kMaxWaves];
  extern __shared__ unsigned long long maxima[];  // Quant without Vec: of the rows' groups
  const int lane = T::lane(), lanes = T::lanes(), N = a.N;
  const int64_t at = (int64_t)blockIdx.x * T::kRows + T::row();
  const bool active = at < a.M;
  const int64_t t = active ? at : a.M - 1;
  float h[C][8];
  const S* res = (const S*)a.res;
  if (a.x && a.res) {
    float y[C][8];
#pragma unroll
    for (int i = 0; i < C; ++i) {
      load_chunk<Vec>(a.x + t * a.ldx, i, lane, lanes, N, h[i]);
      load_chunk<Vec>(res + t * a.ld_res, i, lane, lanes, N, y[i]);
    }
#pragma unroll
    for (int i = 0; i < C; ++i)
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        h[i][q] += y[i][q];
        if constexpr (sizeof(S) == 2) h[i][q] = from_bf16(to_bf16(h[i][q]));
      }
  } else if (a.x) {
#pragma unroll
    for (int i = 0; i < C; ++i) load_chunk<Vec>(a.x + t * a.ldx, i, lane, lanes, N, h[i]);
  } else {
#pragma unroll
    for (int i = 0; i < C; ++i) load_chunk<Vec>(res + t * a.ld_res, i, lane, lanes, N, h[i]);
  }
  double ss = 0.0;
#pragma unroll
  for (int i = 0; i < C; ++i)
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      if (column<Vec>(i, Vec ? 0 : q, lane, lanes) >= N) h[i][q] = 0.0f;  // (Vec: N % 8 == 0)
      ss = fma((double)h[i][q], (double)h[i][q], ss);
    }
  if (a.res_out && active) {
#pragma unroll
    for (int i = 0; i < C; ++i) store_chunk<Vec>((S*)a.res_out + t * a.ld_res_out, i, lane, lanes, N, h[i]);
  }
  ss = T::sum(ss, room);
  const double rr = 1.0 / sqrt(ss / N + a.eps);
  const float r = (float)rr;
  if (a.out && active) {
#pragma unroll
    for (int i = 0; i < C; ++i) {
      float y[8];
      load_chunk<Vec>(a.w, i, lane, lanes, N, y);
#pragma unroll
      for (int q = 0; q < 8; ++q) y[q] *= h[i][q] * r;
      store_chunk<Vec>(a.out + t * a.ld_out, i, lane, lanes, N, y);
    }
  }
  if (a.rstd && active && lane == 0) a.rstd[t] = r;
  if constexpr (Quant) {
    const int group = a.group, groups = N / group;
    auto weights = [&](int i, float (&w)[8]) { load_chunk<Vec>(a.w, i, lane, lanes, N, w); };
    const double unit = rr / kE4m3Max;
    auto scale_of = [&](double top) {
      const float s = (float)(top * unit);
      return s < 0x1p-126f ? 0x1p-126f : s;
    };
    auto value_of = [](unsigned long long m) { return __builtin_bit_cast(double, m); };
    uint8_t* row8 = a.out8 + t * a.ld_out8;
    float one = 0.0f;  // the row's scale
    if (group == N) {
      unsigned long long all = 0;
#pragma unroll
      for (int i = 0; i < C; ++i) {
        float w[8];
        weights(i, w);
        all = larger(all, top_of<double>(h[i], w));
      }
#pragma unroll
      for (int d = 32; d; d >>= 1) all = larger(all, __shfl_xor(all, d, 64));
      if constexpr (Wide) {
        const int waves = blockDim.x >> 6;
        unsigned long long* tops = (unsigned long long*)room;
        if ((threadIdx.x & 63) == 0) tops[threadIdx.x >> 6] = all;
        __syncthreads();
        for (int i = 0; i < waves; ++i) all = larger(all, tops[i]);
      }
      one = scale_of(value_of(all));
      if (active && lane == 0) a.scales[t] = one;
    }
    if constexpr (Vec) {
#pragma unroll
      for (int i = 0; i < C; ++i) {
        float w[8], s = one;
        weights(i, w);
        const int c = column<true>(i, 0, lane, lanes);
        if (group < N) {  // group / 8 neighbouring lanes
          double top;
          bool small = false;
          if constexpr (sizeof(S) == 2) {
            uint32_t m = top_of<float>(h[i], w);
            m = largest_of(m, group / 8);
            small = __all(fp32_top(m) || c >= N);
            top = __uint_as_float(m);
          }
          if (!small) {
            top = value_of(largest_of(top_of<double>(h[i], w), group / 8));
          }
          s = scale_of(top);
          if (active && c < N && c % group == 0) a.scales[t * groups + c / group] = s;
        }
        uint32_t p[2];
        to_e4m3(h[i], w, rr, s, p);
        if (active && c < N) *(uint2*)(row8 + c) = make_uint2(p[0], p[1]);
      }
    } else {
      unsigned long long* mine = maxima + T::row() * groups;
      if (group < N) {
        for (int g = lane; g < groups; g += lanes) mine[g] = 0;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < C; ++i) {
          float w[8];
          weights(i, w);
#pragma unroll
          for (int q = 0; q < 8; ++q) {
            const int c = column<false>(i, q, lane, lanes);
            if (c < N) atomicMax(mine + c / group, magnitude((double)h[i][q] * (double)w[q]));
          }
        }
        __syncthreads();
        for (int g = lane; g < groups && active; g += lanes) a.scales[t * groups + g] = scale_of(value_of(mine[g]));
      }
#pragma unroll
      for (int i = 0; i < C; ++i) {
        float w[8];
        weights(i, w);
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          const int c = column<false>(i, q, lane, lanes);
          const float s = group == N ? one : scale_of(value_of(mine[c < N ? c / group : 0]));
          const float y = to_odd((double)h[i][q] * (double)w[q] * (rr / (double)s));
          if (active && c < N) row8[c] = (uint8_t)__builtin_amdgcn_cvt_pk_fp8_f32(y, y, 0, false);
        }
      }
    }
  }
}

// ---- backward ---------------------------------------------------------------

// A chunk as it was loaded: 16 or 32 bytes of neighbours, else 8 values.
template <bool Vec, typename T>
struct Raw {
  std::conditional_t<Vec, uint4, float> v[Vec ? (sizeof(T) == 2 ? 1 : 2) : 8];
  __device__ __forceinline__ void load(const T* row, int i, int lane, int lanes, int N) {
    if constexpr (Vec) {
      const int c = column<true>(i, 0, lane, lanes);
      const uint4* p = (const uint4*)beside(row, c < N ? c : 0);
      v[0] = p[0];
      if constexpr (sizeof(T) == 4) v[1] = p[1];
    } else {
      load_chunk<false>(row, i, lane, lanes, N, v);
    }
  }
  // What follows does not see that it is the value from before: else the compiler
  // keeps the unpacked values in twice the registers.
  __device__ __forceinline__ void forget() {
    if constexpr (Vec) {
#pragma unroll
      for (auto& x : v) asm volatile("" : "+v"(x.x), "+v"(x.y), "+v"(x.z), "+v"(x.w));
    }
  }
  __device__ __forceinline__ void values(float (&o)[8]) const {
    if constexpr (!Vec) {
#pragma unroll
      for (int q = 0; q < 8; ++q) o[q] = v[q];
    } else if constexpr (sizeof(T) == 2) {
      unpack8(v[0], o);
    } else {
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        o[4 * q] = __uint_as_float(v[q].x);
        o[4 * q + 1] = __uint_as_float(v[q].y);
        o[4 * q + 2] = __uint_as_float(v[q].z);
        o[4 * q + 3] = __uint_as_float(v[q].w);
      }
    }
  }
};

// The rows of a team's turn, one in flight while another is computed where the
// registers allow it (16-byte chunks of bf16, at most 2 a lane).
template <int C, bool Vec, typename S>
struct BackwardRow {
  Raw<Vec, uint16_t> g[C];
  Raw<Vec, S> h[C], d[C];
  float r;
  __device__ __forceinline__ void load(const NormBackwardArgs& a, int64_t t, int lane, int lanes) {
#pragma unroll
    for (int i = 0; i < C; ++i) {
      g[i].load(a.dout + t * a.ld_dout, i, lane, lanes, a.N);
      h[i].load((const S*)a.h + t * a.ld_h, i, lane, lanes, a.N);
      if (C <= 2 && a.dres) d[i].load((const S*)a.dres + t * a.ld_dres, i, lane, lanes, a.N);
    }
    r = a.rstd[t];
  }
};

// Rows that a lane adds for dw in fp32 one after another: at most so many roundings
// of 2^-24, however many rows there are. (Equal rows lost 6e-5 of a sum of 4096.)
constexpr int kRunRows = 64;
constexpr int kRunsMaxWidth = 16384;  // 128 KB of fp64 sums

// A workgroup takes the rows kRows (blockIdx.x + n gridDim.x) + 0 .. kRows - 1
// and leaves their sums for dw in parts[blockIdx.x]: they stay in registers over
// all its rows. [16384, 7168] bf16: 175 us profiled for 947 MB (5.4 TB/s).
// Runs: more than kRunRows rows a lane. After each run of so many the sums are added
// to fp64 ones in LDS, where each lane has places of its own. Back to back calls of
// [131072, 7168] bf16: 1402 us (1399 with one fp32 sum over all rows; 1436 with the
// fp64 sums in HBM, whose loads nothing hides; 1459 with the run's end tested in the
// loop over rows, which then waits for the row in flight).
template <bool Wide, int C, bool Vec, typename S, bool Runs>
__global__ __launch_bounds__(Wide ? 64 * kMaxWaves : 256) void norm_backward_kernel(NormBackwardArgs a) {
  using T = Team<Wide>;
  constexpr bool kAhead = Vec && C <= 2 && sizeof(S) == 2;
  __shared__ float room[kMaxWaves];
  extern __shared__ __align__(16) float sums[];  // not Wide: [kRows][N]; before that with Runs [kRows][8 C lanes] in fp64
  const int lane = T::lane(), lanes = T::lanes(), N = a.N;
  double* whole = (double*)sums + T::row() * (8 * C * lanes) + lane;  // of this lane, `lanes` apart
  bool any = false;  // whether there are sums in `whole`
  const int64_t step = (int64_t)gridDim.x * T::kRows;
  float acc[C][8];
#pragma unroll
  for (int i = 0; i < C; ++i)
#pragma unroll
    for (int q = 0; q < 8; ++q) acc[i][q] = 0.0f;
  Raw<Vec, uint16_t> w[C];
#pragma unroll
  for (int i = 0; i < C; ++i)
    if (C <= 2) w[i].load(a.w, i, lane, lanes, N);
  const float inv_n = 1.0f / (float)N;
  int64_t t = (int64_t)blockIdx.x * T::kRows + T::row();
  BackwardRow<C, Vec, S> next;
  if (kAhead && t < a.M) next.load(a, t, lane, lanes);
  for (;;) {
    const int64_t stop = Runs && t + kRunRows * step < a.M ? t + kRunRows * step : a.M;
    for (; t < stop; t += step) {
      BackwardRow<C, Vec, S> row;
      if constexpr (kAhead) {
        row = next;
        next.load(a, t + step < a.M ? t + step : t, lane, lanes);
      } else {
        row.load(a, t, lane, lanes);
      }
      float dot = 0.0f;
#pragma unroll
      for (int i = 0; i < C; ++i) {
        float g[8], n[8], wv[8];
        row.g[i].values(g);
        row.h[i].values(n);
        if (C > 2) w[i].load(a.w, i, lane, lanes, N);
        w[i].values(wv);
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          if (column<Vec>(i, Vec ? 0 : q, lane, lanes) >= N) g[q] = n[q] = 0.0f;  // (Vec: N % 8 == 0)
          n[q] *= row.r;
          acc[i][q] = fmaf(g[q], n[q], acc[i][q]);
          dot = fmaf(g[q] * wv[q], n[q], dot);
          // now, not behind the row's sum: that would keep g and n unpacked over it
          asm volatile("" : "+v"(acc[i][q]));
        }
      }
      dot = T::sum(dot, room) * inv_n;
      if (a.dh) {
#pragma unroll
        for (int i = 0; i < C; ++i) {
          float y[8], n[8], wv[8];
          row.g[i].forget();
          row.h[i].forget();
          w[i].forget();
          row.g[i].values(y);
          row.h[i].values(n);
          if (C > 2) w[i].load(a.w, i, lane, lanes, N);
          w[i].values(wv);
#pragma unroll
          for (int q = 0; q < 8; ++q) y[q] = row.r * (y[q] * wv[q] - n[q] * row.r * dot);
          if (a.dres) {
            float d[8];
            if (C > 2) row.d[i].load((const S*)a.dres + t * a.ld_dres, i, lane, lanes, N);
            row.d[i].values(d);
#pragma unroll
            for (int q = 0; q < 8; ++q) y[q] += d[q];
          }
          store_chunk<Vec>((S*)a.dh + t * a.ld_dh, i, lane, lanes, N, y);
        }
      }
    }
    if (!Runs || t >= a.M) break;
#pragma unroll
    for (int i = 0; i < C; ++i)
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        double& s = whole[(8 * i + q) * lanes];
        s = (any ? s : 0.0) + (double)acc[i][q];
        acc[i][q] = 0.0f;
      }
    any = true;
  }
  if (!a.dw) return;
  if constexpr (Runs) {
#pragma unroll
    for (int i = 0; i < C; ++i)
#pragma unroll
      for (int q = 0; q < 8; ++q)
        if (any) acc[i][q] = (float)(whole[(8 * i + q) * lanes] + (double)acc[i][q]);
    if (!Wide) __syncthreads();  // `sums` take the place of the waves' fp64 ones
  }
  float* part = a.parts + (int64_t)blockIdx.x * N;
  if constexpr (Wide) {
#pragma unroll
    for (int i = 0; i < C; ++i) store_chunk<Vec>(part, i, lane, lanes, N, acc[i]);
  } else {  // the waves' sums, in order
    float* mine = sums + T::row() * N;
#pragma unroll
    for (int i = 0; i < C; ++i) store_chunk<Vec>(mine, i, lane, lanes, N, acc[i]);
    __syncthreads();
    for (int c = threadIdx.x; c < N; c += 256) {
      float s = sums[c];
#pragma unroll
      for (int k = 1; k < T::kRows; ++k) s += sums[k * N + c];
      part[c] = s;
    }
  }
}

// dw = the workgroups' sums, added in order by 16 rows of lanes, in fp64. Bound by
// latency: 5 us for 256 sums of 7168 columns (7 MB).
constexpr int kJoinRows = 16;
__global__ __launch_bounds__(64 * kJoinRows) void norm_join_kernel(const float* parts, int teams, int N, float* dw) {
  __shared__ double sums[kJoinRows][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int c = blockIdx.x * 64 + lane;
  const float* p = parts + (c < N ? c : N - 1);
  double s = 0.0;
  constexpr int kAhead = 16;  // (a sum of 256 workgroups in one turn of loads)
  for (int i = wave; i < teams; i += kJoinRows * kAhead) {
    float v[kAhead];
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      const int k = i + j * kJoinRows;
      v[j] = p[(int64_t)(k < teams ? k : i) * N];
    }
#pragma unroll
    for (int j = 0; j < kAhead; ++j) s += i + j * kJoinRows < teams ? (double)v[j] : 0.0;
  }
  sums[wave][lane] = s;
  __syncthreads();
  if (wave == 0 && c < N) {
    for (int i = 1; i < kJoinRows; ++i) s += sums[i][lane];
    dw[c] = (float)s;
  }
}

// fn(Wide, C, threads) for the row width. 2 chunks a lane: with 1 or 4 of them
// [16384, 7168] bf16 took 182 and 167 us instead of 163. From 1025 columns on the
// waves of a workgroup share a row ([8192, 2048]: 25.9 us, 28.5 with a wave a row).
template <typename F>
void by_width(int N, F fn) {
  using std::integral_constant;
  auto one = [&](auto c) { fn(std::false_type{}, c, 256u); };
  auto all = [&](auto c) { fn(std::true_type{}, c, 64u * (unsigned)ceil_div(N, 512 * decltype(c)::value)); };
  if (N <= 512) one(integral_constant<int, 1>{});
  else if (N <= 1024) one(integral_constant<int, 2>{});
  else if (N <= kRunsMaxWidth) all(integral_constant<int, 2>{});
  else all(integral_constant<int, 4>{});
}

// 16-byte chunks of 8 columns in every row of a matrix of `size`-byte elements
bool chunks_ok(const void* p, int64_t ld, int size) {
  return !p || ((reinterpret_cast<uintptr_t>(p) & (size == 1 ? 7 : 15)) == 0 && ld % 8 == 0);
}

}  // namespace

// Rows of a launch: a grid has fewer than 2^32 threads.
constexpr int kSlabRows = 1 << 21;

static hipError_t launch_norm_slab(const NormArgs& a, hipStream_t stream) {
  const int size = a.f32 ? 4 : 2;
  const bool vec = a.N % 8 == 0 && chunks_ok(a.x, a.ldx, 2) && chunks_ok(a.res, a.ld_res, size) &&
                   chunks_ok(a.res_out, a.ld_res_out, size) && chunks_ok(a.w, 8, 2) && chunks_ok(a.out, a.ld_out, 2) &&
                   chunks_ok(a.out8, a.ld_out8, 1);
  by_width(a.N, [&](auto wide, auto c, unsigned threads) {
    constexpr bool W = decltype(wide)::value;
    constexpr int C = decltype(c)::value;
    const unsigned grid = (unsigned)ceil_div(a.M, Team<W>::kRows);
    auto go = [&](auto v, auto s, auto quant) {
      constexpr bool V = decltype(v)::value, Q = decltype(quant)::value;
      using S = decltype(s);
      const unsigned lds = Q && !V && a.group < a.N ? (unsigned)(a.N / a.group * 8 * Team<W>::kRows) : 0;
      norm_kernel<W, C, V, S, Q><<<grid, threads, lds, stream>>>(a);
    };
    auto typed = [&](auto v, auto quant) { a.f32 ? go(v, float{}, quant) : go(v, uint16_t{}, quant); };
    auto quanted = [&](auto v) { a.out8 ? typed(v, std::true_type{}) : typed(v, std::false_type{}); };
    vec ? quanted(std::true_type{}) : quanted(std::false_type{});
  });
  return hipGetLastError();
}

hipError_t launch_norm(const NormArgs& a, hipStream_t stream) {
  const int64_t size = a.f32 ? 4 : 2;
  for (int64_t first = 0; first < a.M; first += kSlabRows) {
    NormArgs slab = a;
    slab.M = (int)(a.M - first < kSlabRows ? a.M - first : kSlabRows);
    if (a.x) slab.x += first * a.ldx;
    if (a.res) slab.res = (const uint8_t*)a.res + first * a.ld_res * size;
    if (a.res_out) slab.res_out = (uint8_t*)a.res_out + first * a.ld_res_out * size;
    if (a.out) slab.out += first * a.ld_out;
    if (a.out8) {
      slab.out8 += first * a.ld_out8;
      slab.scales += first * (a.N / a.group);
    }
    if (a.rstd) slab.rstd += first;
    const hipError_t err = launch_norm_slab(slab, stream);
    if (err != hipSuccess) return err;
  }
  return hipSuccess;
}

// Workgroups of a backward pass. A CU's one workgroup of wide rows keeps a row
// in flight while it computes another; more of them only leave more sums and
// spread the rows in flight ([16384, 7168] bf16: 173 us with 256, 189 with 512, 196
// with 1024; of 2048 columns 76, 58 and 58).
// Rows too wide for fp64 sums in LDS have a workgroup for every kRunRows of them.
int norm_backward_parts(int64_t M, int64_t N) {
  int64_t most = N > 2048 ? 256 : N > 1024 ? 512 : 1024;
  if (N > kRunsMaxWidth) most *= ceil_div(M, most * kRunRows);
  const int64_t n = N > 1024 ? M : ceil_div(M, 4);
  return (int)(n < 1 ? 1 : n < most ? n : most);
}

hipError_t launch_norm_backward(const NormBackwardArgs& a, hipStream_t stream) {
  const int size = a.f32 ? 4 : 2;
  const int teams = norm_backward_parts(a.M, a.N);
  if (a.M > 0 && (a.dh || a.dw)) {
    hipError_t allowed = hipSuccess;
    const bool vec = a.N % 8 == 0 && chunks_ok(a.dout, a.ld_dout, 2) && chunks_ok(a.h, a.ld_h, size) &&
                     chunks_ok(a.w, 8, 2) && chunks_ok(a.dres, a.ld_dres, size) && chunks_ok(a.dh, a.ld_dh, size);
    by_width(a.N, [&](auto wide, auto c, unsigned threads) {
      constexpr bool W = decltype(wide)::value;
      constexpr int C = decltype(c)::value;
      const int rows = Team<W>::kRows;
      auto go = [&](auto v, auto s) {
        constexpr bool V = decltype(v)::value;
        using S = decltype(s);
        if constexpr (C <= 2) {
          if (a.M > (int64_t)kRunRows * rows * teams) {
            const unsigned lds = 8u * 8 * C * (W ? threads : 64u * rows);
            constexpr auto kernel = norm_backward_kernel<W, C, V, S, true>;
            if (lds > 64 * 1024) {  // (the limit of a kernel that does not ask for more)
              allowed = hipFuncSetAttribute(reinterpret_cast<const void*>(kernel),
                                            hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
              if (allowed != hipSuccess) return;
            }
            kernel<<<teams, threads, lds, stream>>>(a);
            return;
          }
        }
        const unsigned lds = W ? 0u : (unsigned)(rows * a.N * 4);
        norm_backward_kernel<W, C, V, S, false><<<teams, threads, lds, stream>>>(a);
      };
      auto typed = [&](auto v) { a.f32 ? go(v, float{}) : go(v, uint16_t{}); };
      vec ? typed(std::true_type{}) : typed(std::false_type{});
    });
    if (allowed != hipSuccess) return allowed;
    const hipError_t err = hipGetLastError();
    if (err != hipSuccess) return err;
  }
  if (!a.dw) return hipSuccess;
  norm_join_kernel<<<(unsigned)ceil_div(a.N, 64), 64 * kJoinRows, 0, stream>>>(a.parts, a.M > 0 ? teams : 0, a.N, a.dw);
  return hipGetLastError();
}

}  // namespace moe
