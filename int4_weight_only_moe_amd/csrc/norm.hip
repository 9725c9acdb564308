// Root-mean-square norm with the residual's addition, and its backward pass.
//
//   h = x + residual (rounded to the stream's type), r = 1 / sqrt(mean(h^2) + eps)
//   out = bf16(h r w); out8 = e4m3(h r w / s), s = max |h r w| / 448 of some columns
//   backward, n = h r, u = w g:  dh = dres + r (u - n mean(u n)),  dw = sum_t g n
//
// Both are bound by HBM traffic: a row is read once and stays in registers
// between its sum and its outputs. Rows of up to 2048 columns take one wave,
// wider ones a workgroup of 4 or 16 waves; a lane holds up to 4 chunks of 8
// columns.
#include <type_traits>

#include "device_common.h"
#include "operators.h"

namespace moe {
namespace {

constexpr float kE4m3Max = 448.0f;

// Sums over a wave, every lane gets the same bits.
__device__ __forceinline__ double wave_sum64(double v) {
#pragma unroll
  for (int d = 32; d; d >>= 1) v += __shfl_xor(v, d, 64);
  return v;
}
__device__ __forceinline__ float wave_sum32(float v) {
#pragma unroll
  for (int d = 32; d; d >>= 1) v += __shfl_xor(v, d, 64);
  return v;
}

// The lanes that share a row: a wave, or W waves that exchange through LDS.
template <int W>
struct Team {
  static constexpr int kLanes = 64 * W;
  static constexpr int kThreads = W == 1 ? 256 : 64 * W;
  static constexpr int kRows = W == 1 ? 4 : 1;
  static __device__ __forceinline__ int lane() { return threadIdx.x % kLanes; }
  static __device__ __forceinline__ int row() { return threadIdx.x / kLanes; }
  // (two barriers, so that `room` may be used again)
  template <typename T>
  static __device__ __forceinline__ T sum(T v, T* room) {
    if constexpr (sizeof(T) == 8) v = wave_sum64(v);
    else v = wave_sum32(v);
    if constexpr (W > 1) {
      if ((threadIdx.x & 63) == 0) room[threadIdx.x >> 6] = v;
      __syncthreads();
      v = room[0];
#pragma unroll
      for (int i = 1; i < W; ++i) v += room[i];
      __syncthreads();
    }
    return v;
  }
};

// Element q of a lane's chunk i. Vec: chunks of 8 neighbours (16-byte loads);
// else neighbours lie in neighbouring lanes.
template <int Lanes, bool Vec>
__device__ __forceinline__ int column(int i, int q, int lane) {
  return Vec ? (i * Lanes + lane) * 8 + q : (i * 8 + q) * Lanes + lane;
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

// Chunk i of a row of bf16 or fp32 values (columns past N: what column 0
// holds; the caller drops them). Loads are unconditional, so that those of
// all chunks go out together.
template <int Lanes, bool Vec, typename T>
__device__ __forceinline__ void load_chunk(const T* row, int i, int lane, int N, float (&v)[8]) {
  if constexpr (Vec) {
    const int c = column<Lanes, true>(i, 0, lane);
    const T* p = row + (c < N ? c : 0);
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
      const int c = column<Lanes, false>(i, q, lane);
      const T x = row[c < N ? c : 0];
      if constexpr (sizeof(T) == 2) v[q] = from_bf16(x);
      else v[q] = x;
    }
  }
}

template <int Lanes, bool Vec, typename T>
__device__ __forceinline__ void store_chunk(T* row, int i, int lane, int N, const float (&v)[8]) {
  if constexpr (Vec) {
    const int c = column<Lanes, true>(i, 0, lane);
    if (c >= N) return;
    if constexpr (sizeof(T) == 2) {
      *(uint4*)(row + c) = pack8(v);
    } else {
      ((float4*)(row + c))[0] = make_float4(v[0], v[1], v[2], v[3]);
      ((float4*)(row + c))[1] = make_float4(v[4], v[5], v[6], v[7]);
    }
  } else {
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      const int c = column<Lanes, false>(i, q, lane);
      if (c < N) {
        if constexpr (sizeof(T) == 2) row[c] = to_bf16(v[q]);
        else row[c] = v[q];
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

__device__ __forceinline__ uint64_t magnitude(double v) {  // ordered like |v|, NaN the highest
  return (uint64_t)__double_as_longlong(v) & 0x7FFFFFFFFFFFFFFFull;
}
__device__ __forceinline__ uint64_t larger(uint64_t a, uint64_t b) { return a > b ? a : b; }

template <int W, int C, bool Vec, typename S, bool Quant>
__global__ __launch_bounds__(Team<W>::kThreads) void norm_kernel(NormArgs a) {
  using T = Team<W>;
  constexpr int L = T::kLanes;
  __shared__ double room[W];
  extern __shared__ unsigned long long maxima[];  // Quant without Vec: of the rows' groups
  const int lane = T::lane(), N = a.N;
  const int64_t at = (int64_t)blockIdx.x * T::kRows + T::row();
  const bool active = at < a.M;
  const int64_t t = active ? at : a.M - 1;
  float h[C][8];
  const S* res = (const S*)a.res;
  if (a.x && a.res) {
    float y[C][8];
#pragma unroll
    for (int i = 0; i < C; ++i) {
      load_chunk<L, Vec>(a.x + t * a.ldx, i, lane, N, h[i]);
      load_chunk<L, Vec>(res + t * a.ld_res, i, lane, N, y[i]);
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
    for (int i = 0; i < C; ++i) load_chunk<L, Vec>(a.x + t * a.ldx, i, lane, N, h[i]);
  } else {
#pragma unroll
    for (int i = 0; i < C; ++i) load_chunk<L, Vec>(res + t * a.ld_res, i, lane, N, h[i]);
  }
  float w[C][8];
#pragma unroll
  for (int i = 0; i < C; ++i) load_chunk<L, Vec>(a.w, i, lane, N, w[i]);
  double ss = 0.0;
#pragma unroll
  for (int i = 0; i < C; ++i)
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      if (column<L, Vec>(i, q, lane) >= N) h[i][q] = 0.0f;
      ss = fma((double)h[i][q], (double)h[i][q], ss);
    }
  ss = T::sum(ss, room);
  const double rr = 1.0 / sqrt(ss / N + a.eps);
  const float r = (float)rr;
  if (a.res_out && active) {
#pragma unroll
    for (int i = 0; i < C; ++i) store_chunk<L, Vec>((S*)a.res_out + t * a.ld_res_out, i, lane, N, h[i]);
  }
  if (a.out && active) {
#pragma unroll
    for (int i = 0; i < C; ++i) {
      float y[8];
#pragma unroll
      for (int q = 0; q < 8; ++q) y[q] = h[i][q] * r * w[i][q];
      store_chunk<L, Vec>(a.out + t * a.ld_out, i, lane, N, y);
    }
  }
  if (a.rstd && active && lane == 0) a.rstd[t] = r;
  if constexpr (Quant) {
    const int group = a.group, groups = N / group;
    unsigned long long* mine = maxima + T::row() * groups;
    uint64_t top[C], all = 0;
#pragma unroll
    for (int i = 0; i < C; ++i) {
      top[i] = 0;
#pragma unroll
      for (int q = 0; q < 8; ++q) top[i] = larger(top[i], magnitude((double)h[i][q] * (double)w[i][q]));
      all = larger(all, top[i]);
    }
    auto scale_of = [&](uint64_t m) {
      const float s = (float)(__longlong_as_double((long long)m) * rr / kE4m3Max);
      return s < 0x1p-126f ? 0x1p-126f : s;
    };
    float s[C][Vec ? 1 : 8];
    if (Vec && group < N) {  // group / 8 neighbouring lanes
#pragma unroll
      for (int i = 0; i < C; ++i) {
        uint64_t m = top[i];
        for (int d = 1; d < group / 8; d *= 2) m = larger(m, (uint64_t)__shfl_xor((unsigned long long)m, d, 64));
        s[i][0] = scale_of(m);
        const int c = column<L, true>(i, 0, lane);
        if (active && c < N && c % group == 0) a.scales[t * groups + c / group] = s[i][0];
      }
    } else if (group == N) {
#pragma unroll
      for (int d = 32; d; d >>= 1) all = larger(all, (uint64_t)__shfl_xor((unsigned long long)all, d, 64));
      if constexpr (W > 1) {
        if ((threadIdx.x & 63) == 0) room[threadIdx.x >> 6] = __longlong_as_double((long long)all);
        __syncthreads();
#pragma unroll
        for (int i = 0; i < W; ++i) all = larger(all, (uint64_t)__double_as_longlong(room[i]));
      }
      const float one = scale_of(all);
#pragma unroll
      for (int i = 0; i < C; ++i)
#pragma unroll
        for (int q = 0; q < (Vec ? 1 : 8); ++q) s[i][q] = one;
      if (active && lane == 0) a.scales[t] = one;
    } else {
      for (int g = lane; g < groups; g += L) mine[g] = 0;
      __syncthreads();
#pragma unroll
      for (int i = 0; i < C; ++i)
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          const int c = column<L, Vec>(i, q, lane);
          if (c < N) atomicMax(mine + c / group, (unsigned long long)magnitude((double)h[i][q] * (double)w[i][q]));
        }
      __syncthreads();
      for (int g = lane; g < groups && active; g += L) a.scales[t * groups + g] = scale_of(mine[g]);
#pragma unroll
      for (int i = 0; i < C; ++i)
#pragma unroll
        for (int q = 0; q < (Vec ? 1 : 8); ++q) {
          const int c = column<L, Vec>(i, q, lane);
          s[i][q] = scale_of(mine[c < N ? c / group : 0]);
        }
    }
    if (!active) return;
#pragma unroll
    for (int i = 0; i < C; ++i) {
      float y[8];
#pragma unroll
      for (int q = 0; q < 8; ++q)
        y[q] = to_odd((double)h[i][q] * (double)w[i][q] * (rr / (double)s[i][Vec ? 0 : q]));
      uint32_t p[2];
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        int u = __builtin_amdgcn_cvt_pk_fp8_f32(y[4 * k], y[4 * k + 1], 0, false);
        p[k] = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(y[4 * k + 2], y[4 * k + 3], u, true);
      }
      uint8_t* row8 = a.out8 + t * a.ld_out8;
      if constexpr (Vec) {
        const int c = column<L, true>(i, 0, lane);
        if (c < N) *(uint2*)(row8 + c) = make_uint2(p[0], p[1]);
      } else {
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          const int c = column<L, false>(i, q, lane);
          if (c < N) row8[c] = (uint8_t)(p[q / 4] >> (8 * (q % 4)));
        }
      }
    }
  }
}

// ---- backward ---------------------------------------------------------------

// Team i takes the rows i, i + teams, ...; each leaves its sum for dw in parts[i].
template <int W, int C, bool Vec, typename S>
__global__ __launch_bounds__(Team<W>::kThreads) void norm_backward_kernel(NormBackwardArgs a, int teams) {
  using T = Team<W>;
  constexpr int L = T::kLanes;
  __shared__ float room[W];
  const int lane = T::lane(), N = a.N;
  const int team = blockIdx.x * T::kRows + T::row();
  float w[C][8], acc[C][8];
#pragma unroll
  for (int i = 0; i < C; ++i) {
    load_chunk<L, Vec>(a.w, i, lane, N, w[i]);
#pragma unroll
    for (int q = 0; q < 8; ++q) acc[i][q] = 0.0f;
  }
  if (team >= teams) return;  // (a whole wave of a one-wave team)
  const float inv_n = 1.0f / (float)N;
  for (int64_t t = team; t < a.M; t += teams) {
    float g[C][8], n[C][8], d[C][8];
#pragma unroll
    for (int i = 0; i < C; ++i) {
      load_chunk<L, Vec>(a.dout + t * a.ld_dout, i, lane, N, g[i]);
      load_chunk<L, Vec>((const S*)a.h + t * a.ld_h, i, lane, N, n[i]);
      if (a.dres) load_chunk<L, Vec>((const S*)a.dres + t * a.ld_dres, i, lane, N, d[i]);
    }
    const float r = a.rstd[t];
    float dot = 0.0f;
#pragma unroll
    for (int i = 0; i < C; ++i)
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        if (column<L, Vec>(i, q, lane) >= N) g[i][q] = n[i][q] = 0.0f;
        n[i][q] *= r;
        acc[i][q] = fmaf(g[i][q], n[i][q], acc[i][q]);
        g[i][q] *= w[i][q];
        dot = fmaf(g[i][q], n[i][q], dot);
      }
    dot = T::sum(dot, room) * inv_n;
    if (a.dh) {
#pragma unroll
      for (int i = 0; i < C; ++i) {
        float y[8];
#pragma unroll
        for (int q = 0; q < 8; ++q) y[q] = r * (g[i][q] - n[i][q] * dot) + (a.dres ? d[i][q] : 0.0f);
        store_chunk<L, Vec>((S*)a.dh + t * a.ld_dh, i, lane, N, y);
      }
    }
  }
  if (a.dw) {
#pragma unroll
    for (int i = 0; i < C; ++i) store_chunk<L, Vec>(a.parts + (int64_t)team * N, i, lane, N, acc[i]);
  }
}

// dw = the teams' sums, added in order by 16 rows of lanes, in fp64.
constexpr int kJoinRows = 16;
__global__ __launch_bounds__(64 * kJoinRows) void norm_join_kernel(const float* parts, int teams, int N, float* dw) {
  __shared__ double sums[kJoinRows][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int c = blockIdx.x * 64 + lane;
  const float* p = parts + (c < N ? c : N - 1);
  double s = 0.0;
  constexpr int kAhead = 8;
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

// fn(W, C) for the row width
template <typename F>
void by_width(int N, F fn) {
  auto go = [&](auto w, auto c) { fn(w, c); };
  using std::integral_constant;
  if (N <= 512) go(integral_constant<int, 1>{}, integral_constant<int, 1>{});
  else if (N <= 1024) go(integral_constant<int, 1>{}, integral_constant<int, 2>{});
  else if (N <= 2048) go(integral_constant<int, 1>{}, integral_constant<int, 4>{});
  else if (N <= 4096) go(integral_constant<int, 4>{}, integral_constant<int, 2>{});
  else if (N <= 8192) go(integral_constant<int, 4>{}, integral_constant<int, 4>{});
  else if (N <= 16384) go(integral_constant<int, 16>{}, integral_constant<int, 2>{});
  else go(integral_constant<int, 16>{}, integral_constant<int, 4>{});
}

// 16-byte chunks of 8 columns in every row of a matrix of `size`-byte elements
bool chunks_ok(const void* p, int64_t ld, int size) {
  return !p || ((reinterpret_cast<uintptr_t>(p) & (size == 1 ? 7 : 15)) == 0 && ld % 8 == 0);
}

}  // namespace

hipError_t launch_norm(const NormArgs& a, hipStream_t stream) {
  const int size = a.f32 ? 4 : 2;
  const bool vec = a.N % 8 == 0 && chunks_ok(a.x, a.ldx, 2) && chunks_ok(a.res, a.ld_res, size) &&
                   chunks_ok(a.res_out, a.ld_res_out, size) && chunks_ok(a.w, 8, 2) && chunks_ok(a.out, a.ld_out, 2) &&
                   chunks_ok(a.out8, a.ld_out8, 1);
  by_width(a.N, [&](auto w, auto c) {
    constexpr int W = decltype(w)::value, C = decltype(c)::value;
    const unsigned grid = (unsigned)ceil_div(a.M, Team<W>::kRows);
    auto go = [&](auto v, auto s, auto quant) {
      constexpr bool V = decltype(v)::value, Q = decltype(quant)::value;
      using S = decltype(s);
      const unsigned lds = Q && !V && a.group < a.N ? (unsigned)(a.N / a.group * 8 * Team<W>::kRows) : 0;
      norm_kernel<W, C, V, S, Q><<<grid, Team<W>::kThreads, lds, stream>>>(a);
    };
    auto typed = [&](auto v, auto quant) { a.f32 ? go(v, float{}, quant) : go(v, uint16_t{}, quant); };
    auto quanted = [&](auto v) { a.out8 ? typed(v, std::true_type{}) : typed(v, std::false_type{}); };
    vec ? quanted(std::true_type{}) : quanted(std::false_type{});
  });
  return hipGetLastError();
}

// Teams of a backward pass: enough loads in flight for the memory, few enough
// that the sums they leave are small beside the rows.
int norm_backward_parts(int64_t M) { return (int)(M < 512 ? (M < 1 ? 1 : M) : 512); }

hipError_t launch_norm_backward(const NormBackwardArgs& a, hipStream_t stream) {
  const int size = a.f32 ? 4 : 2;
  const int teams = norm_backward_parts(a.M);
  if (a.M > 0 && (a.dh || a.dw)) {
    const bool vec = a.N % 8 == 0 && chunks_ok(a.dout, a.ld_dout, 2) && chunks_ok(a.h, a.ld_h, size) &&
                     chunks_ok(a.w, 8, 2) && chunks_ok(a.dres, a.ld_dres, size) && chunks_ok(a.dh, a.ld_dh, size);
    by_width(a.N, [&](auto w, auto c) {
      constexpr int W = decltype(w)::value, C = decltype(c)::value;
      const unsigned grid = (unsigned)ceil_div(teams, Team<W>::kRows);
      auto go = [&](auto v, auto s) {
        norm_backward_kernel<W, C, decltype(v)::value, decltype(s)><<<grid, Team<W>::kThreads, 0, stream>>>(a, teams);
      };
      auto typed = [&](auto v) { a.f32 ? go(v, float{}) : go(v, uint16_t{}); };
      vec ? typed(std::true_type{}) : typed(std::false_type{});
    });
    const hipError_t err = hipGetLastError();
    if (err != hipSuccess) return err;
  }
  if (!a.dw) return hipSuccess;
  norm_join_kernel<<<(unsigned)ceil_div(a.N, 64), 64 * kJoinRows, 0, stream>>>(a.parts, a.M > 0 ? teams : 0, a.N, a.dw);
  return hipGetLastError();
}

}  // namespace moe
