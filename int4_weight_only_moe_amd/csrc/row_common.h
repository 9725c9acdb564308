// A row of values (the logits of a token) in the registers of 16 or 32 lanes:
// sums and maxima over the row and loading, shared by the balance loss and the
// routing by scores; and the balance loss's exponentials (the routing keeps the
// logits and has a form of its own, RowSoftmax).
#pragma once

#include "route_common.h"

namespace moe {

// Sum and maximum over the lanes of a row (every lane gets them).
template <int Lanes>
__device__ __forceinline__ float row_sum(float v) {
  v += __uint_as_float(dpp<kQuadSwap1>(__float_as_uint(v)));
  v += __uint_as_float(dpp<kQuadSwap2>(__float_as_uint(v)));
  v += __uint_as_float(dpp<kRowHalfMirror>(__float_as_uint(v)));
  v += __uint_as_float(dpp<kRowMirror>(__float_as_uint(v)));
  if constexpr (Lanes == 32) {
    const auto h = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = __uint_as_float(h[0]) + __uint_as_float(h[1]);
  }
  return v;
}
template <int Lanes>
__device__ __forceinline__ float row_max(float v) {
  v = fmaxf(v, __uint_as_float(dpp<kQuadSwap1>(__float_as_uint(v))));
  v = fmaxf(v, __uint_as_float(dpp<kQuadSwap2>(__float_as_uint(v))));
  v = fmaxf(v, __uint_as_float(dpp<kRowHalfMirror>(__float_as_uint(v))));
  v = fmaxf(v, __uint_as_float(dpp<kRowMirror>(__float_as_uint(v))));
  if constexpr (Lanes == 32) {
    const auto h = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = fmaxf(__uint_as_float(h[0]), __uint_as_float(h[1]));
  }
  return v;
}

// Lane l of a row holds the values 4 Lanes j + 4 l + q, q = 0..3, j < NV.
// Vec: rows are 16-byte aligned and E % 4 == 0.
template <int Lanes, int NV, bool Vec>
__device__ __forceinline__ void load_row(const float* __restrict__ row, int E, int l, float (&v)[4 * NV]) {
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int e = 4 * Lanes * j + 4 * l;
    if constexpr (Vec) {
      const float4 x = *(const float4*)(row + (e < E ? e : 0));
      v[4 * j] = e < E ? x.x : -INFINITY;
      v[4 * j + 1] = e < E ? x.y : -INFINITY;
      v[4 * j + 2] = e < E ? x.z : -INFINITY;
      v[4 * j + 3] = e < E ? x.w : -INFINITY;
    } else {
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const float x = row[e + q < E ? e + q : 0];
        v[4 * j + q] = e + q < E ? x : -INFINITY;
      }
    }
  }
}

// Values become exp(v - max) and the result is what makes them probabilities,
// 1 / their sum. A row of nothing but -inf has none: 0. A NaN or +inf gives NaN.
// exp(v - m) = 2^(v log2(e) - m log2(e)) in one fused step: the rounding of
// m log2(e), at most 2^-4 for |m| < 2^20, is the same factor for the whole row
// and goes out with the sum. What stays is the step's own rounding (a difference
// taken first would have the like) and the constant's, |v - m| 2^-26: in fp32 steps
// |v - m| at most. A larger |m| would make the common factor large (it overflows
// from 2^30 on): there the difference is taken first.
template <int Lanes, int N>
__device__ __forceinline__ float exp_row(float (&v)[N]) {
  constexpr float kLog2e = 1.4426950408889634f;
  float m = v[0];
#pragma unroll
  for (int i = 1; i < N; ++i) m = fmaxf(m, v[i]);
  m = row_max<Lanes>(m);
  m = m == -INFINITY ? 0.0f : m;
  const bool far = fabsf(m) >= 0x1p20f;
  if (__any(far)) {
    const float first = far ? m : 0.0f;
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] -= first;
    m = far ? 0.0f : m;
  }
  const float ml = m * kLog2e;
  float s = 0.0f;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    v[i] = __builtin_amdgcn_exp2f(fmaf(v[i], kLog2e, -ml));
    s += v[i];
  }
  s = row_sum<Lanes>(s);
  return s == 0.0f ? 0.0f : 1.0f / s;
}

}  // namespace moe
