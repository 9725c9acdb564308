// Balance loss of the router, per-expert counts, and the gradient.
//
// For a sequence s of T valid tokens with logits l[t, :] (p = softmax over the
// E experts) and chosen experts ids[t, 0..k), c[s, e] = how often e was chosen:
//   loss[s] = E / (k T^2) * sum_e c[s, e] * P[s, e],  P[s, e] = sum_t p[t, e]
// (E times the dot product of the chosen share c / (k T) with the mean
// probability P / T: 1 when both are uniform). The counts have no gradient, so
//   d loss[s] / d l[t, e] = E / (k T^2) * p[t, e] * (c[s, e] - sum_j c[s, j] p[t, j]).
//
// Both directions read the logits once and are bound by that memory traffic:
// a row fits into the registers of 16 lanes (E <= 1024: 64 values a lane at
// most), so the softmax needs no second pass and the backward pass recomputes
// p rather than reading a stored copy. 16 lanes a row (not a whole wave) makes
// a row's maximum and sum four register exchanges and lets a wave's load
// instruction cover four rows in 256-byte pieces.
#include <type_traits>

#include "device_common.h"
#include "operators.h"
#include "route_common.h"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kRowLanes = 16;
constexpr int kRowsPerPass = kThreads / kRowLanes;
constexpr int kMaxExperts = 1024;

// Sum and maximum over the 16 lanes of a row (every lane gets them).
__device__ __forceinline__ float row_sum(float v) {
  v += __uint_as_float(dpp<kQuadSwap1>(__float_as_uint(v)));
  v += __uint_as_float(dpp<kQuadSwap2>(__float_as_uint(v)));
  v += __uint_as_float(dpp<kRowHalfMirror>(__float_as_uint(v)));
  v += __uint_as_float(dpp<kRowMirror>(__float_as_uint(v)));
  return v;
}
__device__ __forceinline__ float row_max(float v) {
  v = fmaxf(v, __uint_as_float(dpp<kQuadSwap1>(__float_as_uint(v))));
  v = fmaxf(v, __uint_as_float(dpp<kQuadSwap2>(__float_as_uint(v))));
  v = fmaxf(v, __uint_as_float(dpp<kRowHalfMirror>(__float_as_uint(v))));
  v = fmaxf(v, __uint_as_float(dpp<kRowMirror>(__float_as_uint(v))));
  return v;
}

// Lane l of a row's 16 holds the values 64 j + 4 l + q, q = 0..3, j < NV.
// Vec: rows are 16-byte aligned and E % 4 == 0.
template <int NV, bool Vec>
__device__ __forceinline__ void load_row(const float* __restrict__ row, int E, int lane16, float pad,
                                         float (&v)[4 * NV]) {
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int e = 64 * j + 4 * lane16;
    if constexpr (Vec) {
      const float4 x = *(const float4*)(row + (e < E ? e : 0));
      v[4 * j] = e < E ? x.x : pad;
      v[4 * j + 1] = e < E ? x.y : pad;
      v[4 * j + 2] = e < E ? x.z : pad;
      v[4 * j + 3] = e < E ? x.w : pad;
    } else {
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const float x = row[e + q < E ? e + q : 0];
        v[4 * j + q] = e + q < E ? x : pad;
      }
    }
  }
}

// Values become softmax probabilities. A row of nothing but -inf has none: its
// probabilities are 0. A NaN or +inf gives NaN.
template <int N>
__device__ __forceinline__ void softmax_row(float (&v)[N]) {
  float m = v[0];
#pragma unroll
  for (int i = 1; i < N; ++i) m = fmaxf(m, v[i]);
  m = row_max(m);
  m = m == -INFINITY ? 0.0f : m;
  float s = 0.0f;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    v[i] = expf(v[i] - m);
    s += v[i];
  }
  s = row_sum(s);
  const float inv = s == 0.0f ? 0.0f : 1.0f / s;
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] *= inv;
}

// The last sequence that starts at or before row t (offsets ascending).
__device__ __forceinline__ int sequence_of(const int32_t* __restrict__ off, int S, int t) {
  int lo = 0, hi = S - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (off[mid] <= t) lo = mid; else hi = mid - 1;
  }
  return lo;
}

__device__ __forceinline__ int clamp_row(int v, int M) { return v < 0 ? 0 : (v > M ? M : v); }

// One chunk of rows: for each sequence in it, the chunk's sums of
// probabilities, counts and valid rows, to slot chunk + sequence.
template <int NV, bool Vec>
__global__ __launch_bounds__(kThreads) void balance_rows_kernel(BalanceArgs a, int chunk_rows, float* psums,
                                                                int32_t* pcounts, int32_t* ptokens, int32_t* tickets) {
  __shared__ int cnt[kMaxExperts];
  __shared__ float sums[kThreads / 64][kMaxExperts];
  __shared__ int live_rows;
  const int tid = threadIdx.x, lane16 = tid & 15, group = tid >> 4, wave = tid >> 6;
  const int E = a.E, k = a.k;
  // the finalize kernel's tickets start at zero
  for (int s = blockIdx.x * kThreads + tid; s < a.S; s += gridDim.x * kThreads) tickets[s] = 0;
  const int r0 = blockIdx.x * chunk_rows;
  const int r1 = r0 + chunk_rows < a.M ? r0 + chunk_rows : a.M;
  if (r0 >= r1) return;
  const int s_first = a.offsets ? sequence_of(a.offsets, a.S, r0) : 0;
  for (int s = s_first; s < a.S; ++s) {
    int lo = 0, hi = a.M;
    if (a.offsets) {
      lo = clamp_row(a.offsets[s], a.M);
      hi = clamp_row(a.offsets[s + 1], a.M);
      if (lo >= r1) break;
    }
    lo = lo > r0 ? lo : r0;
    hi = hi < r1 ? hi : r1;
    if (lo >= hi) continue;
    for (int e = tid; e < E; e += kThreads) cnt[e] = 0;
    if (tid == 0) live_rows = 0;
    __syncthreads();
    const int32_t* ids = a.topk_ids + (int64_t)lo * k;
    const unsigned nids = (unsigned)(hi - lo) * (unsigned)k;
    for (unsigned i = tid; i < nids; i += kThreads) {
      const int e = ids[i];
      if (e >= 0 && e < E && (!a.valid || a.valid[lo + i / (unsigned)k])) atomicAdd(&cnt[e], 1);
    }
    float acc[4 * NV];
#pragma unroll
    for (int i = 0; i < 4 * NV; ++i) acc[i] = 0.0f;
    int live = 0;
    for (int t = lo + group; t < hi; t += kRowsPerPass) {
      if (a.valid && !a.valid[t]) continue;
      ++live;
      float v[4 * NV];
      load_row<NV, Vec>(a.logits + (int64_t)t * E, E, lane16, -INFINITY, v);
      softmax_row(v);
#pragma unroll
      for (int i = 0; i < 4 * NV; ++i) acc[i] += v[i];
    }
    if (lane16 == 0 && live) atomicAdd(&live_rows, live);
    // the wave's four rows, then the waves
#pragma unroll
    for (int i = 0; i < 4 * NV; ++i) {
      acc[i] += __shfl_xor(acc[i], 16, 64);
      acc[i] += __shfl_xor(acc[i], 32, 64);
    }
    if ((tid & 63) < 16) {
#pragma unroll
      for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int q = 0; q < 4; ++q)
          if (64 * j + 4 * lane16 + q < E) sums[wave][64 * j + 4 * lane16 + q] = acc[4 * j + q];
    }
    __syncthreads();
    const int64_t slot = (int64_t)blockIdx.x + s;
    for (int e = tid; e < E; e += kThreads) {
      psums[slot * E + e] = (sums[0][e] + sums[1][e]) + (sums[2][e] + sums[3][e]);
      pcounts[slot * E + e] = cnt[e];
    }
    if (tid == 0) ptokens[slot] = live_rows;
    __syncthreads();
  }
}

// Sums a sequence's slots for 64 experts at a time, in a fixed order and in
// fp64, and the loss. With several workgroups a sequence (gridDim.x > 1) each
// leaves its part of the loss, and the last one to finish (the ticket) adds
// the parts in order.
constexpr int kFinThreads = 1024;
__global__ __launch_bounds__(kFinThreads) void balance_finalize_kernel(BalanceArgs a, int chunk_rows,
                                                                       const float* psums, const int32_t* pcounts,
                                                                       const int32_t* ptokens, double* ploss,
                                                                       int32_t* tickets) {
  __shared__ double dsum[16][64];
  __shared__ int dcnt[16][64];
  __shared__ int dtok[16];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int s = blockIdx.y, E = a.E;
  int lo = 0, hi = a.M;
  if (a.offsets) {
    lo = clamp_row(a.offsets[s], a.M);
    hi = clamp_row(a.offsets[s + 1], a.M);
  }
  const int c0 = lo / chunk_rows, c1 = lo < hi ? (hi - 1) / chunk_rows + 1 : c0;
  const int groups = (E + 63) / 64;
  int tok = 0;
  for (int c = c0 + tid; c < c1; c += kFinThreads) tok += ptokens[(int64_t)c + s];
#pragma unroll
  for (int d = 32; d; d >>= 1) tok += __shfl_xor(tok, d, 64);
  if (lane == 0) dtok[wave] = tok;
  __syncthreads();
  tok = 0;
#pragma unroll
  for (int w = 0; w < 16; ++w) tok += dtok[w];
  const double scale = tok ? (double)E / ((double)a.k * (double)tok * (double)tok) : 0.0;
  double loss = 0.0;
  for (int g = blockIdx.x; g < groups; g += gridDim.x) {
    const int e = 64 * g + lane;
    double sum = 0.0;
    int cnt = 0;
    if (e < E) {
      for (int c = c0 + wave; c < c1; c += 16) {
        const int64_t at = ((int64_t)c + s) * E + e;
        sum += (double)psums[at];
        cnt += pcounts[at];
      }
    }
    dsum[wave][lane] = sum;
    dcnt[wave][lane] = cnt;
    __syncthreads();
    if (wave == 0) {
      for (int w = 1; w < 16; ++w) {
        sum += dsum[w][lane];
        cnt += dcnt[w][lane];
      }
      if (e < E) {
        a.prob_sums[(int64_t)s * E + e] = (float)sum;
        a.counts[(int64_t)s * E + e] = cnt;
      }
      double part = sum * (double)cnt;
#pragma unroll
      for (int d = 32; d; d >>= 1) part += __shfl_xor(part, d, 64);
      loss += part;
    }
    __syncthreads();
  }
  if (tid != 0) return;
  if (blockIdx.x == 0) a.tokens[s] = tok;
  if (gridDim.x == 1) {
    a.loss[s] = (float)(loss * scale);
    return;
  }
  double* mine = ploss + (int64_t)s * 16;
  __hip_atomic_store(mine + blockIdx.x, loss, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  __threadfence();
  if (__hip_atomic_fetch_add(tickets + s, 1, __ATOMIC_ACQ_REL, __HIP_MEMORY_SCOPE_AGENT) == (int)gridDim.x - 1) {
    __threadfence();
    loss = 0.0;
    for (int i = 0; i < (int)gridDim.x; ++i)
      loss += __hip_atomic_load(mine + i, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    a.loss[s] = (float)(loss * scale);
  }
}

template <int NV, bool Vec>
__global__ __launch_bounds__(kThreads) void balance_backward_kernel(BalanceArgs a, int chunk_rows) {
  const int lane16 = threadIdx.x & 15, group = threadIdx.x >> 4;
  const int E = a.E;
  const int r0 = blockIdx.x * chunk_rows;
  const int r1 = r0 + chunk_rows < a.M ? r0 + chunk_rows : a.M;
  int lo = 0, hi = 0;  // the sequence whose counts are held
  float c[4 * NV], w = 0.0f;
  for (int t = r0 + group; t < r1; t += kRowsPerPass) {
    if (t >= hi || t < lo) {
      int s = 0;
      lo = 0;
      hi = a.M;
      if (a.offsets) {
        s = sequence_of(a.offsets, a.S, t);
        lo = a.offsets[s];
        hi = a.offsets[s + 1];
        if (t < lo || t >= hi) {  // a row of no sequence
          lo = hi = 0;
          continue;
        }
      }
#pragma unroll
      for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int e = 64 * j + 4 * lane16 + q;
          c[4 * j + q] = e < E ? (float)a.counts[(int64_t)s * E + e] : 0.0f;
        }
      const float T = (float)a.tokens[s];
      w = T > 0.0f ? a.dloss[s] * ((float)E / ((float)a.k * T)) / T : 0.0f;
    }
    float* g = a.grad + (int64_t)t * E;
    float v[4 * NV];
    if (a.valid && !a.valid[t]) {
#pragma unroll
      for (int i = 0; i < 4 * NV; ++i) v[i] = 0.0f;
    } else {
      load_row<NV, Vec>(a.logits + (int64_t)t * E, E, lane16, -INFINITY, v);
      softmax_row(v);
      float dot = 0.0f;
#pragma unroll
      for (int i = 0; i < 4 * NV; ++i) dot = fmaf(c[i], v[i], dot);
      dot = row_sum(dot);
#pragma unroll
      for (int i = 0; i < 4 * NV; ++i) v[i] = w * v[i] * (c[i] - dot);
    }
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int e = 64 * j + 4 * lane16;
      if constexpr (Vec) {
        if (e < E) *(float4*)(g + e) = make_float4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
      } else {
#pragma unroll
        for (int q = 0; q < 4; ++q)
          if (e + q < E) g[e + q] = v[4 * j + q];
      }
    }
  }
}

// fn(NV, Vec) for the row width
template <typename F>
hipError_t by_width(const BalanceArgs& a, F fn) {
  const bool vec = a.E % 4 == 0 && (reinterpret_cast<uintptr_t>(a.logits) & 15) == 0 &&
                   (!a.grad || (reinterpret_cast<uintptr_t>(a.grad) & 15) == 0);
  const int nv = (a.E + 63) / 64;
  auto go = [&](auto n) { vec ? fn(n, std::true_type{}) : fn(n, std::false_type{}); };
  if (nv <= 1) go(std::integral_constant<int, 1>{});
  else if (nv <= 2) go(std::integral_constant<int, 2>{});
  else if (nv <= 4) go(std::integral_constant<int, 4>{});
  else if (nv <= 6) go(std::integral_constant<int, 6>{});
  else if (nv <= 8) go(std::integral_constant<int, 8>{});
  else go(std::integral_constant<int, 16>{});
  return hipGetLastError();
}

}  // namespace

int balance_chunk_rows(int64_t M) {
  // at most 512 chunks of whole passes: enough workgroups to fill the chip,
  // few enough that the partials are small beside the logits
  const int64_t rows = ceil_div(ceil_div(M, 512), kRowsPerPass) * kRowsPerPass;
  return (int)(rows < kRowsPerPass ? kRowsPerPass : rows);
}

static int64_t align256(int64_t v) { return (v + 255) & ~int64_t(255); }

BalanceLayout balance_layout(int64_t M, int64_t E, int64_t S) {
  BalanceLayout L;
  L.chunks = ceil_div(M, balance_chunk_rows(M));
  if (L.chunks < 1) L.chunks = 1;
  L.slots = L.chunks + S;
  L.sums_off = 0;
  L.counts_off = align256(L.slots * E * 4);
  L.tokens_off = L.counts_off + align256(L.slots * E * 4);
  L.loss_off = L.tokens_off + align256(L.slots * 4);
  L.ticket_off = L.loss_off + align256(S * 16 * 8);
  L.total = L.ticket_off + align256(S * 4);
  return L;
}

hipError_t launch_balance_loss(const BalanceArgs& a, hipStream_t stream) {
  const BalanceLayout L = balance_layout(a.M, a.E, a.S);
  const int rows = balance_chunk_rows(a.M);
  float* psums = (float*)(a.ws + L.sums_off);
  int32_t* pcounts = (int32_t*)(a.ws + L.counts_off);
  int32_t* ptokens = (int32_t*)(a.ws + L.tokens_off);
  int32_t* tickets = (int32_t*)(a.ws + L.ticket_off);
  hipError_t err = by_width(a, [&](auto nv, auto vec) {
    balance_rows_kernel<decltype(nv)::value, decltype(vec)::value>
        <<<(unsigned)L.chunks, kThreads, 0, stream>>>(a, rows, psums, pcounts, ptokens, tickets);
  });
  if (err != hipSuccess) return err;
  // few sequences: one workgroup per 64 experts of each
  const unsigned groups = a.S >= 32 ? 1u : (unsigned)ceil_div(a.E, 64);
  balance_finalize_kernel<<<dim3(groups, (unsigned)a.S), kFinThreads, 0, stream>>>(
      a, rows, psums, pcounts, ptokens, (double*)(a.ws + L.loss_off), tickets);
  return hipGetLastError();
}

hipError_t launch_balance_backward(const BalanceArgs& a, hipStream_t stream) {
  const int rows = kRowsPerPass * (a.M > 2048 * kRowsPerPass ? 4 : 1);
  return by_width(a, [&](auto nv, auto vec) {
    balance_backward_kernel<decltype(nv)::value, decltype(vec)::value>
        <<<(unsigned)ceil_div(a.M, rows), kThreads, 0, stream>>>(a, rows);
  });
}

}  // namespace moe
