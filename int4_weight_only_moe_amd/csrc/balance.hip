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
// a row fits into the registers of 16 lanes (32 from 513 experts on: at most 32
// values a lane), so the softmax needs no second pass and the backward pass
// recomputes p rather than reading a stored copy. 16 lanes a row (not a whole
// wave) makes a row's maximum and sum four register exchanges and lets a wave's
// load instruction cover four rows in 256-byte pieces.
#include <type_traits>

#include "device_common.h"
#include "operators.h"
#include "row_common.h"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kPassRows = kThreads / 16;  // rows of a backward pass at 16 lanes a row
constexpr int kMaxExperts = 1024;

// A sequence and its rows [lo, hi).
struct Sequence {
  int s, lo, hi;
};

// The last sequence that starts at or before row t (offsets ascending), the
// first if none does; t is the same in all lanes of the wave. 64 offsets are
// compared at a time, one load each where a binary search waits for six.
__device__ __forceinline__ Sequence sequence_of(const BalanceArgs& a, int t) {
  if (!a.offsets) return {0, 0, a.M};
  const int lane = threadIdx.x & 63;
  int base = 0, n = a.S;  // the answer is in [base, base + n)
  while (n >= 64) {
    const int step = (n + 63) / 64;
    const int at = lane * step;
    const uint64_t below = __ballot(at < n && a.offsets[base + (at < n ? at : 0)] <= t);
    const int k = below ? 63 - __builtin_clzll(below) : 0;
    base += k * step;
    n = n - k * step < step ? n - k * step : step;
  }
  const int off = a.offsets[base + (lane <= n ? lane : n)];
  const uint64_t below = __ballot(lane < n && off <= t);
  const int k = below ? 63 - __builtin_clzll(below) : 0;
  return {base + k, __shfl(off, k, 64), __shfl(off, k + 1, 64)};
}

__device__ __forceinline__ int clamp_row(int v, int M) { return v < 0 ? 0 : (v > M ? M : v); }

// Sums of a wave's rows (lanes l, l + Lanes, ...) to out[expert]. Each exchange
// takes two values and leaves one of them summed in either half of the lanes, a
// quarter of the work of summing each value into every lane (the kernel
// 11.5 us instead of 12.8 for [16384, 384], 27 instead of 31 for [32768, 1024]).
__device__ __forceinline__ float half_sums32(float a, float b) {  // lanes 0..31: a's, 32..63: b's
  const auto h = __builtin_amdgcn_permlane32_swap(__float_as_uint(a), __float_as_uint(b), false, false);
  return __uint_as_float(h[0]) + __uint_as_float(h[1]);
}
__device__ __forceinline__ float half_sums16(float a, float b) {  // even 16 lanes: a's, odd 16: b's
  const auto h = __builtin_amdgcn_permlane16_swap(__float_as_uint(a), __float_as_uint(b), false, false);
  return __uint_as_float(h[0]) + __uint_as_float(h[1]);
}
template <int Lanes, int NV>
__device__ __forceinline__ void join_rows(const float (&v)[4 * NV], float* out) {
  const int lane = threadIdx.x & 63, l = lane % Lanes;
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    if constexpr (Lanes == 16) {
      const int q = (lane >> 5) + 2 * ((lane >> 4) & 1);
      out[64 * j + 4 * l + q] = half_sums16(half_sums32(v[4 * j], v[4 * j + 1]), half_sums32(v[4 * j + 2], v[4 * j + 3]));
    } else {
      *(float2*)(out + 128 * j + 4 * l + 2 * (lane >> 5)) =
          make_float2(half_sums32(v[4 * j], v[4 * j + 2]), half_sums32(v[4 * j + 1], v[4 * j + 3]));
    }
  }
}

constexpr int kSumThreads = 1024;
constexpr int kSumWaves = kSumThreads / 64;
constexpr int kSumRows = kSumThreads / 16;  // rows of a forward pass at 16 lanes a row
// Passes whose rows a lane adds in fp32. Longer chunks (from 2^20 rows on) add the
// runs in fp64: equal rows round in the same direction at every addition, and one
// run of 4096 additions was off by 4e-5.
constexpr int kSumRun = 64;

// One chunk of rows: for each sequence in it, the chunk's sums of
// probabilities, counts and valid rows, to slot chunk + sequence. 16 waves, so
// that 64 rows are in flight at once: with 4 waves and the next row prefetched
// [16384, 384] took 13.8 us, bound by the loads' latency. The first row and the
// first choices of the chunk are loaded before the sequence is looked up.
// [16384, 384] with offsets and padding 11.5 us (25 MB: one pass, bound by the
// latencies of that and of the join; 9.7 without exponentials, counts, join and
// stores), [32768, 1024] 27 us (4.9 TB/s).
template <int Lanes, int NV, bool Vec>
__global__ __launch_bounds__(kSumThreads) void balance_rows_kernel(BalanceArgs a, int chunk_rows, float* psums,
                                                                   int32_t* pcounts, int32_t* ptokens,
                                                                   int32_t* tickets, bool only) {
  __shared__ double parts[kSumWaves];
  __shared__ int cnt[kMaxExperts];
  __shared__ __align__(16) float sums[kSumWaves][4 * Lanes * NV];
  __shared__ int live_rows;
  constexpr int kRows = kSumThreads / Lanes;
  const int tid = threadIdx.x, l = tid % Lanes, group = tid / Lanes, wave = tid >> 6;
  const int E = a.E, k = a.k;
  const int r0 = blockIdx.x * chunk_rows;
  const int r1 = r0 + chunk_rows < a.M ? r0 + chunk_rows : a.M;
  float v[4 * NV];
  bool live = false;  // the row in v counts
  auto fetch = [&](int t, int end) {
    if (t < end) {
      load_row<Lanes, NV, Vec>(a.logits + (int64_t)t * E, E, l, v);
      live = !a.valid || a.valid[t];
    }
  };
  fetch(r0 + group, r1);
  const int32_t* chunk_ids = a.topk_ids + (int64_t)r0 * k;
  const unsigned chunk_n = r0 < r1 ? (unsigned)(r1 - r0) * (unsigned)k : 0;
  const int first_id = (unsigned)tid < chunk_n ? chunk_ids[tid] : -1;
  const bool first_live = (unsigned)tid < chunk_n && (!a.valid || a.valid[r0 + (unsigned)tid / (unsigned)k]);
  // the finalize kernel's tickets start at zero
  if (!only)
    for (int s = blockIdx.x * kSumThreads + tid; s < a.S; s += gridDim.x * kSumThreads) tickets[s] = 0;
  if (r0 >= r1 && !only) return;
  Sequence seq = only ? Sequence{0, a.offsets ? clamp_row(a.offsets[0], a.M) : 0,
                                 a.offsets ? clamp_row(a.offsets[1], a.M) : a.M}
                      : sequence_of(a, r0);
  bool fetched = true;  // v holds row r0 + group if that is in this sequence
  for (; seq.s < a.S; ++seq.s, seq.lo = seq.hi, seq.hi = seq.s < a.S ? a.offsets[seq.s + 1] : 0) {
    const int s = seq.s;
    if (seq.lo >= r1 && !only) break;
    const int lo = seq.lo > r0 ? seq.lo : r0;
    int hi = seq.hi < r1 ? seq.hi : r1;
    if (lo >= hi && !only) continue;
    hi = hi < lo ? lo : hi;
    if (tid < E) cnt[tid] = 0;
    if (tid == 0) live_rows = 0;
    __syncthreads();
    const unsigned i0 = (unsigned)(lo - r0) * (unsigned)k, i1 = (unsigned)(hi - r0) * (unsigned)k;
    if ((unsigned)tid >= i0 && (unsigned)tid < i1 && first_live && first_id >= 0 && first_id < E)
      atomicAdd(&cnt[first_id], 1);
    for (unsigned at = tid + kSumThreads; at < i1; at += kSumThreads) {
      if (at < i0) continue;
      const int e = chunk_ids[at];
      if (e >= 0 && e < E && (!a.valid || a.valid[r0 + at / (unsigned)k])) atomicAdd(&cnt[e], 1);
    }
    double total = 0.0;
    for (int from = lo;;) {  // a run of rows
      const int to = hi - from > kSumRun * kRows ? from + kSumRun * kRows : hi;
      float acc[4 * NV];
#pragma unroll
      for (int i = 0; i < 4 * NV; ++i) acc[i] = 0.0f;
      int rows = 0;
      for (int t = from + group; t < to; t += kRows) {
        if (!fetched || t != r0 + group) fetch(t, hi);
        if (!live) continue;
        ++rows;
        const float inv = exp_row<Lanes>(v);
#pragma unroll
        for (int i = 0; i < 4 * NV; ++i) acc[i] = fmaf(v[i], inv, acc[i]);
      }
      fetched = false;
      if (l == 0 && rows) atomicAdd(&live_rows, rows);
      // the wave's rows, then the waves
      join_rows<Lanes, NV>(acc, sums[wave]);
      __syncthreads();
      float sum = 0.0f;
      if (tid < E) {
#pragma unroll
        for (int w = 0; w < kSumWaves; ++w) sum += sums[w][tid];
      }
      total += (double)sum;
      from = to;
      if (from >= hi) break;
      __syncthreads();
    }
    const int64_t slot = (int64_t)blockIdx.x + s;
    if (only) {  // all of the sequence is here
      double part = tid < E ? total * (double)cnt[tid] : 0.0;
#pragma unroll
      for (int d = 32; d; d >>= 1) part += __shfl_xor(part, d, 64);
      if ((tid & 63) == 0) parts[wave] = part;
      if (tid < E) {
        a.prob_sums[(int64_t)s * E + tid] = (float)total;
        a.counts[(int64_t)s * E + tid] = cnt[tid];
      }
      __syncthreads();
      if (tid == 0) {
        double loss = 0.0;
        for (int w = 0; w < kSumWaves; ++w) loss += parts[w];
        const double T = live_rows;
        a.tokens[s] = live_rows;
        a.loss[s] = live_rows ? (float)(loss * (double)E / ((double)k * T * T)) : 0.0f;
      }
      __syncthreads();
      continue;
    }
    if (tid < E) {
      psums[slot * E + tid] = (float)total;
      pcounts[slot * E + tid] = cnt[tid];
    }
    if (tid == 0) ptokens[slot] = live_rows;
    __syncthreads();
  }
}

// Batches that one workgroup sums alone, with no second launch: 128 rows are two
// passes, which cost less than a launch.
bool one_workgroup(int64_t M, int64_t S) { return M <= 2 * kSumRows && S <= 64; }

// Sums a sequence's slots for 64 experts at a time, in a fixed order and in
// fp64, and the loss. With several workgroups a sequence (gridDim.x > 1) each
// leaves its part of the loss, and the last one to finish (the ticket) adds
// the parts in order. Bound by latency: 5.6 us for 4 sequences of 384 experts,
// 7.0 for one of 1024 in 256 chunks.
constexpr int kFinThreads = 1024;
__global__ __launch_bounds__(kFinThreads) void balance_finalize_kernel(BalanceArgs a, int chunk_rows,
                                                                       const float* psums, const int32_t* pcounts,
                                                                       const int32_t* ptokens, double* ploss,
                                                                       int32_t* tickets) {
  constexpr int kAhead = 8;
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
  double loss = 0.0;
  for (int g = blockIdx.x; g < groups; g += gridDim.x) {
    const int e = 64 * g + lane;
    double sum = 0.0;
    int cnt = 0;
    for (int c = c0 + wave; c < c1; c += 16 * kAhead) {  // kAhead slots' loads at once
      float f[kAhead];
      int n[kAhead];
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        const int64_t at = ((int64_t)(c + 16 * i < c1 ? c + 16 * i : c) + s) * E + (e < E ? e : 0);
        f[i] = psums[at];
        n[i] = pcounts[at];
      }
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        sum += c + 16 * i < c1 ? (double)f[i] : 0.0;
        cnt += c + 16 * i < c1 ? n[i] : 0;
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
      double part = e < E ? sum * (double)cnt : 0.0;
#pragma unroll
      for (int d = 32; d; d >>= 1) part += __shfl_xor(part, d, 64);
      loss += part;
    }
    __syncthreads();
  }
#pragma unroll
  for (int d = 32; d; d >>= 1) tok += __shfl_xor(tok, d, 64);
  if (lane == 0) dtok[wave] = tok;
  __syncthreads();
  if (wave != 0) return;
  tok = 0;
#pragma unroll
  for (int w = 0; w < 16; ++w) tok += dtok[w];
  const double scale = tok ? (double)E / ((double)a.k * (double)tok * (double)tok) : 0.0;
  if (blockIdx.x == 0 && lane == 0) a.tokens[s] = tok;
  if (gridDim.x > 1) {
    // The parts and the ticket are exchanged by read-modify-write operations
    // only, which the whole device performs in one place: a part is there once
    // the old value has come back, and the ticket is drawn after that (it adds
    // what came back, masked to nothing, to the one it draws). A fence would
    // write the L2 back: 7.6 us instead of 5.6.
    unsigned long long* mine = (unsigned long long*)ploss + (int64_t)s * 16;
    int drawn = 0;
    if (lane == 0) {
      const unsigned long long old = __hip_atomic_exchange(
          mine + blockIdx.x, __builtin_bit_cast(unsigned long long, loss), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      int none = (int)old;
      asm volatile("v_and_b32 %0, 0, %0" : "+v"(none));
      drawn = __hip_atomic_fetch_add(tickets + s, 1 + none, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
    if (__builtin_amdgcn_readfirstlane(drawn) != (int)gridDim.x - 1) return;
    loss = 0.0;
    if (lane < (int)gridDim.x)
      loss = __builtin_bit_cast(
          double, __hip_atomic_fetch_or(mine + lane, 0ull, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT));
#pragma unroll
    for (int d = 8; d; d >>= 1) loss += __shfl_xor(loss, d, 64);
  }
  if (lane == 0) a.loss[s] = (float)(loss * scale);
}


// A row's lanes take every kRows-th row of a chunk, the next row in flight
// while they compute one. They hold the counts of its current sequence.
// [16384, 384]: 12.6 us for 50 MB read and written (4.0 TB/s; a copy of as much
// takes 9.3 at the rate of a large one).
template <int Lanes, int NV, bool Vec>
__global__ __launch_bounds__(kThreads) void balance_backward_kernel(BalanceArgs a, int chunk_rows) {
  constexpr int kRows = kThreads / Lanes;
  const int l = threadIdx.x % Lanes, group = threadIdx.x / Lanes;
  const int E = a.E;
  const int r0 = blockIdx.x * chunk_rows;
  const int r1 = r0 + chunk_rows < a.M ? r0 + chunk_rows : a.M;
  float v[4 * NV];
  bool live = false;
  auto fetch = [&](int t) {
    if (t < r1) {
      load_row<Lanes, NV, Vec>(a.logits + (int64_t)t * E, E, l, v);
      live = !a.valid || a.valid[t];
    }
  };
  fetch(r0 + group);
  const Sequence seq = sequence_of(a, r0);
  int s = seq.s, lo = seq.lo, hi = seq.hi;
  float c[4 * NV], w = 0.0f;
  auto counts = [&]() {
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int e = 4 * Lanes * j + 4 * l + q;
        const int n = a.counts[(int64_t)s * E + (e < E ? e : 0)];
        c[4 * j + q] = e < E ? (float)n : 0.0f;
      }
    const float T = (float)a.tokens[s];
    w = T > 0.0f ? a.dloss[s] * ((float)E / ((float)a.k * T)) / T : 0.0f;
  };
  counts();
  for (int t = r0 + group; t < r1; t += kRows) {
    float p[4 * NV];
#pragma unroll
    for (int i = 0; i < 4 * NV; ++i) p[i] = v[i];
    const bool use = live;
    fetch(t + kRows);
    if (t >= hi && s + 1 < a.S) {
      while (t >= hi && s + 1 < a.S) {
        lo = hi;
        hi = a.offsets[++s + 1];
      }
      counts();
    }
    if (t < lo || t >= hi) continue;  // a row of no sequence
    float* g = a.grad + (int64_t)t * E;
    if (use) {
      const float inv = exp_row<Lanes>(p);
      float dot = 0.0f;
#pragma unroll
      for (int i = 0; i < 4 * NV; ++i) dot = fmaf(c[i], p[i], dot);
      dot = row_sum<Lanes>(dot) * inv;
      const float scale = w * inv;
#pragma unroll
      for (int i = 0; i < 4 * NV; ++i) p[i] *= scale * (c[i] - dot);
    } else {
#pragma unroll
      for (int i = 0; i < 4 * NV; ++i) p[i] = 0.0f;
    }
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int e = 4 * Lanes * j + 4 * l;
      if constexpr (Vec) {
        if (e < E) *(float4*)(g + e) = make_float4(p[4 * j], p[4 * j + 1], p[4 * j + 2], p[4 * j + 3]);
      } else {
#pragma unroll
        for (int q = 0; q < 4; ++q)
          if (e + q < E) g[e + q] = p[4 * j + q];
      }
    }
  }
}

// fn(Lanes, NV, Vec) for the row width
template <typename F>
hipError_t by_width(const BalanceArgs& a, F fn) {
  const bool vec = a.E % 4 == 0 && (reinterpret_cast<uintptr_t>(a.logits) & 15) == 0 &&
                   (!a.grad || (reinterpret_cast<uintptr_t>(a.grad) & 15) == 0);
  auto go = [&](auto lanes, auto nv) { vec ? fn(lanes, nv, std::true_type{}) : fn(lanes, nv, std::false_type{}); };
  auto row16 = [&](auto nv) { go(std::integral_constant<int, 16>{}, nv); };
  if (a.E <= 64) row16(std::integral_constant<int, 1>{});
  else if (a.E <= 128) row16(std::integral_constant<int, 2>{});
  else if (a.E <= 256) row16(std::integral_constant<int, 4>{});
  else if (a.E <= 384) row16(std::integral_constant<int, 6>{});
  else if (a.E <= 512) row16(std::integral_constant<int, 8>{});
  else go(std::integral_constant<int, 32>{}, std::integral_constant<int, 8>{});
  return hipGetLastError();
}

}  // namespace

int balance_chunk_rows(int64_t M) {
  // at most 256 chunks of whole passes: a workgroup a CU, few enough that the
  // partials are small beside the logits
  const int64_t rows = ceil_div(ceil_div(M, 256), kSumRows) * kSumRows;
  return (int)(rows < kSumRows ? kSumRows : rows);
}

static int64_t align256(int64_t v) { return (v + 255) & ~int64_t(255); }

BalanceLayout balance_layout(int64_t M, int64_t E, int64_t S) {
  BalanceLayout L;
  L.chunks = ceil_div(M, balance_chunk_rows(M));
  if (L.chunks < 1) L.chunks = 1;
  // room for what any smaller batch takes too
  const int64_t most = ceil_div(M, kSumRows);
  L.slots = (most < 1 ? 1 : most > 256 ? 256 : most) + S;
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
  const bool only = one_workgroup(a.M, a.S);
  const int rows = only ? 2 * kSumRows : balance_chunk_rows(a.M);
  float* psums = (float*)(a.ws + L.sums_off);
  int32_t* pcounts = (int32_t*)(a.ws + L.counts_off);
  int32_t* ptokens = (int32_t*)(a.ws + L.tokens_off);
  int32_t* tickets = (int32_t*)(a.ws + L.ticket_off);
  hipError_t err = by_width(a, [&](auto lanes, auto nv, auto vec) {
    balance_rows_kernel<decltype(lanes)::value, decltype(nv)::value, decltype(vec)::value>
        <<<only ? 1u : (unsigned)L.chunks, kSumThreads, 0, stream>>>(a, rows, psums, pcounts, ptokens, tickets, only);
  });
  if (err != hipSuccess || only) return err;
  // few sequences: one workgroup per 64 experts of each
  const unsigned groups = a.S >= 32 ? 1u : (unsigned)ceil_div(a.E, 64);
  balance_finalize_kernel<<<dim3(groups, (unsigned)a.S), kFinThreads, 0, stream>>>(
      a, rows, psums, pcounts, ptokens, (double*)(a.ws + L.loss_off), tickets);
  return hipGetLastError();
}

hipError_t launch_balance_backward(const BalanceArgs& a, hipStream_t stream) {
  // two passes a workgroup, so that the counts are read for more than one row
  // and the second row is in flight, once that leaves two workgroups a CU; more
  // from 2^24 rows on (a grid has fewer than 2^32 threads)
  const int passes = a.M >= 1024 * kPassRows ? 2 * (int)ceil_div(a.M, int64_t(1) << 24) : 1;
  const int rows = kPassRows * passes;
  return by_width(a, [&](auto lanes, auto nv, auto vec) {
    balance_backward_kernel<decltype(lanes)::value, decltype(nv)::value, decltype(vec)::value>
        <<<(unsigned)ceil_div(a.M, rows), kThreads, 0, stream>>>(a, rows);
  });
}

}  // namespace moe
