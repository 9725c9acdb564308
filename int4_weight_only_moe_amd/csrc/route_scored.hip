// Routing by scores and its gradient.
//
// s = softmax(l) or sigmoid(l) of a token's logits, c = s + bias; the groups of
// the highest scores, the k experts of the highest c in them, weights from s.
// A row of logits lies in the registers of 16 or 32 lanes.
//
// Finding the k highest without k passes over the row: the k-th highest of the
// lanes' own maxima (k exchanges within the row) is a threshold that at least k
// values reach and few others do (for 384 values and k = 8 some 11). The places
// of these candidates go to LDS, where each is ranked by counting the higher ones.
//
// The choice is that of c in fp64, but hardly a row needs fp64 for that: only
// where fp32 values that decide the choice are closer than their error bound are
// the candidates' c computed again in fp64. (Equal logits with equal biases need
// no such decision: the lower expert goes first.) Where that decides between
// groups, or a value is NaN (with a bias or groups: not finite, an absent expert's
// too), or the candidates are too many, the wave computes the whole row again in
// fp64 (route_row_exact), some 6 us for one row. Back to back in a graph, sigmoid and a
// bias: [4096, 256] in 8 groups 7.1 to 7.6 us for inputs without such a row (about
// three in four), 13.2 with one; [8192, 1024] in 16 groups 19.4 and 27.8; [16384, 384]
// with every row there (one bias of -inf) 57 instead of 10.8.
#include <type_traits>

#include "device_common.h"
#include "internal.h"
#include "operators.h"
#include "row_common.h"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;
constexpr int kMaxCand = 64;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kDenom = 1e-20f;  // added to the kept sigmoid scores' sum

// LDS written by lanes of this wave becomes visible to its other lanes.
__device__ __forceinline__ void wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

template <int Lanes>
__device__ __forceinline__ uint32_t row_max_u32(uint32_t v) {
  v = umax(v, dpp<kQuadSwap1>(v));
  v = umax(v, dpp<kQuadSwap2>(v));
  v = umax(v, dpp<kRowHalfMirror>(v));
  v = umax(v, dpp<kRowMirror>(v));
  if constexpr (Lanes == 32) {
    const auto h = __builtin_amdgcn_permlane16_swap(v, v, false, false);
    v = umax(h[0], h[1]);
  }
  return v;
}

// Sum over the lower lanes of the row; `total` over all of them.
template <int Lanes>
__device__ __forceinline__ int row_before(int v, int& total) {
  uint32_t incl = (uint32_t)v;
  incl += dpp<0x111>(incl);  // row_shr by 1, 2, 4, 8: lanes without a source add 0
  incl += dpp<0x112>(incl);
  incl += dpp<0x114>(incl);
  incl += dpp<0x118>(incl);
  uint32_t all = row_max_u32<16>(incl);
  if constexpr (Lanes == 32) {
    const auto h = __builtin_amdgcn_permlane16_swap(all, all, false, false);
    const uint32_t both = h[0] + h[1];
    incl += (threadIdx.x & 16) ? both - all : 0u;
    all = both;
  }
  total = (int)all;
  return (int)incl - v;
}

// Whether any lane of the row says so (the whole wave calls it).
template <int Lanes>
__device__ __forceinline__ bool row_any(bool b) {
  const uint64_t m = __ballot(b) >> (threadIdx.x & (64 - Lanes));
  return Lanes == 32 ? (uint32_t)m != 0 : (m & 0xffffu) != 0;
}

// Order-preserving keys: NaN the highest; 0 is below them all.
__device__ __forceinline__ uint64_t key64(double v) {
  const uint64_t u = (uint64_t)__double_as_longlong(v + 0.0);
  const uint64_t k = (u >> 63) ? ~u : (u | 0x8000000000000000ull);
  return v != v ? ~0ull : k;
}
__device__ __forceinline__ double key64_value(uint64_t k) {
  return __longlong_as_double((long long)((k >> 63) ? (k & 0x7FFFFFFFFFFFFFFFull) : ~k));
}

// The softmax of a row as exp2(l' log2(e) - ml) * inv, l' = l - first (see
// exp_row: the rounding of ml is a factor of the whole row).
struct RowSoftmax {
  float first, ml, inv;
  __device__ __forceinline__ float exp_of(float l) const {
    return __builtin_amdgcn_exp2f(fmaf(l - first, kLog2e, -ml));
  }
};
template <int Lanes, int N>
__device__ __forceinline__ RowSoftmax row_softmax(const float (&v)[N]) {
  float m = v[0];
#pragma unroll
  for (int i = 1; i < N; ++i) m = fmaxf(m, v[i]);
  m = row_max<Lanes>(m);
  m = m == -INFINITY ? 0.0f : m;
  const bool far = fabsf(m) >= 0x1p20f;
  RowSoftmax r;
  r.first = far ? m : 0.0f;
  r.ml = far ? 0.0f : m * kLog2e;
  float s = 0.0f;
#pragma unroll
  for (int i = 0; i < N; ++i) s += r.exp_of(v[i]);
  s = row_sum<Lanes>(s);
  r.inv = s == 0.0f ? 0.0f : 1.0f / s;
  return r;
}

__device__ __forceinline__ float sigmoid_of(float l) {  // to the last bits for any l
  const float e = expf(-fabsf(l));
  return l != l ? l : (l >= 0.0f ? 1.0f : e) / (1.0f + e);
}

// A score (or its slope, for logits of either sign) that may be subnormal in fp32 is
// the square of half_exp, which is not: what it is divided or multiplied by goes in
// between the two.
__device__ __forceinline__ bool tiny_exp(float l) { return fabsf(l) > 80.0f; }
__device__ __forceinline__ float half_exp(float l) { return expf(-0.5f * fabsf(l)); }

// Scores as the fast path computes them.
__device__ __forceinline__ float fast_sigmoid(float l) {
  return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-kLog2e * l));
}

struct Chosen {
  int e;    // -1: none
  float l;  // its logit
};

// One row's choice in fp64 by the whole wave, to sel[0..k). keys: E 64-bit words
// of this wave. (Not inlined: its registers would halve the waves of the kernel.)
__device__ __attribute__((noinline)) void route_row_exact(const float* row, const float* bias, int E, int k,
                                                          bool sigmoid, int G, int top_groups, int group_top,
                                                          uint64_t* keys, Chosen* sel) {
  const int lane = threadIdx.x & 63;
  const bool grouped = top_groups < G;
  // without scores in it the choice is that of the logits
  const bool logits = !bias && (!grouped || group_top == 1);
  double m = -INFINITY, sum = 1.0;
  if (!sigmoid && !logits) {
#pragma unroll 1
    for (int e = lane; e < E; e += 64) m = fmax(m, (double)row[e]);
#pragma unroll 1
    for (int d = 32; d; d >>= 1) m = fmax(m, __shfl_xor(m, d, 64));
    sum = 0.0;
#pragma unroll 1
    for (int e = lane; e < E; e += 64) sum += exp((double)row[e] - m);
#pragma unroll 1
    for (int d = 32; d; d >>= 1) sum += __shfl_xor(sum, d, 64);
  }
#pragma unroll 1
  for (int e = lane; e < E; e += 64) {
    const double l = row[e], b = bias ? (double)bias[e] : 0.0;
    uint64_t key = 0;
    if (l != -INFINITY && b != -INFINITY) {
      if (logits) key = key64(l);
      else key = key64((sigmoid ? 1.0 / (1.0 + exp(-l)) : exp(l - m) / sum) + b);
    }
    keys[e] = key;
  }
  wave_sync();
  if (grouped) {
    const int gs = E / G;
    // P lanes a group: lane g P + i takes every P-th of its keys from the i-th on
    int P = 1;
    while (2 * P * G <= 64) P *= 2;
    uint64_t m1 = 0, m2 = 0;
    if (lane < G * P) {
#pragma unroll 4
      for (int i = lane & (P - 1); i < gs; i += P) {
        const uint64_t x = keys[lane / P * gs + i];
        m2 = x > m1 ? m1 : (x > m2 ? x : m2);
        m1 = x > m1 ? x : m1;
      }
    }
#pragma unroll 1
    for (int d = 1; d < P; d *= 2) {
      const uint64_t o1 = __shfl_xor((unsigned long long)m1, d, 64), o2 = __shfl_xor((unsigned long long)m2, d, 64);
      const uint64_t low = o1 > m1 ? m1 : o1;
      m2 = m2 > o2 ? m2 : o2;
      m2 = low > m2 ? low : m2;
      m1 = o1 > m1 ? o1 : m1;
    }
    const uint64_t score = group_top == 2 && m2 ? key64((m1 == ~0ull ? NAN : key64_value(m1)) +
                                                        (m2 == ~0ull ? NAN : key64_value(m2)))
                                                : m1;
    const uint64_t mine = __shfl((unsigned long long)score, lane * P & 63, 64);  // lane g: group g's
    int rank = 0;
    for (int g = 0; g < G; ++g) {
      const uint64_t o = __shfl((unsigned long long)mine, g, 64);
      rank += o > mine || (o == mine && g < lane);
    }
    const uint64_t chosen = __ballot(lane < G && mine && rank < top_groups);
#pragma unroll 1
    for (int e = lane; e < E; e += 64) {
      uint64_t key = keys[e];
      if (!((chosen >> (e / gs)) & 1)) key = 0;
      else if (key && !bias) key = key64((double)row[e]);
      keys[e] = key;
    }
  }
#pragma unroll 1
  for (int r = 0; r < k; ++r) {
    uint64_t best = 0;
    int at = E;
#pragma unroll 4
    for (int e = lane; e < E; e += 64) {
      const uint64_t x = keys[e];
      at = x > best ? e : at;
      best = x > best ? x : best;
    }
    uint32_t hi = (uint32_t)(best >> 32), lo = (uint32_t)best;
    wave_max_pair(hi, lo);
    const bool top = (uint32_t)(best >> 32) == hi && (uint32_t)best == lo;
    const int e = (int)wave_min_u32(top ? (uint32_t)at : 0xFFFFFFFFu);
    const bool none = (hi | lo) == 0;
    if (lane == 0) sel[r] = none ? Chosen{-1, -INFINITY} : Chosen{e, row[e]};
    if (!none && (e & 63) == lane) keys[e] = 0;
  }
  wave_sync();
}

constexpr int kStep = 8;  // keys compared in a step of the ranking

// Dynamic LDS of one wave: with groups the values of its rows, padded so that
// the groups of a row and the rows start in different banks; then the
// candidates' c in fp64; then the 64-bit keys of one row (exact path).
// Groups of 4 n >= 16 experts are 4 words apart, so that 4 neighbours of a lane
// are one 16-byte access; others 1 word.
__host__ __device__ constexpr int group_pad(int size) { return size % 4 == 0 && size >= 16 ? 4 : 1; }
__host__ __device__ constexpr int row_pitch(int E, int groups) {
  return (E + groups * group_pad(E / groups) + 63) / 64 * 64 + 16;
}
__host__ __device__ constexpr int row_buffer_bytes(int lanes, bool biased, bool grouped, int E, int groups) {
  int bytes = E * 8;
  if (grouped) bytes = row_pitch(E, groups) * (64 / lanes) * 4;
  if (biased && bytes < 64 / lanes * kMaxCand * 8) bytes = 64 / lanes * kMaxCand * 8;
  return bytes;
}

template <int Lanes, bool General>
struct RouteShared {
  static constexpr int kRows = kThreads / Lanes;
  Chosen sel[kRows][16];
  union {
    // the candidates: (order key of c) << 32 | ~expert, zeros behind them
    __align__(16) uint64_t key[kMaxCand + kStep];
    float groups[64][2];  // before that, the groups' scores and what they may be off
  } row[kRows];
  // with a bias: what c is computed from, and the candidates by rank
  float l[General ? kRows : 1][kMaxCand], b[General ? kRows : 1][kMaxCand];
  uint8_t by_rank[General ? kRows : 1][kMaxCand];
};

// Routes the rows t0 + wave * (64 / Lanes) + lane / Lanes of this workgroup.
// General: with a bias or groups. copy: also gets the ids (LDS), or null.
template <int Lanes, int NV, bool Vec, bool General>
__device__ __forceinline__ void route_rows(const ScoredArgs& a, int64_t t0, RouteShared<Lanes, General>& sh,
                                           float* buffer,
                                           int32_t* copy) {
  constexpr int N = 4 * NV, kRows = 64 / Lanes;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, l = lane % Lanes, sub = lane / Lanes;
  const int E = a.E, k = a.k;
  const int64_t t = t0 + wave * kRows + sub;
  const bool active = t < a.M;
  const float* row = a.logits + (active ? t : (int64_t)a.M - 1) * E;
  const int r = wave * kRows + sub;
  const bool grouped = General && a.top_groups < a.groups;
  buffer += row_buffer_bytes(Lanes, a.bias != nullptr, grouped, E, a.groups) / 4 * wave;
  float v[N];  // the logits, then what the experts are ordered by
  load_row<Lanes, NV, Vec>(row, E, l, v);
  const bool live = active && (!a.valid || a.valid[t]);
  RowSoftmax soft{0.0f, 0.0f, 0.0f};
  if (!a.sigmoid && (General || !a.renorm)) soft = row_softmax<Lanes>(v);
  auto expert_of = [&](int i) { return 4 * Lanes * (i >> 2) + 4 * l + (i & 3); };
  auto inside = [&](int i) { return expert_of(Vec ? i & ~3 : i) < E; };  // (Vec: E % 4 == 0)
  auto fast_score = [&](float x) { return a.sigmoid ? fast_sigmoid(x) : soft.exp_of(x) * soft.inv; };

  // rows that need the exact path: NaN, and with scores in the choice whatever is not finite
  bool bad = false;
#pragma unroll
  for (int i = 0; i < N; i += 2) bad |= __builtin_isunordered(v[i], v[i + 1]);
  float near = 0.0f;     // closer values need fp64
  float largest = 0.0f;  // of a lane's |l| and |c|
  if constexpr (General) {
    // fp32 errors in roundings of 2^-24: a sigmoid's are (1 - s) s (1.3 |l| + 2) + 3 s
    // < 4; a softmax value's p = pmax e^-x are (1.5 x + 50) p < 50 pmax (x from the
    // exponent, the rest from the row's sum). c adds |c|, a sum of two c its own. Twice
    // the first is `near`; what |c| adds is counted where c is known.
    const float score_error = a.sigmoid ? 0x1p-22f : 0x1p-18f * soft.inv;
#pragma unroll
    for (int i = 0; i < N; ++i) largest = fmaxf(largest, inside(i) ? fabsf(v[i]) : 0.0f);
    if (a.bias) {
      float b[N];
      load_row<Lanes, NV, Vec>(a.bias, E, l, b);
#pragma unroll
      for (int i = 0; i < N; ++i) {
        v[i] = fast_score(v[i]) + b[i];
        largest = fmaxf(largest, inside(i) ? fabsf(v[i]) : 0.0f);
        bad |= __builtin_isunordered(b[i], b[i]);
      }
      near = 2.0f * score_error;
    }
    bad |= !(largest < 1e30f);
    if (grouped) {
      const int G = a.groups, gs = E / G;
      const uint32_t magic = (1u << 20) / (uint32_t)gs + 1u;  // e / gs = e * magic >> 20 for e < 1024
      auto group_of = [&](int e) { return (int)((uint32_t)e * magic >> 20); };
      const int pad = group_pad(gs);
      const bool quads = Vec && pad == 4;
      float* mine = buffer + sub * row_pitch(E, G);  // expert e of group g at e + pad g
      const bool raw = a.bias || a.group_top == 1;   // (the highest logit has the highest score)
      auto write_row = [&](auto value) {
        if (quads) {
#pragma unroll
          for (int j = 0; j < NV; ++j) {
            const int e = expert_of(4 * j);
            if (e < E)
              *(float4*)(mine + e + 4 * group_of(e)) =
                  make_float4(value(4 * j), value(4 * j + 1), value(4 * j + 2), value(4 * j + 3));
          }
        } else {
#pragma unroll
          for (int i = 0; i < N; ++i) {
            const int e = expert_of(i);
            if (inside(i)) mine[e + pad * group_of(e)] = value(i);
          }
        }
      };
      if (raw) write_row([&](int i) { return v[i]; });
      else write_row([&](int i) { return fast_score(v[i]); });
      wave_sync();
      // P lanes a group
      int P = 1;
      while (P < 8 && 2 * P * G <= Lanes) P *= 2;
      const bool quad_scan = pad == 4 && gs % (4 * P) == 0;
      for (int g = l / P; g < G; g += Lanes / P) {
        float m1 = -INFINITY, m2 = -INFINITY;
        auto take = [&](float x) {
          m2 = fmaxf(m2, fminf(m1, x));
          m1 = fmaxf(m1, x);
        };
        const float* from = mine + g * (gs + pad);
        if (quad_scan) {
#pragma unroll 4
          for (int i = 4 * (l % P); i < gs; i += 4 * P) {
            const float4 x = *(const float4*)(from + i);
            take(x.x);
            take(x.y);
            take(x.z);
            take(x.w);
          }
        } else {
#pragma unroll 4
          for (int i = l % P; i < gs; i += P) take(from[i]);
        }
        auto join = [&](uint32_t o1b, uint32_t o2b) {
          const float o1 = __uint_as_float(o1b), o2 = __uint_as_float(o2b);
          m2 = fmaxf(fminf(m1, o1), fmaxf(m2, o2));
          m1 = fmaxf(m1, o1);
        };
        if (P > 1) join(dpp<kQuadSwap1>(__float_as_uint(m1)), dpp<kQuadSwap1>(__float_as_uint(m2)));
        if (P > 2) join(dpp<kQuadSwap2>(__float_as_uint(m1)), dpp<kQuadSwap2>(__float_as_uint(m2)));
        if (P > 4) join(dpp<kRowHalfMirror>(__float_as_uint(m1)), dpp<kRowHalfMirror>(__float_as_uint(m2)));
        const bool two = a.group_top == 2;
        const float off = !two && !a.bias ? 0.0f
                                          : (two ? 2.0f : 1.0f) * score_error +
                                                0x1p-22f * (fabsf(m1) + (two ? fabsf(m2) : 0.0f));
        *(float2*)sh.row[r].groups[g] = make_float2(two ? m1 + m2 : m1, off);
      }
      wave_sync();
      uint64_t chosen = 0;
      float in = INFINITY, out = -INFINITY;
      for (int g0 = 0; g0 < G; g0 += Lanes) {
        const int g = g0 + l;
        const float s = g < G ? sh.row[r].groups[g][0] : 0.0f, off = g < G ? sh.row[r].groups[g][1] : 0.0f;
        int rank = 0;
#pragma unroll 8
        for (int h = 0; h < G; ++h) {
          const float o = sh.row[r].groups[h][0];
          rank += (int)(o > s) | ((int)(o == s) & (int)(h < g));
        }
        const bool take = g < G && rank < a.top_groups;
        const uint64_t m = __ballot(take) >> (lane & (64 - Lanes));
        chosen |= (Lanes == 32 ? (m & 0xffffffffu) : (m & 0xffffu)) << g0;
        in = take ? fminf(in, s - off) : in;
        out = g < G && !take ? fmaxf(out, s + off) : out;
      }
      in = -row_max<Lanes>(-in);
      out = row_max<Lanes>(out);
      if (a.bias || a.group_top == 2) bad |= !(in > out);
      // The values in another order: a lane's experts lie `Lanes` apart, so that
      // a group's are spread over all lanes. (Neighbours of 4 a lane leave lanes
      // empty, the threshold is then low and the candidates are many: ranking
      // them took 8 of 15 us for [4096, 256] in 8 groups.) Those of groups that
      // are not chosen are taken out by the groups' lanes first.
      if (!raw) {
        write_row([&](int i) { return v[i]; });
        wave_sync();
      }
      for (int g = l / P; g < G; g += Lanes / P) {
        if ((chosen >> g) & 1) continue;
        float* from = mine + g * (gs + pad);
        if (quad_scan) {
          for (int i = 4 * (l % P); i < gs; i += 4 * P)
            *(float4*)(from + i) = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
        } else {
          for (int i = l % P; i < gs; i += P) from[i] = -INFINITY;
        }
      }
      wave_sync();
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const int e = l + Lanes * i;
        v[i] = e < E ? mine[e + pad * group_of(e)] : -INFINITY;
      }
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i)
        if (!inside(i)) v[i] = -INFINITY;
    }
  }

  // the threshold (as an integer key: its maxima are one instruction an exchange)
  float top = v[0];
#pragma unroll
  for (int i = 1; i < N; ++i) top = fmaxf(top, v[i]);
  uint32_t top_key = order_key(top), limit_key = 0;
#pragma unroll 1
  for (int i = 0; i < k; ++i) {
    limit_key = row_max_u32<Lanes>(top_key);
    top_key = top_key == limit_key ? 0u : top_key;
  }
  float limit = limit_key ? key_value(limit_key) : -INFINITY;
  if (General && a.bias) {
    // (no limit: fewer than k lanes have a value, and every value is a candidate)
    near += 0x1p-22f * (limit == -INFINITY ? row_max<Lanes>(largest) : fabsf(limit));
    limit -= near;
  }
  limit = fmaxf(limit, -3.402823466e38f);

  // the candidates
  if (l < 16) sh.sel[r][l] = {-1, -INFINITY};
  uint32_t mask = 0;  // bit N - 1 - i: value i
#pragma unroll
  for (int i = 0; i < N; ++i) mask = mask + mask + (v[i] >= limit ? 1u : 0u);
  int n;
  int at = row_before<Lanes>(__builtin_popcount(mask), n);
  while (__any(mask)) {
    const int i = N - 1 - (mask ? __builtin_ctz(mask) : 0);
    if (mask && at < kMaxCand) sh.row[r].key[at] = (uint32_t)(grouped ? l + Lanes * i : expert_of(i));
    ++at;
    mask &= mask - 1;
  }
  wave_sync();
  bad |= n > kMaxCand;
  n = n < kMaxCand ? n : kMaxCand;
  if (l < kStep) sh.row[r].key[n + l] = 0;
  for (int i = l; i < n; i += Lanes) {
    const int e = (int)sh.row[r].key[i];
    const float x = row[e];
    float c = x;
    if constexpr (General) {
      const float b = a.bias ? a.bias[e] : 0.0f;
      sh.l[r][i] = x;
      sh.b[r][i] = b;
      c = a.bias ? fast_score(x) + b : x;
    }
    sh.row[r].key[i] = (uint64_t)order_key(c) << 32 | (uint32_t)~e;
  }
  wave_sync();
  for (int i = l; i < n; i += 2 * Lanes) {  // two candidates of a lane against all
    const int j = i + Lanes;
    const uint64_t me = sh.row[r].key[i], other = j < n ? sh.row[r].key[j] : 0;
    int rank = 0, other_rank = 0;
    for (int h = 0; h < n; h += kStep) {
#pragma unroll
      for (int q = 0; q < kStep; ++q) {
        const uint64_t o = sh.row[r].key[h + q];
        rank += o > me;
        other_rank += o > other;
      }
    }
    auto place = [&](int at, uint64_t k64, int to) {
      if (to < k) sh.sel[r][to] = {(int)~(uint32_t)k64, General ? sh.l[r][at] : key_value((uint32_t)(k64 >> 32))};
      if constexpr (General) sh.by_rank[r][to] = (uint8_t)at;
    };
    place(i, me, rank);
    if (j < n) place(j, other, other_rank);
  }
  if constexpr (General) {
    if (a.bias) {
      // neighbours in this order that are closer than fp32 tells and not equal in
      // all: of such a pair further apart some neighbours between are one too
      wave_sync();
      bool close = false;
      for (int i = l; i + 1 < n; i += Lanes) {
        const int u = sh.by_rank[r][i], w = sh.by_rank[r][i + 1];
        const float cu = key_value((uint32_t)(sh.row[r].key[u] >> 32)), cw = key_value((uint32_t)(sh.row[r].key[w] >> 32));
        close |= (cu - cw <= near + 0x1p-22f * fmaxf(fabsf(cu), fabsf(cw))) &
                 ((sh.l[r][u] != sh.l[r][w]) | (sh.b[r][u] != sh.b[r][w]));
      }
      if (__any(close && live)) {  // the candidates again, in fp64
        uint64_t* c64 = (uint64_t*)buffer + sub * kMaxCand;
        double m = 0.0, sum = 1.0;
        if (!a.sigmoid) {
          float top_l = -INFINITY;
#pragma unroll 1
          for (int e = l; e < E; e += Lanes) top_l = fmaxf(top_l, row[e]);
          m = row_max<Lanes>(top_l);
          sum = 0.0;
#pragma unroll 1
          for (int e = l; e < E; e += Lanes) sum += exp((double)row[e] - m);
#pragma unroll
          for (int d = Lanes / 2; d; d >>= 1) sum += __shfl_xor(sum, d, 64);
        }
#pragma unroll 1
        for (int i = l; i < n; i += Lanes) {
          const double x = sh.l[r][i];
          c64[i] = key64((a.sigmoid ? 1.0 / (1.0 + exp(-x)) : exp(x - m) / sum) + (double)sh.b[r][i]);
        }
        wave_sync();
#pragma unroll 1
        for (int i = l; i < n; i += Lanes) {
          const uint64_t me = c64[i];
          const uint32_t e = (uint32_t)sh.row[r].key[i];  // (its complement: the lower expert is the higher)
          int rank = 0;
          for (int h = 0; h < n; ++h) {
            const uint64_t o = c64[h];
            rank += (int)(o > me) | ((int)(o == me) & (int)((uint32_t)sh.row[r].key[h] > e));
          }
          if (rank < k) sh.sel[r][rank] = {(int)~e, sh.l[r][i]};
        }
      }
    }
  }
  const bool again = row_any<Lanes>(bad && live);
  const uint64_t rows_again = __ballot(again);
  if (rows_again) {
    wave_sync();
    for (int s = 0; s < kRows; ++s)
      if ((rows_again >> (s * Lanes)) & 1)
        route_row_exact(a.logits + (t0 + wave * kRows + s) * E, a.bias, E, k, a.sigmoid, a.groups, a.top_groups,
                        a.group_top, (uint64_t*)buffer, sh.sel[wave * kRows + s]);
  }
  wave_sync();

  // the weights: lane j of the row has slot j
  const Chosen slot = live && l < k ? sh.sel[r][l] : Chosen{-1, -INFINITY};
  const int e = slot.e;
  const bool has = e >= 0;
  const float lg = slot.l;
  float w, scale = a.scale;
  if (a.sigmoid) {
    w = has ? sigmoid_of(lg) : 0.0f;
    const float total = a.renorm ? row_sum<Lanes>(w) + kDenom : 1.0f;
    if (has && lg < 0.0f && tiny_exp(lg)) {
      w = half_exp(lg);
      scale *= w;
    }
    if (a.renorm) w = w / total;
  } else if (a.renorm) {
    // (a NaN has to reach the whole row; fmaxf leaves it out)
    const float top_l = row_max<Lanes>(lg);
    w = has ? expf(lg - top_l) : 0.0f;
    const float s = row_sum<Lanes>(w);
    w = has ? w / s : 0.0f;
  } else {
    w = has ? soft.exp_of(lg) * soft.inv : 0.0f;
  }
  if (active && l < k) {
    a.ids[t * k + l] = e;
    a.weights[t * k + l] = has ? scale * w : 0.0f;
    if (copy) copy[t * k + l] = e;
  }
  wave_sync();
}

// One pass of rows a workgroup, from row `first_row` on: in a loop the compiler
// keeps what does not depend on the row (biases, groups of the experts) in
// registers, twice as many as fit 4 waves a SIMD.
// [16384, 384] softmax, top 8: 9.2 us profiled (26 MB, 5.0 us at the rate of a copy):
// 146 vector instructions a row, 3.9 us of issue, beside the loads. Back to back in a
// graph (the logits then come from the cache) 6.3, sigmoid and a bias 10.8; [16384,
// 256] 8.0, in 8 groups 15.0: the groups' two passes through LDS. [4096, 256] in
// groups has two waves a SIMD and takes 7.3 us of latency (profiled: 10.0; with a row
// on the exact path 15.5).
template <int Lanes, int NV, bool Vec, bool General>
__global__ __launch_bounds__(kThreads) void route_scored_kernel(ScoredArgs a, int64_t first_row) {
  extern __shared__ __align__(16) float buffer[];
  __shared__ RouteShared<Lanes, General> sh;
  constexpr int kRows = kThreads / Lanes;
  if (a.sorted_ids && first_row == 0) {  // what the grouping kernel does not write
    const int64_t first = blockIdx.x * (int64_t)kThreads + threadIdx.x, step = gridDim.x * (int64_t)kThreads;
    for (int64_t i = first; i < a.cap; i += step) a.sorted_ids[i] = a.M * a.k;
    for (int64_t i = first; i < a.cap / a.block_m; i += step) a.block_expert[i] = -1;
  }
  route_rows<Lanes, NV, Vec, General>(a, first_row + (int64_t)blockIdx.x * kRows, sh, buffer, nullptr);
}

// Up to 16 rows: routing and grouping in one workgroup and one launch (two launches
// follow each other every 3.6 us). The grouping's tables take the dynamic LDS after
// the routing. One row of 384: 7.3 us profiled, the latency of one wave's steps.
template <int Lanes, int NV, bool Vec, bool General>
__global__ __launch_bounds__(kThreads) void route_scored_small_kernel(ScoredArgs a) {
  extern __shared__ __align__(16) float buffer[];
  __shared__ RouteShared<Lanes, General> sh;
  __shared__ int32_t ids[kSmallMaxAssign];
  constexpr int kRows = kThreads / Lanes;
  const int tid = threadIdx.x, MK = a.M * a.k;
  if constexpr (kRows >= kSmallMaxTokens) {
    route_rows<Lanes, NV, Vec, General>(a, 0, sh, buffer, ids);
  } else {
    for (int64_t t0 = 0; t0 < a.M; t0 += kRows) route_rows<Lanes, NV, Vec, General>(a, t0, sh, buffer, ids);
  }
  __syncthreads();
  SmallRoute& small = *(SmallRoute*)buffer;
  if (tid < MK) small.ids[tid] = ids[tid];  // (MK <= kThreads)
  if (tid < (a.E + 31) / 32) small.bits[tid] = 0u;
  const int nd = small_group<kThreads, true>(small, MK, a.E);
  const int bm = a.block_m;
  for (int64_t i = tid; i < a.cap; i += kThreads) {
    const int b = (int)(i / bm), p = (int)(i % bm);
    a.sorted_ids[i] = b < nd && p < kSmallMaxTokens ? small.blk_rows[b][p] : MK;
  }
  for (int64_t b = tid; b < a.cap / bm; b += kThreads) a.block_expert[b] = b < nd ? small.blk_e[b] : -1;
  for (int x = tid; x <= a.E; x += kThreads) a.offsets[x] = bm * (x < a.E ? small_rank(small, x) : nd);
  if (tid == 0) *a.npp = bm * nd;
}
static_assert(kSmallMaxAssign <= kThreads, "one id a thread");

// fn(Lanes, NV, Vec) for the row width. Few rows (kFewRows: below that 16 lanes a
// row are less than two waves a SIMD) take 32 lanes from 65 experts on: the work of
// a row is then done sooner (top 8, back to back in a graph: [64, 384] 4.3 us instead
// of 5.6, [4096, 256] in groups 7.3 instead of 8.0), while a full device takes longer
// ([16384, 384] softmax 8.5 instead of 6.5, with a bias 11.7 instead of 10.7). For top
// 16 the lowest of 16 lanes' maxima is a low threshold, and more than 64 candidates
// send many rows to the exact path: there 16 lanes take 49 us for [16384, 384]
// (67 with a bias), 32 lanes would take 10.5 (15.1).
constexpr int kFewRows = 8192;
template <typename F>
void by_width(int E, bool vec, bool few, F fn) {
  auto go = [&](auto lanes, auto nv) { vec ? fn(lanes, nv, std::true_type{}) : fn(lanes, nv, std::false_type{}); };
  auto row16 = [&](auto nv) { go(std::integral_constant<int, 16>{}, nv); };
  auto row32 = [&](auto nv) { go(std::integral_constant<int, 32>{}, nv); };
  if (E <= 64) row16(std::integral_constant<int, 1>{});
  else if (E > 512) row32(std::integral_constant<int, 8>{});
  else if (few && E <= 128) row32(std::integral_constant<int, 1>{});
  else if (few && E <= 256) row32(std::integral_constant<int, 2>{});
  else if (few && E <= 384) row32(std::integral_constant<int, 3>{});
  else if (few) row32(std::integral_constant<int, 4>{});
  else if (E <= 128) row16(std::integral_constant<int, 2>{});
  else if (E <= 256) row16(std::integral_constant<int, 4>{});
  else if (E <= 384) row16(std::integral_constant<int, 6>{});
  else row16(std::integral_constant<int, 8>{});
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

// ---- backward ---------------------------------------------------------------

// The slots' values lie in lanes 0..k of the row. Full (softmax over all
// experts): every logit has a gradient. Otherwise only the kept ones have;
// the rest of the row is grad_base or zeros, and is not touched in place.
// The slots' values reach the row's order through LDS.
// Bound by HBM: [16384, 384] full: calls of a program every 9.6 us for 51 MB
// (5.4 TB/s; 10.4 us profiled).
template <int Lanes, int NV, bool Vec, bool Full>
__global__ __launch_bounds__(kThreads) void route_scored_backward_kernel(ScoredBackwardArgs a, int64_t first_row) {
  extern __shared__ __align__(16) float buffer[];
  constexpr int N = 4 * NV, kRows = kThreads / Lanes;
  const int l = threadIdx.x % Lanes, r = threadIdx.x / Lanes;
  const int E = a.E, k = a.k, pitch = (E + 3) & ~3;
  float* mine = buffer + r * pitch;
  const bool in_place = a.base == a.grad;
  const int64_t t = first_row + (int64_t)blockIdx.x * kRows + r;
  const bool active = t < a.M;
  const float* row = a.logits + (active ? t : (int64_t)a.M - 1) * E;
  float v[N];
  if constexpr (Full) load_row<Lanes, NV, Vec>(row, E, l, v);
  // (unconditional loads go out together)
  const int64_t slot = (active ? t : (int64_t)a.M - 1) * k + (l < k ? l : 0);
  const int e0 = a.ids[slot];
  const float g0 = a.dweights[slot];
  const int e = active && l < k ? e0 : -1;
  const bool has = (unsigned)e < (unsigned)E;
  const float g = has ? a.scale * g0 : 0.0f;
  const float l0 = row[has ? e : 0];
  const float lg = has ? l0 : -INFINITY;
  const bool any = row_any<Lanes>(has);
  RowSoftmax soft{0.0f, 0.0f, 0.0f};
  float d;  // what goes to the slot's expert
  float dot = 0.0f;
  if constexpr (Full) {
    soft = row_softmax<Lanes>(v);
    dot = row_sum<Lanes>(has ? g * (soft.exp_of(lg) * soft.inv) : 0.0f);
    d = g;
  } else if (!a.sigmoid) {
    const float top = row_max<Lanes>(lg);
    const float x = has ? expf(lg - top) : 0.0f;
    const float s = row_sum<Lanes>(x);
    const float w = has ? x / s : 0.0f;
    d = w * (g - row_sum<Lanes>(g * w));
  } else {
    const float x = expf(-fabsf(lg)), y = 1.0f + x;
    const float s = has ? (lg >= 0.0f ? 1.0f : x) / y : 0.0f;
    float slope = has ? x / (y * y) : 0.0f, half = 1.0f;
    if (has && tiny_exp(lg)) slope = half = half_exp(lg);
    if (a.renorm) {
      const float total = row_sum<Lanes>(s) + kDenom;
      d = half * (slope / total * (g - row_sum<Lanes>(g * s / total)));
    } else {
      d = half * (slope * g);
    }
  }
  if (!Full && in_place) {
    if (has) a.grad[t * E + e] += d;
    return;
  }
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int c = 4 * Lanes * j + 4 * l;
    if (c < E) *(float4*)(mine + c) = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  }
  wave_sync();
  if (has) mine[e] = d;
  wave_sync();
  if (active) {
    const float* base = a.base ? a.base + t * E : nullptr;
    float* grad = a.grad + t * E;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = 4 * Lanes * j + 4 * l;
      float o[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        o[q] = c < E ? mine[c + q] : 0.0f;
        if constexpr (Full) o[q] = any ? soft.exp_of(v[4 * j + q]) * soft.inv * (o[q] - dot) : 0.0f;
      }
      if constexpr (Vec) {
        if (c < E) {
          float4 b = base ? *(const float4*)(base + c) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
          *(float4*)(grad + c) = make_float4(o[0] + b.x, o[1] + b.y, o[2] + b.z, o[3] + b.w);
        }
      } else {
#pragma unroll
        for (int q = 0; q < 4; ++q)
          if (c + q < E) grad[c + q] = o[q] + (base ? base[c + q] : 0.0f);
      }
    }
  }
}

// Workgroups of a launch: enough for the rows, at most 2^23 (a grid has fewer
// than 2^32 threads).
constexpr int kMaxGrid = 1 << 23;
unsigned grid_for(int64_t M, int rows) {
  const int64_t n = ceil_div(M, rows);
  return (unsigned)(n < kMaxGrid ? n : kMaxGrid);
}

}  // namespace

hipError_t launch_route_scored(const ScoredArgs& a, hipStream_t stream) {
  const bool grouping = a.sorted_ids != nullptr;
  const bool small = grouping && a.M <= kSmallMaxTokens;
  const bool general = a.bias || a.top_groups < a.groups;
  const bool vec = a.E % 4 == 0 && aligned16(a.logits) && (!a.bias || aligned16(a.bias));
  by_width(a.E, vec, a.M < kFewRows, [&](auto lanes, auto nv, auto v) {
    constexpr int L = decltype(lanes)::value, NV = decltype(nv)::value;
    constexpr bool V = decltype(v)::value;
    unsigned lds = (unsigned)row_buffer_bytes(L, a.bias != nullptr, a.top_groups < a.groups, a.E, a.groups) * kWaves;
    if (small && lds < sizeof(SmallRoute)) lds = sizeof(SmallRoute);
    constexpr int kRows = kThreads / L;
    if constexpr (L == 32 || NV == 1) {  // (up to 16 rows are few)
      if (small) {
        general ? route_scored_small_kernel<L, NV, V, true><<<1, kThreads, lds, stream>>>(a)
                : route_scored_small_kernel<L, NV, V, false><<<1, kThreads, lds, stream>>>(a);
        return;
      }
    }
    for (int64_t first = 0; first < a.M; first += (int64_t)kMaxGrid * kRows) {
      const unsigned grid = grid_for(a.M - first, kRows);
      general ? route_scored_kernel<L, NV, V, true><<<grid, kThreads, lds, stream>>>(a, first)
              : route_scored_kernel<L, NV, V, false><<<grid, kThreads, lds, stream>>>(a, first);
    }
  });
  const hipError_t err = hipGetLastError();
  if (err != hipSuccess || small || !grouping) return err;
  return launch_align(a.ids, a.M * a.k, a.E, a.block_m, a.sorted_ids, a.block_expert, a.offsets, a.npp, stream);
}

hipError_t launch_route_scored_backward(const ScoredBackwardArgs& a, hipStream_t stream) {
  const bool full = !a.sigmoid && !a.renorm;
  const bool vec = a.E % 4 == 0 && aligned16(a.logits) && aligned16(a.grad) && (!a.base || aligned16(a.base));
  by_width(a.E, vec, false, [&](auto lanes, auto nv, auto v) {
    constexpr int L = decltype(lanes)::value, NV = decltype(nv)::value;
    constexpr bool V = decltype(v)::value;
    const unsigned lds = (unsigned)(((a.E + 3) & ~3) * 4 * (kThreads / L));
    constexpr int kRows = kThreads / L;
    for (int64_t first = 0; first < a.M; first += (int64_t)kMaxGrid * kRows) {
      const unsigned grid = grid_for(a.M - first, kRows);
      full ? route_scored_backward_kernel<L, NV, V, true><<<grid, kThreads, lds, stream>>>(a, first)
           : route_scored_backward_kernel<L, NV, V, false><<<grid, kThreads, lds, stream>>>(a, first);
    }
  });
  return hipGetLastError();
}

}  // namespace moe
