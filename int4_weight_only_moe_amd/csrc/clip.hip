// Global gradient norm over many tensors, and clipping by it.
//
//   sumsq = sum of g^2 over all elements (fp64);  out = g * min(1, max_norm / sqrt(sumsq))
//
// Both passes are bound by the tensors' traffic. The tensors of a launch are cut
// into units of 4096 elements (each tensor's last one may be short), workgroup b
// takes the units b, b + blocks, ...: the work is even however large the tensors
// are, and what is in flight lies together in memory (with a run of units a
// workgroup the squares of 705 MB took 157 us). Squares are summed in fp64: no
// gradient over- or underflows, and the conversions hide behind the loads.
#include "../../include/moe_w4a16.h"
#include "device_common.h"
#include "operators.h"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kPasses = 2;  // of 8 elements a thread
constexpr int kUnit = 8 * kThreads * kPasses;
constexpr int kTensors = kClipTensorsPerLaunch;

// The tensors of a launch, in its arguments. Few tensors have a small table: the
// host writes all of it for each launch.
constexpr int kFewTensors = 12;
template <int kN>
struct Table {
  const void* grad[kN];
  void* out[kN];
  int64_t size[kN];
  int64_t end[kN];  // units up to and including this tensor's
  uint8_t f32[kN];
  int n;
};

__device__ __forceinline__ double wave_sum64(double v) {
#pragma unroll
  for (int d = 32; d; d >>= 1) v += __shfl_xor(v, d, 64);
  return v;
}

__device__ __forceinline__ bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

// The first tensor that holds unit u or a later one.
template <int kN>
__device__ __forceinline__ int tensor_of(const Table<kN>& tab, int64_t u) {
  int lo = 0, hi = tab.n;
  while (lo < hi) {
    const int mid = (lo + hi) / 2;
    if (tab.end[mid] <= u) lo = mid + 1;
    else hi = mid;
  }
  return lo;
}

__device__ __forceinline__ void unpack8(uint4 p, float (&v)[8]) {
  const uint32_t u[4] = {p.x, p.y, p.z, p.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(u[i] << 16);
    v[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ uint16_t to_bf16(float v) { return __builtin_bit_cast(uint16_t, (__bf16)v); }

// The elements of a thread in a whole unit, as they lie in memory: in each pass 8,
// fp32 as two runs of 4, each instruction a contiguous 4 KB of the workgroup's.
struct Unit {
  uint4 v[2 * kPasses];
  __device__ __forceinline__ void load(const void* p, bool f32, int64_t first) {
    if (f32) {
      const uint4* q = (const uint4*)((const float*)p + first) + threadIdx.x;
#pragma unroll
      for (int j = 0; j < 2 * kPasses; ++j) v[j] = q[j * kThreads];
    } else {
      const uint4* q = (const uint4*)((const uint16_t*)p + first) + threadIdx.x;
#pragma unroll
      for (int j = 0; j < kPasses; ++j) v[j] = q[j * kThreads];
    }
  }
};
__device__ __forceinline__ void four(uint4 u, float (&o)[4]) {
  o[0] = __uint_as_float(u.x);
  o[1] = __uint_as_float(u.y);
  o[2] = __uint_as_float(u.z);
  o[3] = __uint_as_float(u.w);
}
__device__ __forceinline__ float load_one(const void* p, bool f32, int64_t i) {
  return f32 ? ((const float*)p)[i] : __uint_as_float((uint32_t)((const uint16_t*)p)[i] << 16);
}
__device__ __forceinline__ void store_one(void* p, bool f32, int64_t i, float v) {
  if (f32) ((float*)p)[i] = v;
  else ((uint16_t*)p)[i] = to_bf16(v);
}

// Workgroup b's units, with `blocks` of them, one after another: whole(i, first)
// for a unit of tensor i from element `first` on, part(i, first, last) for
// elements that are to be taken one by one. Back: from the last unit to the first.
template <bool kBack, int kN, typename Whole, typename Part>
__device__ __forceinline__ void walk(const Table<kN>& tab, int64_t b, int64_t blocks, Whole whole, Part part) {
  const int64_t units = tab.end[tab.n - 1];
  int i = kBack ? tab.n - 1 : 0;
  for (int64_t k = b; k < units; k += blocks) {
    const int64_t u = kBack ? units - 1 - k : k;
    if (kBack ? (i > 0 && tab.end[i - 1] > u) : tab.end[i] <= u) i = tensor_of(tab, u);
    const int64_t first = (u - (i ? tab.end[i - 1] : 0)) * kUnit;
    const int64_t size = tab.size[i];
    if (first + kUnit <= size && aligned16(tab.grad[i]) && aligned16(tab.out[i])) whole(i, first);
    else part(i, first, first + kUnit < size ? first + kUnit : size);
  }
}

// The sum of a workgroup's threads' values, in every thread.
template <int kWaves>
__device__ __forceinline__ double block_sum(double s, double (&room)[kWaves]) {
  s = wave_sum64(s);
  if ((threadIdx.x & 63) == 0) room[threadIdx.x >> 6] = s;
  __syncthreads();
  s = room[0];
#pragma unroll
  for (int w = 1; w < kWaves; ++w) s += room[w];
  return s;
}

// 176 M fp32 values in 48 tensors (705 MB): 117 us profiled (6.0 TB/s).
template <int kN>
__global__ __launch_bounds__(kThreads) void grad_sumsq_kernel(Table<kN> tab, double* parts, double* direct) {
  __shared__ double room[kThreads / 64];
  double s = 0.0;
  if (tab.n) {
    walk<false>(
        tab, blockIdx.x, gridDim.x,
        [&](int i, int64_t first) {
          const bool f32 = tab.f32[i];
          Unit unit;
          unit.load(tab.grad[i], f32, first);
          if (f32) {
#pragma unroll
            for (int j = 0; j < 2 * kPasses; ++j) {
              float v[4];
              four(unit.v[j], v);
#pragma unroll
              for (int q = 0; q < 4; ++q) s = fma((double)v[q], (double)v[q], s);
            }
          } else {
#pragma unroll
            for (int j = 0; j < kPasses; ++j) {
              float v[8];
              unpack8(unit.v[j], v);
#pragma unroll
              for (int q = 0; q < 8; ++q) s = fma((double)v[q], (double)v[q], s);
            }
          }
        },
        [&](int i, int64_t first, int64_t stop) {
          for (int64_t e = first + threadIdx.x; e < stop; e += kThreads) {
            const double v = load_one(tab.grad[i], tab.f32[i], e);
            s = fma(v, v, s);
          }
        });
  }
  s = block_sum(s, room);
  if (threadIdx.x == 0) {
    if (direct) *direct = s;
    else parts[blockIdx.x] = s;
  }
}

// The parts of all launches, in order.
constexpr int kJoinThreads = 1024;
__global__ __launch_bounds__(kJoinThreads) void grad_join_kernel(const double* parts, int64_t n, double* sumsq) {
  __shared__ double room[kJoinThreads / 64];
  double s = 0.0;
  for (int64_t i = threadIdx.x; i < n; i += kJoinThreads) s += parts[i];
  s = block_sum(s, room);
  if (threadIdx.x == 0) *sumsq = s;
}

// Results go around the cache: the gradients are then found there, and what reads
// the results next takes no longer (squares, clipping and a reader of 705 MB of
// results: 490 us, 518 with ordinary stores; of 88 MB 72 and 78; of 44 MB the same).
typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));
__device__ __forceinline__ void put(uint4* p, uint4 v) {
  __builtin_nontemporal_store(__builtin_bit_cast(u32x4_t, v), (u32x4_t*)p);
}

// The workgroups go through the tensors from the last to the first: what the
// pass over the squares read last is still in the cache. 705 MB read and written:
// 251 us profiled (5.6 TB/s); from the first to the last the two passes take 383 us, not 372.
//
// n_parts > 0: sumsq is still in that many parts, which every workgroup adds
// itself, in the same order: one launch less, and up to kJoinParts of them cost less
// than that.
template <int kN>
__global__ __launch_bounds__(kThreads) void grad_clip_kernel(Table<kN> tab, const double* parts, int n_parts,
                                                             double* sumsq, float max_norm, float* norm) {
  __shared__ double room[kThreads / 64];
  double total;
  if (n_parts > 0) {
    double s = 0.0;
#pragma unroll 8
    for (int i = threadIdx.x; i < n_parts; i += kThreads) s += parts[i];
    total = block_sum(s, room);
  } else {
    total = *sumsq;
  }
  const double root = sqrt(total);
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    if (norm) *norm = (float)root;
    if (n_parts > 0 && sumsq) *sumsq = total;
  }
  const bool over = root > (double)max_norm && root < INFINITY;
  // in fp64 where the factor may be too small for a normal fp32 number (down to
  // 2^-270 with results that are normal ones)
  const double ratio = over ? (double)max_norm / root : 1.0;
  const float factor = (float)ratio;
  const bool tiny = ratio < 0x1p-100;
  auto scaled = [&](float v) { return tiny ? (float)((double)v * ratio) : v * factor; };
  if (!tab.n) return;
  walk<true>(
      tab, blockIdx.x, gridDim.x,
      [&](int i, int64_t first) {
        if (!over && tab.grad[i] == tab.out[i]) return;
        const bool f32 = tab.f32[i];
        Unit unit;
        unit.load(tab.grad[i], f32, first);
        if (f32) {
          uint4* q = (uint4*)((float*)tab.out[i] + first) + threadIdx.x;
#pragma unroll
          for (int j = 0; j < 2 * kPasses; ++j) {
            float v[4];
            four(unit.v[j], v);
            put(q + j * kThreads, make_uint4(__float_as_uint(scaled(v[0])), __float_as_uint(scaled(v[1])),
                                             __float_as_uint(scaled(v[2])), __float_as_uint(scaled(v[3]))));
          }
        } else {
          uint4* q = (uint4*)((uint16_t*)tab.out[i] + first) + threadIdx.x;
#pragma unroll
          for (int j = 0; j < kPasses; ++j) {
            float v[8];
            unpack8(unit.v[j], v);
            uint32_t u[4];
#pragma unroll
            for (int k = 0; k < 4; ++k)
              u[k] = (uint32_t)to_bf16(scaled(v[2 * k])) | ((uint32_t)to_bf16(scaled(v[2 * k + 1])) << 16);
            put(q + j * kThreads, make_uint4(u[0], u[1], u[2], u[3]));
          }
        }
      },
      [&](int i, int64_t first, int64_t stop) {
        if (!over && tab.grad[i] == tab.out[i]) return;
        for (int64_t e = first + threadIdx.x; e < stop; e += kThreads)
          store_one(tab.out[i], tab.f32[i], e, scaled(load_one(tab.grad[i], tab.f32[i], e)));
      });
}

// fn(table, units) of the tensors [from, from + kTensors) of the call.
template <int kN, typename F>
void with_table_of(const ClipArgs& a, int64_t from, F fn) {
  Table<kN> tab;
  tab.n = 0;
  int64_t units = 0;
  for (int64_t i = from; i < a.n && i < from + kN; ++i) {
    const int k = tab.n++;
    tab.grad[k] = a.grads[i];
    tab.out[k] = a.outs ? a.outs[i] : const_cast<void*>(a.grads[i]);
    tab.size[k] = a.sizes[i];
    tab.f32[k] = a.dtypes[i] == MOE_DTYPE_F32;
    units += ceil_div(a.sizes[i], kUnit);
    tab.end[k] = units;
  }
  fn(tab, units);
}
template <typename F>
void with_table(const ClipArgs& a, int64_t from, F fn) {
  if (a.n - from <= kFewTensors) with_table_of<kFewTensors>(a, from, fn);
  else with_table_of<kTensors>(a, from, fn);
}

constexpr int64_t kJoinParts = 2 * kSumsqBlocks;

// Workgroups of a launch: a unit each, at most kSumsqBlocks (8 a CU).
unsigned blocks_for(int64_t units) { return (unsigned)(units < 1 ? 1 : units < kSumsqBlocks ? units : kSumsqBlocks); }

}  // namespace

// The squares of all tensors, in `parts` pieces; a call of one workgroup writes
// them to `direct` instead (if that is not null; 0 pieces).
static hipError_t launch_squares(const ClipArgs& a, double* direct, int64_t& parts, hipStream_t stream) {
  const int64_t launches = clip_launches(a.n);
  parts = 0;
  for (int64_t i = 0; i < (launches ? launches : 1); ++i) {
    bool only = false;
    with_table(a, i * kTensors, [&](const auto& tab, int64_t units) {
      const unsigned blocks = blocks_for(units);
      only = direct && launches <= 1 && blocks == 1;
      grad_sumsq_kernel<<<blocks, kThreads, 0, stream>>>(tab, a.parts + parts, only ? direct : nullptr);
      parts += only ? 0 : blocks;
    });
    const hipError_t err = hipGetLastError();
    if (err != hipSuccess || only) return err;
  }
  return hipSuccess;
}

static hipError_t launch_join(const double* parts, int64_t n, double* sumsq, hipStream_t stream) {
  grad_join_kernel<<<1, kJoinThreads, 0, stream>>>(parts, n, sumsq);
  return hipGetLastError();
}

static hipError_t launch_scale(const ClipArgs& a, int n_parts, hipStream_t stream) {
  const int64_t launches = clip_launches(a.n);
  for (int64_t i = (launches ? launches : 1) - 1; i >= 0; --i) {
    with_table(a, i * kTensors, [&](const auto& tab, int64_t units) {
      // (with parts, sumsq is written by one launch and read by none)
      grad_clip_kernel<<<blocks_for(units), kThreads, 0, stream>>>(
          tab, a.parts, n_parts, n_parts == 0 || i == 0 ? a.sumsq : nullptr, a.max_norm, i == 0 ? a.norm : nullptr);
    });
    const hipError_t err = hipGetLastError();
    if (err != hipSuccess) return err;
  }
  return hipSuccess;
}

hipError_t launch_grad_sumsq(const ClipArgs& a, hipStream_t stream) {
  int64_t parts;
  const hipError_t err = launch_squares(a, a.sumsq, parts, stream);
  return err != hipSuccess || parts == 0 ? err : launch_join(a.parts, parts, a.sumsq, stream);
}

hipError_t launch_grad_clip(const ClipArgs& a, hipStream_t stream) { return launch_scale(a, 0, stream); }

hipError_t launch_clip_grad_norm(const ClipArgs& a, hipStream_t stream) {
  int64_t parts;
  hipError_t err = launch_squares(a, nullptr, parts, stream);
  if (err != hipSuccess) return err;
  if (parts <= kJoinParts) return launch_scale(a, (int)parts, stream);
  ClipArgs joined = a;
  if (!joined.sumsq) joined.sumsq = a.parts + clip_parts(a.n);
  err = launch_join(a.parts, parts, joined.sumsq, stream);
  return err != hipSuccess ? err : launch_scale(joined, 0, stream);
}

}  // namespace moe
