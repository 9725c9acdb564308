// Global gradient norm over many tensors, and clipping by it.
//
//   sumsq = sum of g^2 over all elements (fp64);  out = g * min(1, max_norm / sqrt(sumsq))
//
// Both passes are bound by the tensors' traffic. The tensors of a launch lie
// end to end in units of 2048 elements (each tensor's last unit may be short);
// every workgroup takes an equal run of units, so the work is even however
// large the tensors are. Squares are summed in fp64: no gradient over- or
// underflows, and the conversions hide behind the loads.
#include "../../include/moe_w4a16.h"
#include "device_common.h"
#include "operators.h"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kUnit = 8 * kThreads;
constexpr int kTensors = kClipTensorsPerLaunch;

struct Table {
  const void* grad[kTensors];
  void* out[kTensors];
  int64_t size[kTensors];
  int64_t end[kTensors];  // units up to and including this tensor's
  uint8_t f32[kTensors];
  int n;
};

__device__ __forceinline__ double wave_sum64(double v) {
#pragma unroll
  for (int d = 32; d; d >>= 1) v += __shfl_xor(v, d, 64);
  return v;
}

__device__ __forceinline__ bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

// The first tensor that holds unit u or a later one.
__device__ __forceinline__ int tensor_of(const Table& tab, int64_t u) {
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

// Eight elements of a thread in a whole unit. fp32: two runs of 4, each
// instruction a contiguous 4 KB of the workgroup's.
__device__ __forceinline__ void load_unit(const void* p, bool f32, int64_t first, float (&v)[8]) {
  const int tid = threadIdx.x;
  if (f32) {
    const float4* q = (const float4*)((const float*)p + first);
    const float4 a = q[tid], b = q[kThreads + tid];
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  } else {
    unpack8(((const uint4*)((const uint16_t*)p + first))[tid], v);
  }
}
__device__ __forceinline__ void store_unit(void* p, bool f32, int64_t first, const float (&v)[8]) {
  const int tid = threadIdx.x;
  if (f32) {
    float4* q = (float4*)((float*)p + first);
    q[tid] = make_float4(v[0], v[1], v[2], v[3]);
    q[kThreads + tid] = make_float4(v[4], v[5], v[6], v[7]);
  } else {
    uint32_t u[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) u[i] = (uint32_t)to_bf16(v[2 * i]) | ((uint32_t)to_bf16(v[2 * i + 1]) << 16);
    ((uint4*)((uint16_t*)p + first))[tid] = make_uint4(u[0], u[1], u[2], u[3]);
  }
}
__device__ __forceinline__ float load_one(const void* p, bool f32, int64_t i) {
  return f32 ? ((const float*)p)[i] : __uint_as_float((uint32_t)((const uint16_t*)p)[i] << 16);
}
__device__ __forceinline__ void store_one(void* p, bool f32, int64_t i, float v) {
  if (f32) ((float*)p)[i] = v;
  else ((uint16_t*)p)[i] = to_bf16(v);
}

// Workgroup b's run of the launch's units, one tensor after another: whole(i,
// first, count) for `count` whole units of tensor i from element `first` on,
// part(i, first, last) for elements that are to be taken one by one.
template <typename Whole, typename Part>
__device__ __forceinline__ void walk(const Table& tab, int64_t b, int64_t blocks, Whole whole, Part part) {
  const int64_t units = tab.end[tab.n - 1];
  int64_t u = units * b / blocks;
  const int64_t last = units * (b + 1) / blocks;
  for (int i = tensor_of(tab, u); u < last; ++i) {
    const int64_t start = i ? tab.end[i - 1] : 0;
    const int64_t to = tab.end[i] < last ? tab.end[i] : last;
    const int64_t first = (u - start) * kUnit;
    int64_t stop = (to - start) * kUnit;
    stop = stop < tab.size[i] ? stop : tab.size[i];
    const int64_t count = aligned16(tab.grad[i]) && aligned16(tab.out[i]) ? (stop - first) / kUnit : 0;
    if (count) whole(i, first, count);
    if (first + count * kUnit < stop) part(i, first + count * kUnit, stop);
    u = to;
  }
}

constexpr int kAhead = 4;  // units in flight

__global__ __launch_bounds__(kThreads) void grad_sumsq_kernel(Table tab, double* parts, double* direct) {
  __shared__ double room[kThreads / 64];
  double s = 0.0;
  auto add = [&](const float (&v)[8]) {
#pragma unroll
    for (int q = 0; q < 8; ++q) s = fma((double)v[q], (double)v[q], s);
  };
  if (tab.n) {
    walk(
        tab, blockIdx.x, gridDim.x,
        [&](int i, int64_t first, int64_t count) {
          const void* p = tab.grad[i];
          const bool f32 = tab.f32[i];
          int64_t c = 0;
          for (; c + kAhead <= count; c += kAhead) {
            float v[kAhead][8];
#pragma unroll
            for (int j = 0; j < kAhead; ++j) load_unit(p, f32, first + (c + j) * kUnit, v[j]);
#pragma unroll
            for (int j = 0; j < kAhead; ++j) add(v[j]);
          }
          for (; c < count; ++c) {
            float v[8];
            load_unit(p, f32, first + c * kUnit, v);
            add(v);
          }
        },
        [&](int i, int64_t first, int64_t stop) {
          for (int64_t e = first + threadIdx.x; e < stop; e += kThreads) {
            const double v = load_one(tab.grad[i], tab.f32[i], e);
            s = fma(v, v, s);
          }
        });
  }
  s = wave_sum64(s);
  if ((threadIdx.x & 63) == 0) room[threadIdx.x >> 6] = s;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int w = 1; w < kThreads / 64; ++w) s += room[w];
    if (direct) *direct = s;
    else parts[blockIdx.x] = s;
  }
  if (!direct && blockIdx.x == 0)  // the places of workgroups that this launch does not have
    for (int b = gridDim.x + threadIdx.x; b < kSumsqBlocks; b += kThreads) parts[b] = 0.0;
}

// The launches' parts, in order.
constexpr int kJoinThreads = 1024;
__global__ __launch_bounds__(kJoinThreads) void grad_join_kernel(const double* parts, int64_t n, double* sumsq) {
  __shared__ double room[kJoinThreads / 64];
  double s = 0.0;
  for (int64_t i = threadIdx.x; i < n; i += kJoinThreads) s += parts[i];
  s = wave_sum64(s);
  if ((threadIdx.x & 63) == 0) room[threadIdx.x >> 6] = s;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int w = 1; w < kJoinThreads / 64; ++w) s += room[w];
    *sumsq = s;
  }
}

// The workgroups go through the tensors from the last to the first: what the
// pass over the squares read last is still in the cache.
__global__ __launch_bounds__(kThreads) void grad_clip_kernel(Table tab, const double* sumsq, float max_norm,
                                                             float* norm) {
  const double total = *sumsq, root = sqrt(total);
  if (norm && blockIdx.x == 0 && threadIdx.x == 0) *norm = (float)root;
  const bool over = root > (double)max_norm && root < INFINITY;
  const float factor = over ? (float)((double)max_norm / root) : 1.0f;
  if (!tab.n) return;
  walk(
      tab, gridDim.x - 1 - blockIdx.x, gridDim.x,
      [&](int i, int64_t first, int64_t count) {
        const void* p = tab.grad[i];
        void* o = tab.out[i];
        const bool f32 = tab.f32[i];
        if (!over && p == o) return;
        int64_t c = 0;
        for (; c + kAhead <= count; c += kAhead) {
          float v[kAhead][8];
#pragma unroll
          for (int j = 0; j < kAhead; ++j) load_unit(p, f32, first + (c + j) * kUnit, v[j]);
#pragma unroll
          for (int j = 0; j < kAhead; ++j) {
#pragma unroll
            for (int q = 0; q < 8; ++q) v[j][q] *= factor;
            store_unit(o, f32, first + (c + j) * kUnit, v[j]);
          }
        }
        for (; c < count; ++c) {
          float v[8];
          load_unit(p, f32, first + c * kUnit, v);
#pragma unroll
          for (int q = 0; q < 8; ++q) v[q] *= factor;
          store_unit(o, f32, first + c * kUnit, v);
        }
      },
      [&](int i, int64_t first, int64_t stop) {
        if (!over && tab.grad[i] == tab.out[i]) return;
        for (int64_t e = first + threadIdx.x; e < stop; e += kThreads)
          store_one(tab.out[i], tab.f32[i], e, load_one(tab.grad[i], tab.f32[i], e) * factor);
      });
}

// The tensors [from, from + kTensors) of the call.
Table table_of(const ClipArgs& a, int64_t from, int64_t& units) {
  Table tab{};
  units = 0;
  for (int64_t i = from; i < a.n && i < from + kTensors; ++i) {
    const int k = tab.n++;
    tab.grad[k] = a.grads[i];
    tab.out[k] = a.outs ? a.outs[i] : const_cast<void*>(a.grads[i]);
    tab.size[k] = a.sizes[i];
    tab.f32[k] = a.dtypes[i] == MOE_DTYPE_F32;
    units += ceil_div(a.sizes[i], kUnit);
    tab.end[k] = units;
  }
  return tab;
}

// Workgroups of a launch: a unit each, at most kSumsqBlocks (8 a CU).
unsigned blocks_for(int64_t units) { return (unsigned)(units < 1 ? 1 : units < kSumsqBlocks ? units : kSumsqBlocks); }

}  // namespace

hipError_t launch_grad_sumsq(const ClipArgs& a, hipStream_t stream) {
  const int64_t launches = clip_launches(a.n);
  for (int64_t i = 0; i < (launches ? launches : 1); ++i) {
    int64_t units;
    const Table tab = table_of(a, i * kTensors, units);
    const unsigned blocks = blocks_for(units);
    const bool only = launches <= 1 && blocks == 1;
    grad_sumsq_kernel<<<blocks, kThreads, 0, stream>>>(tab, a.parts + i * kSumsqBlocks, only ? a.sumsq : nullptr);
    const hipError_t err = hipGetLastError();
    if (err != hipSuccess || only) return err;
  }
  grad_join_kernel<<<1, kJoinThreads, 0, stream>>>(a.parts, launches * kSumsqBlocks, a.sumsq);
  return hipGetLastError();
}

hipError_t launch_grad_clip(const ClipArgs& a, hipStream_t stream) {
  const int64_t launches = clip_launches(a.n);
  for (int64_t i = (launches ? launches : 1) - 1; i >= 0; --i) {
    int64_t units;
    const Table tab = table_of(a, i * kTensors, units);
    grad_clip_kernel<<<blocks_for(units), kThreads, 0, stream>>>(tab, a.sumsq, a.max_norm, i == 0 ? a.norm : nullptr);
    const hipError_t err = hipGetLastError();
    if (err != hipSuccess) return err;
  }
  return hipSuccess;
}

}  // namespace moe
