// The norm of all gradients of a step and the factor that clips it, and the
// scaling of gradients in place:
//   norm = |c| sqrt(sum g^2),  scale = c min(1, max_norm / (norm + 1e-6)),
// c a device scalar (1 / loss scale) or 1.  Both stay on the device, where the
// AdamW step takes them.
#include <algorithm>
#include <cmath>
#include <utility>
#include <vector>

#include "i8lt.h"
#include "i8lt_internal.h"

namespace i8lt {
namespace {

constexpr int kThreads = 256;
constexpr int kPerThread = 32;                     // elements of a unit that a thread has
constexpr int kUnit = kThreads * kPerThread;
constexpr int kMaxBlocks = 2048;                   // partial sums of a call
constexpr double kClipEps = 1e-6;

// A list of tensors travels in the kernel's parameters.  A tensor's first
// elements, up to a 16-byte boundary, belong to its first unit; units start on
// such boundaries.
template <int kCap>
struct GradList {
  void* g[kCap];
  int64_t n[kCap];
  int first[kCap + 1];       // first unit of each tensor
  int8_t dt[kCap];
  int count;
};
constexpr int kFewTensors = 32;
constexpr int kMaxTensors = 1024;
static_assert(sizeof(GradList<kMaxTensors>) + 64 <= 32764, "kernel parameter space");

int elem_bytes(int dt) { return dt == DT_F32 ? 4 : 2; }
__host__ __device__ inline int64_t head_of(uintptr_t p, int elem, int64_t n) {
  const int64_t h = static_cast<int64_t>((16 - (p & 15)) & 15) / elem;
  return h < n ? h : n;
}

template <int kCap>
__device__ __forceinline__ int find_tensor(const GradList<kCap>& L, int u) {
  int lo = 0, hi = L.count;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (L.first[mid] <= u) lo = mid;
    else hi = mid;
  }
  return lo;
}

// f(tag, p, left, head, unit) for the units [u, end) of the list: the unit's first
// element (16-byte aligned), the elements from there to the tensor's end, and
// the tensor's elements before that, for its first unit.
template <int kCap, typename F>
__device__ __forceinline__ void each_unit(const GradList<kCap>& L, int u, int end, F f) {
  for (int t = find_tensor(L, u); u < end; ++t) {
    const int stop = min(end, L.first[t + 1]);
    if (stop <= u) continue;
    auto run = [&](auto* base) {
      const int64_t head = head_of(reinterpret_cast<uintptr_t>(base), sizeof(*base), L.n[t]);
      for (; u < stop; ++u) {
        const int64_t at = head + static_cast<int64_t>(u - L.first[t]) * kUnit;
        f(base + at, L.n[t] - at, u == L.first[t] ? head : 0);
      }
    };
    if (L.dt[t] == DT_F16) run(static_cast<__half*>(L.g[t]));
    else if (L.dt[t] == DT_BF16) run(static_cast<__nv_bfloat16*>(L.g[t]));
    else run(static_cast<float*>(L.g[t]));
  }
}

template <typename T>
struct alignas(16) Pack {
  T v[16 / sizeof(T)];
};
template <typename T>
constexpr int kPack = 16 / sizeof(T);
template <typename T>
constexpr int kPacks = kPerThread / kPack<T>;     // 16-byte accesses of a thread and unit

__device__ __forceinline__ double squares(float x) { return static_cast<double>(x) * static_cast<double>(x); }

// One block's part of the sum of squares.  A thread sums the squares of its 32
// elements of a unit in fp32 and those sums in fp64 (one fp64 addition per 32
// elements: the machine has few fp64 units).  A sum so large or small that
// squares may have left fp32's range is taken again in fp64.
template <int kCap>
__global__ void __launch_bounds__(kThreads) grad_norm_kernel(const __grid_constant__ GradList<kCap> L, double* partial,
                                                             bool first) {
  grid_dependents_launch();
  __shared__ double sums[kThreads / 32];
  const int64_t units = L.first[L.count];
  const int u0 = static_cast<int>(units * blockIdx.x / gridDim.x), u1 = static_cast<int>(units * (blockIdx.x + 1) / gridDim.x);
  double sum = 0.0;
  if (u0 < u1)
    each_unit(L, u0, u1, [&](auto* p, int64_t left, int64_t head) {
      using T = std::remove_pointer_t<decltype(p)>;
      constexpr int V = kPack<T>;
      if (threadIdx.x < head) sum += squares(to_float(p[-1 - static_cast<int>(threadIdx.x)]));
      Pack<T> x[kPacks<T>];
#pragma unroll
      for (int j = 0; j < kPacks<T>; ++j) {
        const int e = (j * kThreads + static_cast<int>(threadIdx.x)) * V;
        if (e + V <= left) {
          x[j] = *reinterpret_cast<const Pack<T>*>(p + e);
        } else {
#pragma unroll
          for (int i = 0; i < V; ++i) x[j].v[i] = e + i < left ? p[e + i] : from_float<T>(0.f);
        }
      }
      float s[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int j = 0; j < kPacks<T>; ++j)
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const float f = to_float(x[j].v[i]);
          s[i & 3] = fmaf(f, f, s[i & 3]);
        }
      const float all = (s[0] + s[1]) + (s[2] + s[3]);
      if (all >= 0x1p-80f && all <= 0x1p100f) {
        sum += all;
      } else {
        double d = 0.0;
#pragma unroll
        for (int j = 0; j < kPacks<T>; ++j)
#pragma unroll
          for (int i = 0; i < V; ++i) {
            const float f = to_float(x[j].v[i]);
            if (f != 0.f) d += squares(f);
          }
        sum += d;
      }
    });
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if ((threadIdx.x & 31) == 0) sums[threadIdx.x >> 5] = sum;
  __syncthreads();
  if (threadIdx.x == 0) {
    double s = 0.0;
    for (int i = 0; i < kThreads / 32; ++i) s += sums[i];
    partial[blockIdx.x] = first ? s : partial[blockIdx.x] + s;
  }
}

__global__ void __launch_bounds__(kThreads) grad_norm_finish_kernel(const double* partial, int n, const float* grad_scale,
                                                                    const float* found_inf, double max_norm,
                                                                    float* result) {
  grid_dependency_wait();
  __shared__ double sums[kThreads / 32];
  double sum = 0.0;
  for (int i = threadIdx.x; i < n; i += kThreads) sum += partial[i];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if ((threadIdx.x & 31) == 0) sums[threadIdx.x >> 5] = sum;
  __syncthreads();
  if (threadIdx.x == 0) {
    double s = 0.0;
    for (int i = 0; i < kThreads / 32; ++i) s += sums[i];
    const double c = grad_scale != nullptr ? *grad_scale : 1.0;
    const double norm = fabs(c) * sqrt(s), q = max_norm / (norm + kClipEps);
    const float rounded = static_cast<float>(norm);
    result[0] = rounded;
    result[1] = static_cast<float>(q >= 1.0 || max_norm == INFINITY ? c : c * q);   // a NaN stays one
    result[2] = isfinite(rounded) && (found_inf == nullptr || *found_inf == 0.f) ? 0.f : 1.f;
  }
}

// g *= scale, rounded once; nothing is read or written for a scale of 1.
template <int kCap>
__global__ void __launch_bounds__(kThreads) scale_grads_kernel(const __grid_constant__ GradList<kCap> L,
                                                               const float* scale) {
  const float c = *scale;
  if (c == 1.f) return;
  const int64_t units = L.first[L.count];
  const int u0 = static_cast<int>(units * blockIdx.x / gridDim.x), u1 = static_cast<int>(units * (blockIdx.x + 1) / gridDim.x);
  if (u0 >= u1) return;
  each_unit(L, u0, u1, [&](auto* p, int64_t left, int64_t head) {
    using T = std::remove_pointer_t<decltype(p)>;
    constexpr int V = kPack<T>;
    if (threadIdx.x < head) {
      T* q = p - 1 - static_cast<int>(threadIdx.x);
      *q = from_float<T>(__fmul_rn(to_float(*q), c));
    }
    Pack<T> x[kPacks<T>];
#pragma unroll
    for (int j = 0; j < kPacks<T>; ++j) {
      const int e = (j * kThreads + static_cast<int>(threadIdx.x)) * V;
      if (e + V <= left) x[j] = *reinterpret_cast<const Pack<T>*>(p + e);
    }
#pragma unroll
    for (int j = 0; j < kPacks<T>; ++j) {
      const int e = (j * kThreads + static_cast<int>(threadIdx.x)) * V;
      if (e + V <= left) {
#pragma unroll
        for (int i = 0; i < V; ++i) x[j].v[i] = from_float<T>(__fmul_rn(to_float(x[j].v[i]), c));
        *reinterpret_cast<Pack<T>*>(p + e) = x[j];
      } else {
#pragma unroll
        for (int i = 0; i < V; ++i)
          if (e + i < left) p[e + i] = from_float<T>(__fmul_rn(to_float(p[e + i]), c));
      }
    }
  });
}

// The tensors in lists of kCap; a list also ends before its units pass 2^30.
template <int kCap, typename F>
cudaError_t each_list(void* const* grads, const int32_t* dtypes, const int64_t* sizes, int64_t count, F launch) {
  GradList<kCap> L;
  L.count = 0;
  L.first[0] = 0;
  for (int64_t i = 0; i < count; ++i) {
    if (sizes[i] == 0 || grads[i] == nullptr) continue;
    const int64_t body = sizes[i] - head_of(reinterpret_cast<uintptr_t>(grads[i]), elem_bytes(dtypes[i]), sizes[i]);
    const int64_t units = std::max<int64_t>(1, ceil_div(body, kUnit));
    if (L.count == kCap || L.first[L.count] + units > (int64_t(1) << 30)) {
      if (cudaError_t e = launch(L)) return e;
      L.count = 0;
    }
    L.g[L.count] = grads[i];
    L.n[L.count] = sizes[i];
    L.dt[L.count] = static_cast<int8_t>(dtypes[i]);
    L.first[L.count + 1] = L.first[L.count] + static_cast<int>(units);
    ++L.count;
  }
  return L.count > 0 ? launch(L) : cudaSuccess;
}

constexpr int kBlocksPerSm = 4;
template <int kCap>
unsigned blocks_of(const GradList<kCap>& L) {
  return static_cast<unsigned>(std::min(L.first[L.count], std::min(kMaxBlocks, 152 * kBlocksPerSm)));
}

int check_list(void* const* grads, const int32_t* dtypes, const int64_t* sizes, int64_t count) {
  if (count < 0) return ST_INVALID_ARG;
  if (count > 0 && (grads == nullptr || dtypes == nullptr || sizes == nullptr)) return ST_INVALID_ARG;
  for (int64_t i = 0; i < count; ++i) {
    if (!valid_dt(dtypes[i])) return ST_UNSUPPORTED_DTYPE;
    if (sizes[i] < 0 || sizes[i] > (int64_t(1) << 37)) return ST_INVALID_ARG;
    if ((reinterpret_cast<uintptr_t>(grads[i]) & (elem_bytes(dtypes[i]) - 1)) != 0) return ST_MISALIGNED;
  }
  return ST_OK;
}

template <int kCap>
cudaError_t norm_lists(void* const* grads, const int32_t* dtypes, const int64_t* sizes, int64_t count,
                       const float* grad_scale, const float* found_inf, double max_norm, float* result, double* partial,
                       cudaStream_t s) {
  unsigned used = 0;
  cudaError_t e = each_list<kCap>(grads, dtypes, sizes, count, [&](const GradList<kCap>& L) {
    // every list but the first adds to the sums of the same number of blocks
    const bool first = used == 0;
    if (first) used = count > kCap ? static_cast<unsigned>(152 * kBlocksPerSm) : blocks_of(L);
    ProfScope ps(K_GRAD_NORM, s);
    grad_norm_kernel<kCap><<<used, kThreads, 0, s>>>(L, partial, first);
    return cudaGetLastError();
  });
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(1);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = used > 0 ? 1 : 0;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  ProfScope ps(K_GRAD_NORM, s);
  return cudaLaunchKernelEx(&cfg, grad_norm_finish_kernel, static_cast<const double*>(partial), static_cast<int>(used),
                            grad_scale, found_inf, max_norm, result);
}

template <int kCap>
cudaError_t scale_lists(void* const* grads, const int32_t* dtypes, const int64_t* sizes, int64_t count,
                        const float* scale, cudaStream_t s) {
  return each_list<kCap>(grads, dtypes, sizes, count, [&](const GradList<kCap>& L) {
    ProfScope ps(K_SCALE_GRADS, s);
    scale_grads_kernel<kCap><<<blocks_of(L), kThreads, 0, s>>>(L, scale);
    return cudaGetLastError();
  });
}

}  // namespace
}  // namespace i8lt

extern "C" {

using namespace i8lt;

size_t i8lt_grad_norm_workspace_size(void) { return kMaxBlocks * sizeof(double); }

int i8lt_grad_norm(const void* const* grads, const int32_t* dtypes, const int64_t* sizes, int64_t count,
                   const float* grad_scale, const float* found_inf, double max_norm, float* result, void* ws,
                   size_t ws_bytes, void* stream) {
  void* const* g = const_cast<void* const*>(grads);
  if (int e = check_list(g, dtypes, sizes, count)) return e;
  if (!(max_norm >= 0.0) || result == nullptr) return ST_INVALID_ARG;
  if (ws == nullptr || ws_bytes < i8lt_grad_norm_workspace_size()) return ST_WORKSPACE;
  if ((reinterpret_cast<uintptr_t>(ws) & 255) != 0 || (reinterpret_cast<uintptr_t>(result) & 3) != 0) return ST_MISALIGNED;
  if (int d = check_device()) return d;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  double* partial = static_cast<double*>(ws);
  return cuda_status(count <= kFewTensors
                         ? norm_lists<kFewTensors>(g, dtypes, sizes, count, grad_scale, found_inf, max_norm, result, partial, s)
                         : norm_lists<kMaxTensors>(g, dtypes, sizes, count, grad_scale, found_inf, max_norm, result, partial, s));
}

int i8lt_scale_grads(void* const* grads, const int32_t* dtypes, const int64_t* sizes, int64_t count, const float* scale,
                     void* stream) {
  if (int e = check_list(grads, dtypes, sizes, count)) return e;
  if (scale == nullptr) return ST_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(scale) & 3) != 0) return ST_MISALIGNED;
  // one launch scales all of them at once: none may share memory with another
  try {
    std::vector<std::pair<uintptr_t, uintptr_t>> spans;
    spans.reserve(static_cast<size_t>(count));
    for (int64_t i = 0; i < count; ++i)
      if (grads[i] != nullptr && sizes[i] > 0) {
        const uintptr_t a = reinterpret_cast<uintptr_t>(grads[i]);
        spans.emplace_back(a, a + static_cast<uintptr_t>(sizes[i]) * static_cast<uintptr_t>(elem_bytes(dtypes[i])));
      }
    if (spans.empty()) return ST_OK;
    std::sort(spans.begin(), spans.end());
    for (size_t i = 1; i < spans.size(); ++i)
      if (spans[i - 1].second > spans[i].first) return ST_INVALID_ARG;
  } catch (...) {
    return ST_INVALID_ARG;
  }
  if (int d = check_device()) return d;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return cuda_status(count <= kFewTensors ? scale_lists<kFewTensors>(grads, dtypes, sizes, count, scale, s)
                                          : scale_lists<kMaxTensors>(grads, dtypes, sizes, count, scale, s));
}

}  // extern "C"
