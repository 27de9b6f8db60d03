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
constexpr int kPacks = 8;                          // 16-byte accesses of a thread and unit
constexpr int kUnitBytes = kThreads * kPacks * 16;
constexpr int kBlocks = 152 * 4;                   // at most, and so the partial sums of a call
constexpr int kCluster = 8, kSmallGroups = 2, kClusterUnits = 64;    // gradients of 2 MB in all: one cluster, one launch
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
        const int64_t at = head + static_cast<int64_t>(u - L.first[t]) * (kUnitBytes / static_cast<int>(sizeof(*base)));
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
__device__ __forceinline__ double squares(float x) { return static_cast<double>(x) * static_cast<double>(x); }

// The sum over the block, in thread 0 (elsewhere a part of it): every addition
// that another thread need not make is left out, fp64 runs at 2 a clock and SM.
template <int kWarps>
__device__ __forceinline__ double block_total(double sum, double* sums) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const double other = __shfl_down_sync(0xffffffffu, sum, o);
    if (lane < o) sum += other;
  }
  if (lane == 0) sums[threadIdx.x >> 5] = sum;
  __syncthreads();
  if (threadIdx.x == 0)
    for (int i = 1; i < kWarps; ++i) sum += sums[i];
  return sum;
}

// One block's part of the sum of squares, in thread 0: the units [from, to).
// A thread sums the squares of 32 elements of a unit in fp32 and those sums in
// fp64 (one fp64 addition for so many elements: the machine has few fp64
// units; 62 million bf16 values, 64 elements: 1 us less).  A sum so large or
// small that squares may have left fp32's range is taken again in fp64, unless
// all bits that were loaded are zeros.  Bound by HBM: 8 loads of 16 bytes a
// thread under way.  90 million f32 gradients: 58 us, 6.2 TB/s; 62 million bf16
// ones in 128 tensors 26 us, 4.8 TB/s, start and end of the launch included;
// zeros the same.
template <int kGroups, int kCap>
__device__ __forceinline__ double block_sum(const GradList<kCap>& L, int from, int to) {
  __shared__ double sums[kGroups * kThreads / 32];
  double sum = 0.0;
  // groups of kThreads threads take a part of the units each
  const int group = threadIdx.x / kThreads, thread = threadIdx.x % kThreads;
  const int u0 = from + (to - from) * group / kGroups, u1 = from + (to - from) * (group + 1) / kGroups;
  if (u0 < u1)
    each_unit(L, u0, u1, [&](auto* p, int64_t left, int64_t head) {
      using T = std::remove_pointer_t<decltype(p)>;
      constexpr int V = kPack<T>;
      if (thread < head) sum += squares(to_float(p[-1 - thread]));
      float s[4] = {0.f, 0.f, 0.f, 0.f};
      uint32_t any = 0;   // the bits of all elements, to tell zeros from squares that were lost
      auto add = [&](const Pack<T>& x) {
        const uint4 w = *reinterpret_cast<const uint4*>(&x);
        any |= w.x | w.y | w.z | w.w;
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const float f = to_float(x.v[i]);
          s[i & 3] = fmaf(f, f, s[i & 3]);
        }
      };
      // the sums of packs [j - kRun, j), 32 elements, to fp64
      constexpr int kRun = 32 / V;
      auto close = [&](int j) {
        const float all = (s[0] + s[1]) + (s[2] + s[3]);
        if (all >= 0x1p-80f && all <= 0x1p100f) {
          sum += all;
        } else if ((any & (sizeof(T) == 2 ? 0x7fff7fffu : 0x7fffffffu)) != 0) {
#pragma unroll 1
          for (int k = j - kRun; k < j; ++k) {
            const int e = (k * kThreads + thread) * V;
#pragma unroll
            for (int i = 0; i < V; ++i) {
              const float f = e + i < left ? to_float(p[e + i]) : 0.f;
              if (f != 0.f) sum += squares(f);
            }
          }
        }
        s[0] = s[1] = s[2] = s[3] = 0.f;
        any = 0;
      };
      const T* q = p + thread * V;
      if (left >= kUnitBytes / static_cast<int>(sizeof(T))) {
        Pack<T> x[kPacks];
#pragma unroll
        for (int j = 0; j < kPacks; ++j) x[j] = *reinterpret_cast<const Pack<T>*>(q + j * kThreads * V);
#pragma unroll
        for (int j = 0; j < kPacks; ++j) {
          add(x[j]);
          if ((j + 1) % kRun == 0) close(j + 1);
        }
      } else {
#pragma unroll 1
        for (int j = 0; j < kPacks; ++j) {
          const int e = (j * kThreads + thread) * V;
          if (e + V <= left) {
            add(*reinterpret_cast<const Pack<T>*>(p + e));
          } else {
            for (int i = e; i < left; ++i) {
              const float f = to_float(p[i]);
              any |= __float_as_uint(f);
              s[0] = fmaf(f, f, s[0]);
            }
          }
          if ((j + 1) % kRun == 0) close(j + 1);
        }
      }
    });
  return block_total<kGroups * kThreads / 32>(sum, sums);
}

struct Clip {
  const float *grad_scale, *found_inf;
  double max_norm;
  float* result;
};

// In fp64, each result rounded once: neither the norm without c nor c need keep
// the product inside fp32's range (1e39 times 2^-16).
__device__ __forceinline__ void write_result(const Clip& c, double s) {
  const float f = c.grad_scale != nullptr ? *c.grad_scale : 1.f;
  const bool found = c.found_inf != nullptr && *c.found_inf != 0.f;
  const double norm = __dmul_rn(fabs(static_cast<double>(f)), sqrt(s));
  const float norm32 = static_cast<float>(norm);
  const double q = isinf(norm32) ? 0.0 : c.max_norm / (norm + kClipEps);
  c.result[0] = norm32;
  c.result[1] = q >= 1.0 || isinf(c.max_norm) ? f : static_cast<float>(f * q);   // a NaN stays one
  c.result[2] = isfinite(norm32) && !found ? 0.f : 1.f;
}

template <int kCap>
__device__ __forceinline__ int unit_at(const GradList<kCap>& L, unsigned block) {
  return static_cast<int>(static_cast<int64_t>(L.first[L.count]) * block / gridDim.x);
}

template <int kCap>
__global__ void __launch_bounds__(kThreads, 4) grad_norm_kernel(const __grid_constant__ GradList<kCap> L,
                                                                double* partial, bool first) {
  grid_dependents_launch();
  const double s = block_sum<1>(L, unit_at(L, blockIdx.x), unit_at(L, blockIdx.x + 1));
  if (threadIdx.x == 0) partial[blockIdx.x] = first ? s : partial[blockIdx.x] + s;
}

__global__ void __launch_bounds__(kThreads) grad_norm_finish_kernel(const double* partial, int n, const Clip c) {
  grid_dependency_wait();
  __shared__ double sums[kThreads / 32];
  double sum = 0.0;
  for (int i = threadIdx.x; i < n; i += kThreads) sum += partial[i];
  sum = block_total<kThreads / 32>(sum, sums);
  if (threadIdx.x == 0) write_result(c, sum);
}

// Few gradients (1 MB: 11 us, two launches 9 and 4 us, but one launch less on
// the host, which bounds it): one cluster, whose first block adds up the others' sums from
// their shared memory.
__global__ void __cluster_dims__(kCluster, 1, 1) __launch_bounds__(kSmallGroups * kThreads)
    grad_norm_small_kernel(const __grid_constant__ GradList<kFewTensors> L, const Clip c) {
  __shared__ double part;
  const double s = block_sum<kSmallGroups>(L, unit_at(L, blockIdx.x), unit_at(L, blockIdx.x + 1));
  if (threadIdx.x == 0) part = s;
  cluster_sync();
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    double sum = 0.0;
    for (int k = 0; k < kCluster; ++k) {
      double v;
      asm volatile("ld.shared::cluster.f64 %0, [%1];" : "=d"(v) : "r"(mapa_shared(&part, static_cast<uint32_t>(k))) : "memory");
      sum += v;
    }
    write_result(c, sum);
  }
  cluster_sync();   // no block leaves before its sum has been read
}

// g *= scale, rounded once; nothing is read or written for a scale of 1.  62
// million bf16 gradients in 128 tensors of odd length: 41 us, 6.1 TB/s.
template <int kCap>
__global__ void __launch_bounds__(kThreads, 4) scale_grads_kernel(const __grid_constant__ GradList<kCap> L,
                                                               const float* scale) {
  const float c = *scale;
  if (c == 1.f) return;
  const int u0 = unit_at(L, blockIdx.x), u1 = unit_at(L, blockIdx.x + 1);
  if (u0 >= u1) return;
  each_unit(L, u0, u1, [&](auto* p, int64_t left, int64_t head) {
    using T = std::remove_pointer_t<decltype(p)>;
    constexpr int V = kPack<T>;
    if (threadIdx.x < head) {
      T* q = p - 1 - static_cast<int>(threadIdx.x);
      *q = from_float<T>(__fmul_rn(to_float(*q), c));
    }
    auto scaled = [c](Pack<T> x) {
#pragma unroll
      for (int i = 0; i < V; ++i) x.v[i] = from_float<T>(__fmul_rn(to_float(x.v[i]), c));
      return x;
    };
    T* q = p + static_cast<int>(threadIdx.x) * V;
    if (left >= kUnitBytes / static_cast<int>(sizeof(T))) {
      Pack<T> x[kPacks];
#pragma unroll
      for (int j = 0; j < kPacks; ++j) x[j] = *reinterpret_cast<const Pack<T>*>(q + j * kThreads * V);
#pragma unroll
      for (int j = 0; j < kPacks; ++j) *reinterpret_cast<Pack<T>*>(q + j * kThreads * V) = scaled(x[j]);
    } else {
#pragma unroll 1
      for (int e = static_cast<int>(threadIdx.x) * V; e < left; e += kThreads * V) {
        if (e + V <= left) {
          *reinterpret_cast<Pack<T>*>(p + e) = scaled(*reinterpret_cast<const Pack<T>*>(p + e));
        } else {
          for (int i = e; i < left; ++i) p[i] = from_float<T>(__fmul_rn(to_float(p[i]), c));
        }
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
    const int elem = elem_bytes(dtypes[i]);
    const int64_t body = sizes[i] - head_of(reinterpret_cast<uintptr_t>(grads[i]), elem, sizes[i]);
    const int64_t units = std::max<int64_t>(1, ceil_div(body * elem, kUnitBytes));
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

template <int kCap>
unsigned blocks_of(const GradList<kCap>& L) {
  return static_cast<unsigned>(std::min(L.first[L.count], kBlocks));
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
cudaError_t norm_lists(void* const* grads, const int32_t* dtypes, const int64_t* sizes, int64_t count, const Clip& c,
                       double* partial, cudaStream_t s) {
  unsigned used = 0;
  bool done = false;
  cudaError_t e = each_list<kCap>(grads, dtypes, sizes, count, [&](const GradList<kCap>& L) {
    if constexpr (kCap == kFewTensors) {
      if (L.first[L.count] <= kClusterUnits) {   // so it is the only list
        done = true;
        ProfScope ps(K_GRAD_NORM, s);
        grad_norm_small_kernel<<<kCluster, kSmallGroups * kThreads, 0, s>>>(L, c);
        return cudaGetLastError();
      }
    }
    // every list but the first adds to the sums of the same number of blocks
    const bool first = used == 0;
    if (first) used = count > kCap ? static_cast<unsigned>(kBlocks) : blocks_of(L);
    ProfScope ps(K_GRAD_NORM, s);
    grad_norm_kernel<kCap><<<used, kThreads, 0, s>>>(L, partial, first);
    return cudaGetLastError();
  });
  if (e != cudaSuccess || done) return e;
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
  return cudaLaunchKernelEx(&cfg, grad_norm_finish_kernel, static_cast<const double*>(partial), static_cast<int>(used), c);
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

size_t i8lt_grad_norm_workspace_size(void) { return kBlocks * sizeof(double); }

int i8lt_grad_norm(const void* const* grads, const int32_t* dtypes, const int64_t* sizes, int64_t count,
                   const float* grad_scale, const float* found_inf, double max_norm, float* result, void* ws,
                   size_t ws_bytes, void* stream) {
  void* const* g = const_cast<void* const*>(grads);
  if (int e = check_list(g, dtypes, sizes, count)) return e;
  if (!(max_norm >= 0.0) || result == nullptr) return ST_INVALID_ARG;
  if (ws == nullptr || ws_bytes < i8lt_grad_norm_workspace_size()) return ST_WORKSPACE;
  if ((reinterpret_cast<uintptr_t>(ws) & 255) != 0) return ST_MISALIGNED;
  for (const float* p : {static_cast<const float*>(result), grad_scale, found_inf})
    if ((reinterpret_cast<uintptr_t>(p) & 3) != 0) return ST_MISALIGNED;
  if (int d = check_device()) return d;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  double* partial = static_cast<double*>(ws);
  const Clip c{grad_scale, found_inf, max_norm, result};
  return cuda_status(count <= kFewTensors ? norm_lists<kFewTensors>(g, dtypes, sizes, count, c, partial, s)
                                          : norm_lists<kMaxTensors>(g, dtypes, sizes, count, c, partial, s));
}

int i8lt_scale_grads(void* const* grads, const int32_t* dtypes, const int64_t* sizes, int64_t count, const float* scale,
                     void* stream) {
  if (int e = check_list(grads, dtypes, sizes, count)) return e;
  if (scale == nullptr) return ST_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(scale) & 3) != 0) return ST_MISALIGNED;
  // one launch scales all of them at once: none may share memory with another
  try {
    std::vector<std::pair<uintptr_t, uintptr_t>> spans;
    spans.reserve(static_cast<size_t>(count) + 1);
    for (int64_t i = 0; i < count; ++i)
      if (grads[i] != nullptr && sizes[i] > 0) {
        const uintptr_t a = reinterpret_cast<uintptr_t>(grads[i]);
        spans.emplace_back(a, a + static_cast<uintptr_t>(sizes[i]) * static_cast<uintptr_t>(elem_bytes(dtypes[i])));
      }
    if (spans.empty()) return ST_OK;
    // nor with the scale, which some thread blocks would read before and some after its change
    spans.emplace_back(reinterpret_cast<uintptr_t>(scale), reinterpret_cast<uintptr_t>(scale) + sizeof(float));
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
