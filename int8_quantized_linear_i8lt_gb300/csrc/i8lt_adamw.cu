// One AdamW step over many tensors, states in 32 bits or in 8 bits:
//   m = b1 m + (1 - b1) g,  v = b2 v + (1 - b2) g^2,
//   p = p (1 - lr wd) - size m / (sqrt(v) root + eps),
//   size = lr / (1 - b1^step), root = 1 / sqrt(1 - b2^step),
// where step is the number of updates that m and v have seen: the caller's, or
// a count per tensor on the device, which a skipped step does not raise.
// 8 bits: m and r = sqrt(v) are E4M3 codes in blocks of 256 elements with
// one fp32 absmax each (the block storage of the double-quantized 4-bit
// absmax).  r rather than v is stored: its block spans half the octaves, so
// the 2^18 between E4M3's largest and smallest value cover 2^36 of v; and a
// second moment above zero never takes the code of zero, which would leave
// eps alone in the denominator.
// Every state value is one chain of IEEE fp32 operations in the written
// order (no fused multiply-add), so its codes are the same on every run and
// follow from the formulas alone.
#include <cuda_fp8.h>

#include <algorithm>
#include <cmath>
#include <type_traits>

#include "i8lt.h"
#include "i8lt_internal.h"

namespace i8lt {
namespace {

constexpr int kBlockElems = 256;   // elements per absmax; every tensor's states start at a multiple of it
constexpr int kWarps = 8;
constexpr float kE4M3Max = 448.0f;
constexpr float kE4M3Min = 0x1p-9f;

struct Hyper {
  float b1, b2, c1, c2;      // the decays and 1 - decay
  float keep, size, root, eps;
  const float* grad_scale;   // optional device scalar: multiplies every gradient
  const float* found_inf;    // optional device scalar: a value other than 0 skips the step
};

// A tensor's updates so far, and the corrections of the one under way.
struct Count {
  int64_t updates;
  float size, root;
};

// A list of tensors travels in the kernel's parameters: no device copy whose
// host source would have to outlive the call.  kMaxTensors of them fit the
// 32764 bytes a launch may pass; the short list keeps the launch of a few
// tensors small.
template <int kCap>
struct TensorList {
  void* p[kCap];
  const void* g[kCap];
  int64_t n[kCap];
  int first[kCap + 1];       // first 256-element block of each tensor in this list's numbering
  int count;
  int64_t block0;            // the list's first block in the flat state
  int64_t tensor0;           // and its first tensor among the call's
};
constexpr int kFewTensors = 32;
constexpr int kMaxTensors = 1024;
static_assert(sizeof(TensorList<kMaxTensors>) + sizeof(Hyper) + 64 <= 32764, "kernel parameter space");

// The tensor that holds block `b` (of several with the same first block, the
// last: the others are empty).
template <int kCap>
__device__ __forceinline__ int find_tensor(const TensorList<kCap>& L, int b) {
  int lo = 0, hi = L.count;   // first[lo] <= b < first[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (L.first[mid] <= b) lo = mid;
    else hi = mid;
  }
  return lo;
}

// The larger of two values; a NaN wins (fmaxf drops it, and a block with a NaN
// would keep a finite absmax).
__device__ __forceinline__ float max_or_nan(float a, float b) {
  float m;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(m) : "f"(a), "f"(b));
  return m;
}
// Maximum over the warp of values >= 0: their bits are ordered like integers
// (a NaN above all).
__device__ __forceinline__ float warp_max(float v) {
  return __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(v)));
}

// N consecutive elements as fp32: 16-byte accesses when `whole` (they exist
// and start on min(16, their size) bytes), else the first `valid` one by one.
template <typename T, int N>
struct alignas(N * sizeof(T) < 16 ? N * sizeof(T) : 16) Run {
  T v[N];
};
template <typename T, int N>
__device__ __forceinline__ Run<T, N> load_run(const T* p, bool whole, int valid) {
  Run<T, N> r;
  if (whole) {
    r = *reinterpret_cast<const Run<T, N>*>(p);
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) r.v[i] = i < valid ? p[i] : from_float<T>(0.f);
  }
  return r;
}
template <typename T, int N>
__device__ __forceinline__ void widen(const Run<T, N>& r, float (&f)[N]) {
#pragma unroll
  for (int i = 0; i < N; i += 2) {
    if constexpr (sizeof(T) == 4) {
      f[i] = r.v[i];
      f[i + 1] = r.v[i + 1];
    } else {
      const uint32_t u = *reinterpret_cast<const uint32_t*>(r.v + i);
      if constexpr (std::is_same<T, __half>::value) {
        const float2 q = __half22float2(*reinterpret_cast<const __half2*>(&u));
        f[i] = q.x;
        f[i + 1] = q.y;
      } else {
        f[i] = __uint_as_float(u << 16);
        f[i + 1] = __uint_as_float(u & 0xffff0000u);
      }
    }
  }
}
template <typename T, int N>
__device__ __forceinline__ void store_run(T* p, bool whole, int valid, const float (&f)[N]) {
  Run<T, N> r;
#pragma unroll
  for (int i = 0; i < N; i += 2) {
    if constexpr (sizeof(T) == 4) {
      r.v[i] = f[i];
      r.v[i + 1] = f[i + 1];
    } else if constexpr (std::is_same<T, __half>::value) {
      *reinterpret_cast<__half2*>(r.v + i) = __floats2half2_rn(f[i], f[i + 1]);
    } else {
      *reinterpret_cast<__nv_bfloat162*>(r.v + i) = __floats2bfloat162_rn(f[i], f[i + 1]);
    }
  }
  if (whole) {
    *reinterpret_cast<Run<T, N>*>(p) = r;
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (i < valid) p[i] = r.v[i];
  }
}
template <typename T, int N>
__device__ __forceinline__ bool aligned_run(const T* p) {
  return (reinterpret_cast<uintptr_t>(p) & (alignof(Run<T, N>) - 1)) == 0;
}

// 8 E4M3 codes to their values (exact in fp16) and back (nearest even).
__device__ __forceinline__ void decode8(uint2 c, float d, float (&f)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t w = i < 2 ? c.x : c.y;
    const __half2 h(__nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(w >> (16 * (i & 1))), __NV_E4M3));
    const float2 v = __half22float2(h);
    f[2 * i] = __fmul_rn(v.x, d);
    f[2 * i + 1] = __fmul_rn(v.y, d);
  }
}
__device__ __forceinline__ uint2 encode8(const float (&f)[8]) {
  uint32_t q[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    q[i] = __nv_cvt_float2_to_fp8x2(make_float2(f[2 * i], f[2 * i + 1]), __NV_SATFINITE, __NV_E4M3);
  return make_uint2(q[0] | (q[1] << 16), q[2] | (q[3] << 16));
}

// 448 / absmax as the product with the rounded reciprocal.  A block whose
// absmax is below 2^-100 gets the codes of zeros: its reciprocal could
// overflow, and such values do not move a parameter.
__device__ __forceinline__ float code_scale(float top) {
  return top >= 0x1p-100f ? __fmul_rn(kE4M3Max, __frcp_rn(top)) : 0.f;
}

// The moments after this step's gradient, then the parameter, whose division
// is a product with the hardware's reciprocal (1 ulp; the update is a small
// part of the parameter).
__device__ __forceinline__ void moments(const Hyper& h, float g, float& m, float& v) {
  m = __fadd_rn(__fmul_rn(m, h.b1), __fmul_rn(g, h.c1));
  v = __fadd_rn(__fmul_rn(v, h.b2), __fmul_rn(__fmul_rn(g, g), h.c2));
}
__device__ __forceinline__ float updated(const Hyper& h, float size, float root, float p, float m, float r) {
  float inv;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(fmaf(r, root, h.eps)));
  return fmaf(-(m * size), inv, p * h.keep);
}

// One more update of the tensors with a gradient: its number and corrections,
// by the host's formulas.  In a kernel of its own, so that a block of 256
// elements reads two floats instead of computing two powers; 2 us.
template <int kCap>
__global__ void __launch_bounds__(128) adamw_count_kernel(const __grid_constant__ TensorList<kCap> L, double lr,
                                                          double beta1, double beta2, const float* found_inf,
                                                          Count* counts) {
  const int t = blockIdx.x * 128 + threadIdx.x;
  if (t >= L.count || L.g[t] == nullptr) return;
  if (found_inf != nullptr && *found_inf != 0.f) return;
  Count& c = counts[L.tensor0 + t];
  const int64_t n = c.updates + 1;
  c = Count{n, static_cast<float>(lr / (1.0 - pow(beta1, static_cast<double>(n)))),
            static_cast<float>(1.0 / sqrt(1.0 - pow(beta2, static_cast<double>(n))))};
}

// The blocks [b, end) of a list, tensor by tensor: f(t, p, g, left, blocks,
// state) with the tensor, the run's first block, its elements left in the
// tensor and its place in the flat state.  Tensors without a gradient are left
// out.
template <int kCap, typename P, typename G, typename F>
__device__ __forceinline__ void each_run(const TensorList<kCap>& L, int b, int end, F f) {
  for (int t = find_tensor(L, b); b < end; ++t) {
    const int stop = min(end, L.first[t + 1]);
    if (stop <= b) continue;
    const int64_t e0 = static_cast<int64_t>(b - L.first[t]) * kBlockElems;
    if (L.g[t] != nullptr)
      f(t, static_cast<P*>(L.p[t]) + e0, static_cast<const G*>(L.g[t]) + e0, L.n[t] - e0, stop - b, L.block0 + b);
    b = stop;
  }
}

// 32-bit states.  One warp per block of 256 elements, lane l on the elements
// 4 l .. 4 l + 3 and 128 more on: every access of a warp is one run of
// memory.  A warp takes `per_warp` blocks in turn, so that the search for its
// tensor is paid once.  Bound by HBM: 16 bytes of states, and the parameter
// and gradient, read or written once.  90 million f32 parameters: 364 us,
// 6.9 TB/s.
template <int kCap, typename P, typename G, bool kCounted>
__global__ void __launch_bounds__(kWarps * 32) adamw_kernel(const __grid_constant__ TensorList<kCap> L,
                                                            const __grid_constant__ Hyper h, float* mv, float* rv,
                                                            const Count* counts, int per_warp) {
  const int lane = threadIdx.x & 31;
  const int b = (blockIdx.x * kWarps + (threadIdx.x >> 5)) * per_warp;
  const int end = min(b + per_warp, L.first[L.count]);
  if (b >= end) return;
  if (h.found_inf != nullptr && *h.found_inf != 0.f) return;
  const float gs = h.grad_scale != nullptr ? *h.grad_scale : 1.f;
  each_run<kCap, P, G>(L, b, end, [&](int t, P* p, const G* g, int64_t left, int blocks, int64_t state) {
    const bool pa = aligned_run<P, 4>(p), ga = aligned_run<G, 4>(g);
    const float size = kCounted ? counts[L.tensor0 + t].size : h.size;
    const float root = kCounted ? counts[L.tensor0 + t].root : h.root;
    float *ms = mv + state * kBlockElems, *vs = rv + state * kBlockElems;
    for (; blocks > 0; --blocks, p += kBlockElems, g += kBlockElems, ms += kBlockElems, vs += kBlockElems,
                       left -= kBlockElems) {
      const int valid = static_cast<int>(min(left, static_cast<int64_t>(kBlockElems)));
      float gv[2][4], pv[2][4], m[2][4], v[2][4];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int e = 4 * (lane + 32 * i);
        const bool in = e + 4 <= valid;
        widen(load_run<G, 4>(g + e, ga && in, valid - e), gv[i]);
        widen(load_run<P, 4>(p + e, pa && in, valid - e), pv[i]);
        *reinterpret_cast<float4*>(m[i]) = *reinterpret_cast<const float4*>(ms + e);
        *reinterpret_cast<float4*>(v[i]) = *reinterpret_cast<const float4*>(vs + e);
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int e = 4 * (lane + 32 * i);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          moments(h, __fmul_rn(gv[i][k], gs), m[i][k], v[i][k]);
          pv[i][k] = updated(h, size, root, pv[i][k], m[i][k], sqrtf(v[i][k]));
        }
        store_run<P, 4>(p + e, pa && e + 4 <= valid, valid - e, pv[i]);
        *reinterpret_cast<float4*>(ms + e) = *reinterpret_cast<const float4*>(m[i]);
        *reinterpret_cast<float4*>(vs + e) = *reinterpret_cast<const float4*>(v[i]);
      }
    }
  });
}

// 8-bit states.  One warp per block, lane l on the elements 8 l .. 8 l + 7:
// the block's two absmax are reductions over the warp's registers.  With 4
// bytes of states per element the arithmetic weighs as much as HBM: two
// blocks are loaded before either is worked on, and the codes of zero are
// behind a branch that a block without them does not take.  90 million f16
// parameters: 186 us, 4.9 TB/s, with neither HBM nor issue saturated: 64
// registers a thread, and spills.
template <int kCap, typename P, typename G, bool kCounted>
__global__ void __launch_bounds__(kWarps * 32, 4) adamw8_kernel(const __grid_constant__ TensorList<kCap> L,
                                                                const __grid_constant__ Hyper h, uint8_t* mv,
                                                                uint8_t* rv, float* m_top, float* r_top,
                                                                const Count* counts, int per_warp) {
  const int lane = threadIdx.x & 31;
  const int b = (blockIdx.x * kWarps + (threadIdx.x >> 5)) * per_warp;
  const int end = min(b + per_warp, L.first[L.count]);
  if (b >= end) return;
  if (h.found_inf != nullptr && *h.found_inf != 0.f) return;
  const bool scaled = h.grad_scale != nullptr;
  const float gs = scaled ? *h.grad_scale : 1.f;
  struct Loaded {
    Run<G, 8> g;
    Run<P, 8> p;
    uint2 m, r;
    float mt, rt;
  };
  each_run<kCap, P, G>(L, b, end, [&](int t, P* p, const G* g, int64_t left, int blocks, int64_t state) {
    const bool pa = aligned_run<P, 8>(p), ga = aligned_run<G, 8>(g);
    const float size = kCounted ? counts[L.tensor0 + t].size : h.size;
    const float root = kCounted ? counts[L.tensor0 + t].root : h.root;
    p += 8 * lane;
    g += 8 * lane;
    // this lane's elements from here to the tensor's end
    int rest = static_cast<int>(min(left, static_cast<int64_t>(1) << 30)) - 8 * lane;
    uint8_t *ms = mv + state * kBlockElems + 8 * lane, *rs = rv + state * kBlockElems + 8 * lane;
    float *mt = m_top + state, *rt = r_top + state;
    // whole: every access is of 8 aligned elements
    auto fetch = [&](auto whole, int i, Loaded& x) {
      const int valid = whole ? 8 : min(rest - i * kBlockElems, 8);
      x.g = load_run<G, 8>(g + i * kBlockElems, whole || (ga && valid == 8), valid);
      x.p = load_run<P, 8>(p + i * kBlockElems, whole || (pa && valid == 8), valid);
      x.m = *reinterpret_cast<const uint2*>(ms + i * kBlockElems);
      x.r = *reinterpret_cast<const uint2*>(rs + i * kBlockElems);
      x.mt = mt[i];
      x.rt = rt[i];
    };
    auto work = [&](auto whole, int i, const Loaded& x) {
      float gv[8], pv[8], m[8], v[8];
      widen(x.g, gv);
      widen(x.p, pv);
      decode8(x.m, __fmul_rn(x.mt, 1.0f / kE4M3Max), m);
      decode8(x.r, __fmul_rn(x.rt, 1.0f / kE4M3Max), v);
      if (scaled)
#pragma unroll
        for (int k = 0; k < 8; ++k) gv[k] = __fmul_rn(gv[k], gs);
      const int valid = whole ? 8 : min(rest - i * kBlockElems, 8);
      float low = INFINITY, mtop = 0.f, vtop = 0.f;
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        v[k] = __fmul_rn(v[k], v[k]);
        moments(h, gv[k], m[k], v[k]);
        if (!whole && k >= valid) m[k] = v[k] = 0.f;   // past the tensor's end, whatever its codes were
        low = fminf(low, v[k]);
        mtop = max_or_nan(mtop, fabsf(m[k]));
      }
      const bool ordinary = low > 0.f;   // no second moment of zero
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        v[k] = __fsqrt_rn(v[k]);
        vtop = max_or_nan(vtop, v[k]);
        pv[k] = updated(h, size, root, pv[k], m[k], v[k]);
      }
      store_run<P, 8>(p + i * kBlockElems, whole || (pa && valid == 8), valid, pv);
      mtop = warp_max(mtop);
      vtop = warp_max(vtop);
      // even lanes work out m's scale, odd lanes r's
      const float top = lane & 1 ? vtop : mtop, scale = code_scale(top);
      const float mscale = __shfl_sync(0xffffffffu, scale, 0), rscale = __shfl_sync(0xffffffffu, scale, 1);
      if (lane < 2) (lane == 0 ? mt : rt)[i] = top;
#pragma unroll
      for (int k = 0; k < 8; ++k) m[k] = __fmul_rn(m[k], mscale);
      if (ordinary) {
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] = max_or_nan(__fmul_rn(v[k], rscale), kE4M3Min);
      } else {
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] = v[k] == 0.f ? 0.f : max_or_nan(__fmul_rn(v[k], rscale), kE4M3Min);
      }
      *reinterpret_cast<uint2*>(ms + i * kBlockElems) = encode8(m);
      *reinterpret_cast<uint2*>(rs + i * kBlockElems) = encode8(v);
    };
    auto run = [&](auto whole) {
      for (; blocks > 0; blocks -= 2) {
        Loaded x, z;
        fetch(whole, 0, x);
        if (blocks > 1) fetch(whole, 1, z);
        work(whole, 0, x);
        if (blocks > 1) work(whole, 1, z);
        p += 2 * kBlockElems;
        g += 2 * kBlockElems;
        ms += 2 * kBlockElems;
        rs += 2 * kBlockElems;
        mt += 2;
        rt += 2;
        rest -= 2 * kBlockElems;
      }
    };
    if (pa && ga && left >= static_cast<int64_t>(blocks) * kBlockElems) run(std::true_type());
    else run(std::false_type());
  });
}

// What all lists of a call share.
struct Call {
  Hyper h;
  double lr, beta1, beta2;
  Count* counts;             // or NULL: h's corrections for every tensor
  void *m, *r;
  float *m_top, *r_top;
  cudaStream_t s;
};

template <int kCap, typename P, typename G, bool k8, bool kCounted>
cudaError_t launch_kernel(const TensorList<kCap>& L, const Call& c) {
  const int blocks = L.first[L.count];
  // more blocks per warp only when every SM still gets several rounds of warps
  const int per_warp = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(k8 ? 8 : 4, blocks / (152 * 64))));
  const unsigned grid = static_cast<unsigned>(ceil_div(blocks, kWarps * per_warp));
  ProfScope ps(K_ADAMW, c.s);
  if constexpr (k8)
    adamw8_kernel<kCap, P, G, kCounted><<<grid, kWarps * 32, 0, c.s>>>(
        L, c.h, static_cast<uint8_t*>(c.m), static_cast<uint8_t*>(c.r), c.m_top, c.r_top, c.counts, per_warp);
  else
    adamw_kernel<kCap, P, G, kCounted>
        <<<grid, kWarps * 32, 0, c.s>>>(L, c.h, static_cast<float*>(c.m), static_cast<float*>(c.r), c.counts, per_warp);
  return cudaGetLastError();
}

template <int kCap, typename P, typename G, bool k8>
cudaError_t launch_list(const TensorList<kCap>& L, const Call& c) {
  if (L.first[L.count] == 0) return cudaSuccess;
  if (c.counts == nullptr) return launch_kernel<kCap, P, G, k8, false>(L, c);
  {
    ProfScope ps(K_ADAMW, c.s);
    adamw_count_kernel<kCap><<<static_cast<unsigned>(ceil_div(L.count, 128)), 128, 0, c.s>>>(
        L, c.lr, c.beta1, c.beta2, c.h.found_inf, c.counts);
    if (cudaError_t e = cudaGetLastError()) return e;
  }
  return launch_kernel<kCap, P, G, k8, true>(L, c);
}

// The tensors in lists of kCap; a list also ends before its blocks pass 2^30.
template <int kCap, typename P, typename G, bool k8>
cudaError_t run_lists(void* const* params, const void* const* grads, const int64_t* sizes, int64_t count,
                      const Call& c) {
  TensorList<kCap> L;
  L.count = 0;
  L.first[0] = 0;
  L.block0 = L.tensor0 = 0;
  for (int64_t i = 0; i < count; ++i) {
    const int64_t blocks = ceil_div(sizes[i], kBlockElems);
    if (L.count == kCap || L.first[L.count] + blocks > (int64_t(1) << 30)) {
      if (cudaError_t e = launch_list<kCap, P, G, k8>(L, c)) return e;
      L.block0 += L.first[L.count];
      L.tensor0 = i;
      L.count = 0;
    }
    L.p[L.count] = params[i];
    L.g[L.count] = grads[i];
    L.n[L.count] = sizes[i];
    L.first[L.count + 1] = L.first[L.count] + static_cast<int>(blocks);
    ++L.count;
  }
  return launch_list<kCap, P, G, k8>(L, c);
}

template <typename P, typename G, bool k8>
cudaError_t run_sized(void* const* params, const void* const* grads, const int64_t* sizes, int64_t count,
                      const Call& c) {
  if (count <= kFewTensors) return run_lists<kFewTensors, P, G, k8>(params, grads, sizes, count, c);
  return run_lists<kMaxTensors, P, G, k8>(params, grads, sizes, count, c);
}

template <typename P, bool k8>
cudaError_t run_grad(int gt, void* const* params, const void* const* grads, const int64_t* sizes, int64_t count,
                     const Call& c) {
  if (gt == DT_F16) return run_sized<P, __half, k8>(params, grads, sizes, count, c);
  if (gt == DT_BF16) return run_sized<P, __nv_bfloat16, k8>(params, grads, sizes, count, c);
  return run_sized<P, float, k8>(params, grads, sizes, count, c);
}

// counts NULL: update number `step` of every tensor.
template <bool k8>
int adamw(void* const* params, int pt, const void* const* grads, int gt, const int64_t* sizes, int64_t count,
          void* m, float* mt, void* r, float* rt, int64_t step, void* counts, double lr, double beta1, double beta2,
          double eps, double weight_decay, const float* grad_scale, const float* found_inf, void* stream) {
  if (!valid_dt(pt) || !valid_dt(gt)) return I8LT_ERR_UNSUPPORTED_DTYPE;
  if (count < 0 || step < 1) return I8LT_ERR_INVALID_ARG;
  if (!(beta1 >= 0.0 && beta1 < 1.0) || !(beta2 >= 0.0 && beta2 < 1.0) || !(eps >= 0.0)) return I8LT_ERR_INVALID_ARG;
  if (!std::isfinite(lr) || !std::isfinite(weight_decay) || !std::isfinite(eps)) return I8LT_ERR_INVALID_ARG;
  if (count > 0 && (params == nullptr || grads == nullptr || sizes == nullptr)) return I8LT_ERR_INVALID_ARG;
  int64_t total = 0;
  for (int64_t i = 0; i < count; ++i) {
    if (sizes[i] < 0 || sizes[i] > (int64_t(1) << 37)) return I8LT_ERR_INVALID_ARG;
    if (sizes[i] > 0 && params[i] == nullptr) return I8LT_ERR_INVALID_ARG;
    const uintptr_t pa = reinterpret_cast<uintptr_t>(params[i]), ga = reinterpret_cast<uintptr_t>(grads[i]);
    if ((pa & (pt == DT_F32 ? 3u : 1u)) != 0 || (ga & (gt == DT_F32 ? 3u : 1u)) != 0) return I8LT_ERR_MISALIGNED;
    total += sizes[i];
  }
  if (total == 0) return I8LT_OK;
  if (m == nullptr || r == nullptr || (k8 && (mt == nullptr || rt == nullptr))) return I8LT_ERR_INVALID_ARG;
  if (!aligned16(m) || !aligned16(r) || !aligned16(counts)) return I8LT_ERR_MISALIGNED;
  if (int d = check_device()) return d;
  Call c;
  c.h.b1 = static_cast<float>(beta1);
  c.h.b2 = static_cast<float>(beta2);
  c.h.c1 = static_cast<float>(1.0 - beta1);
  c.h.c2 = static_cast<float>(1.0 - beta2);
  c.h.keep = static_cast<float>(1.0 - lr * weight_decay);
  c.h.size = static_cast<float>(lr / (1.0 - std::pow(beta1, static_cast<double>(step))));
  c.h.root = static_cast<float>(1.0 / std::sqrt(1.0 - std::pow(beta2, static_cast<double>(step))));
  c.h.eps = static_cast<float>(eps);
  c.h.grad_scale = grad_scale;
  c.h.found_inf = found_inf;
  c.lr = lr;
  c.beta1 = beta1;
  c.beta2 = beta2;
  c.counts = static_cast<Count*>(counts);
  c.m = m;
  c.r = r;
  c.m_top = mt;
  c.r_top = rt;
  c.s = static_cast<cudaStream_t>(stream);
  if (pt == DT_F16) return cuda_status(run_grad<__half, k8>(gt, params, grads, sizes, count, c));
  if (pt == DT_BF16) return cuda_status(run_grad<__nv_bfloat16, k8>(gt, params, grads, sizes, count, c));
  return cuda_status(run_grad<float, k8>(gt, params, grads, sizes, count, c));
}

}  // namespace
}  // namespace i8lt

extern "C" {

int i8lt_adamw_step(void* const* params, int pt, const void* const* grads, int gt, const int64_t* sizes,
                    int64_t count, float* m, float* v, int64_t step, double lr, double beta1, double beta2, double eps,
                    double weight_decay, const float* grad_scale, const float* found_inf, void* stream) {
  return i8lt::adamw<false>(params, pt, grads, gt, sizes, count, m, nullptr, v, nullptr, step, nullptr, lr, beta1,
                            beta2, eps, weight_decay, grad_scale, found_inf, stream);
}

int i8lt_adamw_step_8bit(void* const* params, int pt, const void* const* grads, int gt, const int64_t* sizes,
                         int64_t count, uint8_t* m, float* m_absmax, uint8_t* r, float* r_absmax, int64_t step,
                         double lr, double beta1, double beta2, double eps, double weight_decay,
                         const float* grad_scale, const float* found_inf, void* stream) {
  return i8lt::adamw<true>(params, pt, grads, gt, sizes, count, m, m_absmax, r, r_absmax, step, nullptr, lr, beta1,
                           beta2, eps, weight_decay, grad_scale, found_inf, stream);
}

int i8lt_adamw_step_counted(void* const* params, int pt, const void* const* grads, int gt, const int64_t* sizes,
                            int64_t count, float* m, float* v, int64_t* counts, double lr, double beta1, double beta2,
                            double eps, double weight_decay, const float* grad_scale, const float* found_inf,
                            void* stream) {
  if (count > 0 && counts == nullptr) return I8LT_ERR_INVALID_ARG;
  return i8lt::adamw<false>(params, pt, grads, gt, sizes, count, m, nullptr, v, nullptr, 1, counts, lr, beta1, beta2,
                            eps, weight_decay, grad_scale, found_inf, stream);
}

int i8lt_adamw_step_8bit_counted(void* const* params, int pt, const void* const* grads, int gt, const int64_t* sizes,
                                 int64_t count, uint8_t* m, float* m_absmax, uint8_t* r, float* r_absmax,
                                 int64_t* counts, double lr, double beta1, double beta2, double eps,
                                 double weight_decay, const float* grad_scale, const float* found_inf, void* stream) {
  if (count > 0 && counts == nullptr) return I8LT_ERR_INVALID_ARG;
  return i8lt::adamw<true>(params, pt, grads, gt, sizes, count, m, m_absmax, r, r_absmax, 1, counts, lr, beta1, beta2,
                           eps, weight_decay, grad_scale, found_inf, stream);
}

}  // extern "C"
