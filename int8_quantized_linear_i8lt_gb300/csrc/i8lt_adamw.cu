// One AdamW step over many tensors, states in 32 bits or in 8 bits:
//   m = b1 m + (1 - b1) g,  v = b2 v + (1 - b2) g^2,
//   p = p (1 - lr wd) - size m / (sqrt(v) root + eps),
//   size = lr / (1 - b1^step), root = 1 / sqrt(1 - b2^step).
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

#include <cmath>

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
};
constexpr int kFewTensors = 32;
constexpr int kMaxTensors = 1024;
static_assert(sizeof(TensorList<kMaxTensors>) + sizeof(Hyper) + 64 <= 32764, "kernel parameter space");

// The tensor that holds block `b`: the last one whose first block is <= b
// and that is not empty.
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

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

// 4 consecutive elements: one access when `whole` (they exist and are aligned
// to their size together), else the first `valid` one by one.
template <typename T>
__device__ __forceinline__ void load4(const T* p, bool whole, int valid, float (&f)[4]) {
  if (whole) {
    if constexpr (sizeof(T) == 4) {
      *reinterpret_cast<float4*>(f) = *reinterpret_cast<const float4*>(p);
    } else {
      const uint2 u = *reinterpret_cast<const uint2*>(p);
      const T* q = reinterpret_cast<const T*>(&u);
#pragma unroll
      for (int i = 0; i < 4; ++i) f[i] = to_float(q[i]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = i < valid ? to_float(p[i]) : 0.f;
  }
}
__device__ __forceinline__ uint32_t pack16(float lo, float hi, __half*) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint32_t pack16(float lo, float hi, __nv_bfloat16*) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
template <typename T>
__device__ __forceinline__ void store4(T* p, bool whole, int valid, const float (&f)[4]) {
  if (whole) {
    if constexpr (sizeof(T) == 4)
      *reinterpret_cast<float4*>(p) = make_float4(f[0], f[1], f[2], f[3]);
    else
      *reinterpret_cast<uint2*>(p) = make_uint2(pack16(f[0], f[1], p), pack16(f[2], f[3], p));
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i < valid) p[i] = from_float<T>(f[i]);
  }
}

// 4 E4M3 codes to their values (exact in fp16) and back (nearest even).
__device__ __forceinline__ void decode4(uint32_t c, float d, float (&f)[4]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const __half2 h(__nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(c >> (16 * i)), __NV_E4M3));
    const float2 v = __half22float2(h);
    f[2 * i] = __fmul_rn(v.x, d);
    f[2 * i + 1] = __fmul_rn(v.y, d);
  }
}
__device__ __forceinline__ uint32_t encode4(const float (&f)[4]) {
  const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(f[0], f[1]), __NV_SATFINITE, __NV_E4M3);
  const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(f[2], f[3]), __NV_SATFINITE, __NV_E4M3);
  return lo | (hi << 16);
}

// 448 / absmax as the product with the rounded reciprocal.  A block whose
// absmax is below 2^-100 gets the codes of zeros: its reciprocal could
// overflow, and such values do not move a parameter.
__device__ __forceinline__ float code_scale(float top) {
  return top >= 0x1p-100f ? __fmul_rn(kE4M3Max, __frcp_rn(top)) : 0.f;
}

// The moments after this step's gradient, then the parameter.  The
// parameter's division is the fast one (2 ulp of the update).
__device__ __forceinline__ void moments(const Hyper& h, float g, float& m, float& v) {
  m = __fadd_rn(__fmul_rn(m, h.b1), __fmul_rn(g, h.c1));
  v = __fadd_rn(__fmul_rn(v, h.b2), __fmul_rn(__fmul_rn(g, g), h.c2));
}
__device__ __forceinline__ float updated(const Hyper& h, float p, float m, float r) {
  return fmaf(p, h.keep, -__fdividef(m * h.size, fmaf(r, h.root, h.eps)));
}

// One warp per block of 256 elements, lane l on the elements 4 l .. 4 l + 3
// and 128 more on: every access of a warp is one run of memory, and the
// block's absmax is a reduction over the warp's registers.  A warp takes
// kPerWarp blocks in turn, so that the search for its tensor is paid once.
// Bound by HBM: the tensors and states are read and written once.
constexpr int kPerWarp = 4;
template <int kCap, typename P, typename G, bool k8>
__global__ void __launch_bounds__(kWarps * 32) adamw_kernel(const __grid_constant__ TensorList<kCap> L,
                                                            const __grid_constant__ Hyper h, void* mv, void* rv,
                                                            float* m_top, float* r_top) {
  const int lane = threadIdx.x & 31;
  int b = (blockIdx.x * kWarps + (threadIdx.x >> 5)) * kPerWarp;
  const int end = min(b + kPerWarp, L.first[L.count]);
  if (b >= end) return;
  if (h.found_inf != nullptr && *h.found_inf != 0.f) return;
  const float gs = h.grad_scale != nullptr ? *h.grad_scale : 1.f;
  int t = find_tensor(L, b);
  for (; b < end; ++b) {
    while (b >= L.first[t + 1]) ++t;
    const G* g = static_cast<const G*>(L.g[t]);
    if (g == nullptr) continue;   // no gradient: the tensor and its states stay
    const int64_t e0 = static_cast<int64_t>(b - L.first[t]) * kBlockElems;
    const int valid = static_cast<int>(min(L.n[t] - e0, static_cast<int64_t>(kBlockElems)));
    P* p = static_cast<P*>(L.p[t]) + e0;
    g += e0;
    const bool pw = (reinterpret_cast<uintptr_t>(p) & (4 * sizeof(P) - 1)) == 0;
    const bool gw = (reinterpret_cast<uintptr_t>(g) & (4 * sizeof(G) - 1)) == 0;
    const int64_t sb = L.block0 + b, s0 = sb * kBlockElems;
    float gv[2][4], pv[2][4], m[2][4], v[2][4];
    const float md = k8 ? __fmul_rn(m_top[sb], 1.0f / kE4M3Max) : 0.f;
    const float rd = k8 ? __fmul_rn(r_top[sb], 1.0f / kE4M3Max) : 0.f;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int e = 4 * (lane + 32 * i);
      load4(g + e, gw && e + 4 <= valid, valid - e, gv[i]);
      load4(p + e, pw && e + 4 <= valid, valid - e, pv[i]);
      if constexpr (k8) {
        decode4(*reinterpret_cast<const uint32_t*>(static_cast<const uint8_t*>(mv) + s0 + e), md, m[i]);
        decode4(*reinterpret_cast<const uint32_t*>(static_cast<const uint8_t*>(rv) + s0 + e), rd, v[i]);
      } else {
        *reinterpret_cast<float4*>(m[i]) = *reinterpret_cast<const float4*>(static_cast<const float*>(mv) + s0 + e);
        *reinterpret_cast<float4*>(v[i]) = *reinterpret_cast<const float4*>(static_cast<const float*>(rv) + s0 + e);
      }
    }
    float mt = 0.f, rt = 0.f;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int e = 4 * (lane + 32 * i);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if constexpr (k8) v[i][k] = __fmul_rn(v[i][k], v[i][k]);
        moments(h, __fmul_rn(gv[i][k], gs), m[i][k], v[i][k]);
        const float r = __fsqrt_rn(v[i][k]);
        pv[i][k] = updated(h, pv[i][k], m[i][k], r);
        if constexpr (k8) {
          v[i][k] = r;
          mt = fmaxf(mt, fabsf(m[i][k]));
          rt = fmaxf(rt, r);
        }
      }
      store4(p + e, pw && e + 4 <= valid, valid - e, pv[i]);
      if constexpr (!k8) {
        *reinterpret_cast<float4*>(static_cast<float*>(mv) + s0 + e) = *reinterpret_cast<const float4*>(m[i]);
        *reinterpret_cast<float4*>(static_cast<float*>(rv) + s0 + e) = *reinterpret_cast<const float4*>(v[i]);
      }
    }
    if constexpr (k8) {
      mt = warp_max(mt);
      rt = warp_max(rt);
      const float ms = code_scale(mt), rs = code_scale(rt);
      if (lane == 0) {
        m_top[sb] = mt;
        r_top[sb] = rt;
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int e = 4 * (lane + 32 * i);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          m[i][k] = __fmul_rn(m[i][k], ms);
          const float y = __fmul_rn(v[i][k], rs);
          v[i][k] = v[i][k] > 0.f ? fmaxf(y, kE4M3Min) : y;
        }
        *reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(mv) + s0 + e) = encode4(m[i]);
        *reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(rv) + s0 + e) = encode4(v[i]);
      }
    }
  }
}

template <int kCap, typename P, typename G, bool k8>
cudaError_t launch_list(const TensorList<kCap>& L, const Hyper& h, void* m, void* r, float* mt, float* rt,
                        cudaStream_t s) {
  const int blocks = L.first[L.count];
  if (blocks == 0) return cudaSuccess;
  ProfScope ps(K_ADAMW, s);
  adamw_kernel<kCap, P, G, k8><<<static_cast<unsigned>(ceil_div(blocks, kWarps * kPerWarp)), kWarps * 32, 0, s>>>(L, h, m, r, mt,
                                                                                                      rt);
  return cudaGetLastError();
}

// The tensors in lists of kCap; a list also ends before its blocks pass 2^30.
template <int kCap, typename P, typename G, bool k8>
cudaError_t run_lists(void* const* params, const void* const* grads, const int64_t* sizes, int64_t count,
                      const Hyper& h, void* m, void* r, float* mt, float* rt, cudaStream_t s) {
  TensorList<kCap> L;
  L.count = 0;
  L.first[0] = 0;
  L.block0 = 0;
  for (int64_t i = 0; i < count; ++i) {
    const int64_t blocks = ceil_div(sizes[i], kBlockElems);
    if (blocks == 0) continue;
    if (L.count == kCap || L.first[L.count] + blocks > (int64_t(1) << 30)) {
      if (cudaError_t e = launch_list<kCap, P, G, k8>(L, h, m, r, mt, rt, s)) return e;
      L.block0 += L.first[L.count];
      L.count = 0;
    }
    L.p[L.count] = params[i];
    L.g[L.count] = grads[i];
    L.n[L.count] = sizes[i];
    L.first[L.count + 1] = L.first[L.count] + static_cast<int>(blocks);
    ++L.count;
  }
  return launch_list<kCap, P, G, k8>(L, h, m, r, mt, rt, s);
}

template <typename P, typename G, bool k8>
cudaError_t run_sized(void* const* params, const void* const* grads, const int64_t* sizes, int64_t count,
                      const Hyper& h, void* m, void* r, float* mt, float* rt, cudaStream_t s) {
  if (count <= kFewTensors) return run_lists<kFewTensors, P, G, k8>(params, grads, sizes, count, h, m, r, mt, rt, s);
  return run_lists<kMaxTensors, P, G, k8>(params, grads, sizes, count, h, m, r, mt, rt, s);
}

template <typename P, bool k8>
cudaError_t run_grad(int gt, void* const* params, const void* const* grads, const int64_t* sizes, int64_t count,
                     const Hyper& h, void* m, void* r, float* mt, float* rt, cudaStream_t s) {
  if (gt == DT_F16) return run_sized<P, __half, k8>(params, grads, sizes, count, h, m, r, mt, rt, s);
  if (gt == DT_BF16) return run_sized<P, __nv_bfloat16, k8>(params, grads, sizes, count, h, m, r, mt, rt, s);
  return run_sized<P, float, k8>(params, grads, sizes, count, h, m, r, mt, rt, s);
}

template <bool k8>
int adamw(void* const* params, int pt, const void* const* grads, int gt, const int64_t* sizes, int64_t count,
          void* m, float* mt, void* r, float* rt, int64_t step, double lr, double beta1, double beta2, double eps,
          double weight_decay, const float* grad_scale, const float* found_inf, void* stream) {
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
  if (!aligned16(m) || !aligned16(r)) return I8LT_ERR_MISALIGNED;
  if (int d = check_device()) return d;
  Hyper h;
  h.b1 = static_cast<float>(beta1);
  h.b2 = static_cast<float>(beta2);
  h.c1 = static_cast<float>(1.0 - beta1);
  h.c2 = static_cast<float>(1.0 - beta2);
  h.keep = static_cast<float>(1.0 - lr * weight_decay);
  h.size = static_cast<float>(lr / (1.0 - std::pow(beta1, static_cast<double>(step))));
  h.root = static_cast<float>(1.0 / std::sqrt(1.0 - std::pow(beta2, static_cast<double>(step))));
  h.eps = static_cast<float>(eps);
  h.grad_scale = grad_scale;
  h.found_inf = found_inf;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (pt == DT_F16) return cuda_status(run_grad<__half, k8>(gt, params, grads, sizes, count, h, m, r, mt, rt, s));
  if (pt == DT_BF16)
    return cuda_status(run_grad<__nv_bfloat16, k8>(gt, params, grads, sizes, count, h, m, r, mt, rt, s));
  return cuda_status(run_grad<float, k8>(gt, params, grads, sizes, count, h, m, r, mt, rt, s));
}

}  // namespace
}  // namespace i8lt

extern "C" {

int i8lt_adamw_step(void* const* params, int pt, const void* const* grads, int gt, const int64_t* sizes,
                    int64_t count, float* m, float* v, int64_t step, double lr, double beta1, double beta2, double eps,
                    double weight_decay, const float* grad_scale, const float* found_inf, void* stream) {
  return i8lt::adamw<false>(params, pt, grads, gt, sizes, count, m, nullptr, v, nullptr, step, lr, beta1, beta2, eps,
                            weight_decay, grad_scale, found_inf, stream);
}

int i8lt_adamw_step_8bit(void* const* params, int pt, const void* const* grads, int gt, const int64_t* sizes,
                         int64_t count, uint8_t* m, float* m_absmax, uint8_t* r, float* r_absmax, int64_t step,
                         double lr, double beta1, double beta2, double eps, double weight_decay,
                         const float* grad_scale, const float* found_inf, void* stream) {
  return i8lt::adamw<true>(params, pt, grads, gt, sizes, count, m, m_absmax, r, r_absmax, step, lr, beta1, beta2, eps,
                           weight_decay, grad_scale, found_inf, stream);
}

}  // extern "C"
