// Layer norm over the last dimension, forward and backward:
//   mean = sum_n x / N, rstd = 1 / sqrt(sum_n (x - mean)^2 / N + eps),
//   h = (x - mean) * rstd, y = h * w + b;
//   gx = rstd * (g w - mean_n(g w) - h * mean_n(g w h)),
//   gw = sum_m g h, gb = sum_m g.
// Statistics and sums are fp32; each output is rounded once.
#include <algorithm>

#include "i8lt.h"
#include "i8lt_internal.h"

namespace i8lt {
namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ float load_any(const void* p, int dt, int64_t i) {
  if (dt == DT_F16) return to_float(static_cast<const __half*>(p)[i]);
  if (dt == DT_BF16) return to_float(static_cast<const __nv_bfloat16*>(p)[i]);
  return static_cast<const float*>(p)[i];
}
__device__ __forceinline__ void store_any(void* p, int dt, int64_t i, float v) {
  if (dt == DT_F16) static_cast<__half*>(p)[i] = from_float<__half>(v);
  else if (dt == DT_BF16) static_cast<__nv_bfloat16*>(p)[i] = from_float<__nv_bfloat16>(v);
  else static_cast<float*>(p)[i] = v;
}

// Sum over the block, the same value in every thread.
__device__ __forceinline__ float block_sum(float v, float* scratch) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) scratch[threadIdx.x >> 5] = v;
  __syncthreads();
  float t = 0.f;
#pragma unroll
  for (int i = 0; i < kThreads / 32; ++i) t += scratch[i];
  return t;
}

// One block per row; the row is read once per pass from L1 / L2.
template <typename T>
__global__ void __launch_bounds__(kThreads) norm_forward_kernel(const T* x, int64_t N, const void* w, const void* b,
                                                                int wt, float eps, T* y, float* mean, float* rstd) {
  __shared__ float scratch[kThreads / 32];
  const int64_t m = blockIdx.x;
  x += m * N;
  y += m * N;
  float s = 0.f;
  for (int64_t n = threadIdx.x; n < N; n += kThreads) s += to_float(x[n]);
  const float mu = block_sum(s, scratch) / static_cast<float>(N);
  s = 0.f;
  for (int64_t n = threadIdx.x; n < N; n += kThreads) {
    const float d = to_float(x[n]) - mu;
    s += d * d;
  }
  const float r = 1.0f / sqrtf(block_sum(s, scratch) / static_cast<float>(N) + eps);
  for (int64_t n = threadIdx.x; n < N; n += kThreads) {
    float v = (to_float(x[n]) - mu) * r;
    if (w != nullptr) v *= load_any(w, wt, n);
    if (b != nullptr) v += load_any(b, wt, n);
    y[n] = from_float<T>(v);
  }
  if (threadIdx.x == 0) {
    if (mean != nullptr) mean[m] = mu;
    if (rstd != nullptr) rstd[m] = r;
  }
}

template <typename T>
__global__ void __launch_bounds__(kThreads) norm_backward_kernel(const T* g, const T* x, int64_t N, const float* mean,
                                                                 const float* rstd, const void* w, int wt, T* gx) {
  __shared__ float scratch[kThreads / 32];
  const int64_t m = blockIdx.x;
  g += m * N;
  x += m * N;
  gx += m * N;
  const float mu = mean[m], r = rstd[m];
  float s1 = 0.f, s2 = 0.f;
  for (int64_t n = threadIdx.x; n < N; n += kThreads) {
    const float gw = to_float(g[n]) * (w != nullptr ? load_any(w, wt, n) : 1.f);
    s1 += gw;
    s2 += gw * ((to_float(x[n]) - mu) * r);
  }
  const float c1 = block_sum(s1, scratch) / static_cast<float>(N);
  const float c2 = block_sum(s2, scratch) / static_cast<float>(N);
  for (int64_t n = threadIdx.x; n < N; n += kThreads) {
    const float gw = to_float(g[n]) * (w != nullptr ? load_any(w, wt, n) : 1.f);
    gx[n] = from_float<T>(r * (gw - c1 - ((to_float(x[n]) - mu) * r) * c2));
  }
}

// partial[0][c][n], partial[1][c][n]: sums of g h and g over the rows of chunk c.
template <typename T>
__global__ void __launch_bounds__(kThreads) norm_grad_partial_kernel(const T* g, const T* x, int64_t M, int64_t N,
                                                                     const float* mean, const float* rstd,
                                                                     int64_t rows, float* partial) {
  const int64_t n = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
  if (n >= N) return;
  const int64_t c = blockIdx.y, m0 = c * rows, m1 = min(m0 + rows, M);
  float sw = 0.f, sb = 0.f;
  for (int64_t m = m0; m < m1; ++m) {
    const float gv = to_float(g[m * N + n]);
    sw += gv * ((to_float(x[m * N + n]) - mean[m]) * rstd[m]);
    sb += gv;
  }
  partial[c * N + n] = sw;
  partial[(gridDim.y + c) * N + n] = sb;
}

__global__ void __launch_bounds__(kThreads) norm_grad_sum_kernel(const float* partial, int chunks, int64_t N, int wt,
                                                                 void* gw, void* gb) {
  const int64_t n = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
  if (n >= N) return;
  float sw = 0.f, sb = 0.f;
  for (int64_t c = 0; c < chunks; ++c) {
    sw += partial[c * N + n];
    sb += partial[(chunks + c) * N + n];
  }
  if (gw != nullptr) store_any(gw, wt, n, sw);
  if (gb != nullptr) store_any(gb, wt, n, sb);
}

// Row chunks of the weight gradient's partial sums.
int grad_chunks(int64_t M) { return static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(ceil_div(M, 16), 152))); }

template <typename T>
cudaError_t forward(const void* x, int64_t M, int64_t N, const void* w, const void* b, int wt, float eps, void* y,
                    float* mean, float* rstd, cudaStream_t s) {
  ProfScope ps(K_LAYER_NORM, s);
  norm_forward_kernel<T><<<static_cast<unsigned>(M), kThreads, 0, s>>>(static_cast<const T*>(x), N, w, b, wt, eps,
                                                                      static_cast<T*>(y), mean, rstd);
  return cudaGetLastError();
}

template <typename T>
cudaError_t backward(const void* g, const void* x, int64_t M, int64_t N, const float* mean, const float* rstd,
                     const void* w, int wt, void* gx, void* gw, void* gb, float* partial, cudaStream_t s) {
  if (gx != nullptr) {
    ProfScope ps(K_LAYER_NORM_BWD, s);
    norm_backward_kernel<T><<<static_cast<unsigned>(M), kThreads, 0, s>>>(
        static_cast<const T*>(g), static_cast<const T*>(x), N, mean, rstd, w, wt, static_cast<T*>(gx));
    if (cudaError_t e = cudaGetLastError()) return e;
  }
  if (gw == nullptr && gb == nullptr) return cudaSuccess;
  const int chunks = grad_chunks(M);
  const unsigned cols = static_cast<unsigned>(ceil_div(N, kThreads));
  {
    ProfScope ps(K_LAYER_NORM_BWD, s);
    norm_grad_partial_kernel<T><<<dim3(cols, chunks), kThreads, 0, s>>>(static_cast<const T*>(g),
                                                                       static_cast<const T*>(x), M, N, mean, rstd,
                                                                       ceil_div(M, chunks), partial);
    if (cudaError_t e = cudaGetLastError()) return e;
  }
  ProfScope ps(K_LAYER_NORM_GRAD_SUM, s);
  norm_grad_sum_kernel<<<cols, kThreads, 0, s>>>(partial, chunks, N, wt, gw, gb);
  return cudaGetLastError();
}

}  // namespace
}  // namespace i8lt

using namespace i8lt;

extern "C" {

int i8lt_layer_norm_forward(const void* x, int xt, int64_t M, int64_t N, const void* w, const void* b, int wt,
                            float eps, void* y, float* mean, float* rstd, void* stream) {
  if (!valid_dt(xt) || ((w != nullptr || b != nullptr) && !valid_dt(wt))) return I8LT_ERR_UNSUPPORTED_DTYPE;
  if (M < 0 || N <= 0 || M > INT32_MAX / 2 || N > INT32_MAX / 2 || !(eps >= 0.0f)) return I8LT_ERR_INVALID_ARG;
  if (M == 0) return I8LT_OK;
  if (x == nullptr || y == nullptr) return I8LT_ERR_INVALID_ARG;
  if (!aligned16(x) || !aligned16(y) || !aligned16(w) || !aligned16(b)) return I8LT_ERR_MISALIGNED;
  if (int d = check_device()) return d;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (xt == DT_F16) return cuda_status(forward<__half>(x, M, N, w, b, wt, eps, y, mean, rstd, s));
  if (xt == DT_BF16) return cuda_status(forward<__nv_bfloat16>(x, M, N, w, b, wt, eps, y, mean, rstd, s));
  return cuda_status(forward<float>(x, M, N, w, b, wt, eps, y, mean, rstd, s));
}

size_t i8lt_layer_norm_backward_workspace_size(int64_t M, int64_t N) {
  if (M < 0 || N <= 0 || M > INT32_MAX / 2 || N > INT32_MAX / 2) return 0;
  return static_cast<size_t>(round_up(static_cast<int64_t>(grad_chunks(M)) * N * 8, 256));
}

int i8lt_layer_norm_backward(const void* g, const void* x, int xt, int64_t M, int64_t N, const float* mean,
                             const float* rstd, const void* w, int wt, void* gx, void* gw, void* gb, void* ws,
                             size_t ws_bytes, void* stream) {
  const bool grads = gw != nullptr || gb != nullptr;
  if (!valid_dt(xt) || ((w != nullptr || grads) && !valid_dt(wt))) return I8LT_ERR_UNSUPPORTED_DTYPE;
  if (M < 0 || N <= 0 || M > INT32_MAX / 2 || N > INT32_MAX / 2) return I8LT_ERR_INVALID_ARG;
  if (gx == nullptr && !grads) return I8LT_ERR_INVALID_ARG;
  if (M > 0 && (g == nullptr || x == nullptr || mean == nullptr || rstd == nullptr)) return I8LT_ERR_INVALID_ARG;
  if (!aligned16(g) || !aligned16(x) || !aligned16(w) || !aligned16(gx) || !aligned16(gw) || !aligned16(gb))
    return I8LT_ERR_MISALIGNED;
  if (grads) {
    if (ws == nullptr || ws_bytes < i8lt_layer_norm_backward_workspace_size(M, N)) return I8LT_ERR_WORKSPACE;
    if ((reinterpret_cast<uintptr_t>(ws) & 255u) != 0) return I8LT_ERR_MISALIGNED;
  }
  if (int d = check_device()) return d;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (M == 0) {
    const size_t bytes = static_cast<size_t>(N) * (wt == DT_F32 ? 4 : 2);
    if (gw != nullptr && cudaMemsetAsync(gw, 0, bytes, s) != cudaSuccess) return I8LT_ERR_CUDA;
    if (gb != nullptr && cudaMemsetAsync(gb, 0, bytes, s) != cudaSuccess) return I8LT_ERR_CUDA;
    return I8LT_OK;
  }
  float* partial = static_cast<float*>(ws);
  if (xt == DT_F16) return cuda_status(backward<__half>(g, x, M, N, mean, rstd, w, wt, gx, gw, gb, partial, s));
  if (xt == DT_BF16)
    return cuda_status(backward<__nv_bfloat16>(g, x, M, N, mean, rstd, w, wt, gx, gw, gb, partial, s));
  return cuda_status(backward<float>(g, x, M, N, mean, rstd, w, wt, gx, gw, gb, partial, s));
}

}  // extern "C"
