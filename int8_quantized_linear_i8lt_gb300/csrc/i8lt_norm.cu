// Layer norm over the last dimension, forward and backward:
//   mean = sum_n x / N, rstd = 1 / sqrt(sum_n (x - mean)^2 / N + eps),
//   h = (x - mean) * rstd, y = h * w + b;
//   gx = rstd * (g w - mean_n(g w) - h * mean_n(g w h)),
//   gw = sum_m g h, gb = sum_m g.
// Statistics and sums are fp32; each output is rounded once.  Both
// directions are bound by HBM: the forward reads x and writes y, the backward
// reads x and g and writes gx, each once; everything between stays in
// registers and shared memory.
#include <algorithm>
#include <type_traits>

#include "i8lt.h"
#include "i8lt_internal.h"

namespace i8lt {
namespace {

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

// W consecutive elements held in their storage type: one 16-byte access, or
// a single element in rows that are not 16-byte aligned.
template <typename T, int W>
struct Pack {
  T v[W];
};
template <typename T, int W>
__device__ __forceinline__ Pack<T, W> load_pack(const T* p) {
  Pack<T, W> r;
  if constexpr (W == 1) {
    r.v[0] = p[0];
  } else {
    static_assert(W * sizeof(T) == 16, "one 16-byte access");
    *reinterpret_cast<uint4*>(r.v) = *reinterpret_cast<const uint4*>(p);
  }
  return r;
}
template <typename T, int W>
__device__ __forceinline__ void store_pack(T* p, const Pack<T, W>& r) {
  if constexpr (W == 1) p[0] = r.v[0];
  else *reinterpret_cast<uint4*>(p) = *reinterpret_cast<const uint4*>(r.v);
}
// W elements of a parameter vector of runtime type, widened.
template <int W>
__device__ __forceinline__ void load_param(const void* p, int dt, int64_t i, float (&f)[W]) {
  if constexpr (W == 1) {
    f[0] = load_any(p, dt, i);
  } else if (dt == DT_F32) {
#pragma unroll
    for (int k = 0; k < W; k += 4)
      *reinterpret_cast<float4*>(f + k) = __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(p) + i + k));
  } else {
    using U = typename std::conditional<W == 8, uint4, uint2>::type;
    const U u = __ldg(reinterpret_cast<const U*>(static_cast<const uint16_t*>(p) + i));
    const uint16_t* q = reinterpret_cast<const uint16_t*>(&u);
#pragma unroll
    for (int k = 0; k < W; ++k)
      f[k] = dt == DT_BF16 ? __uint_as_float(static_cast<uint32_t>(q[k]) << 16) : __half2float(__ushort_as_half(q[k]));
  }
}

// A row is shared by kLanes threads: kLanes <= 32 lanes of a warp, or a block
// of kLanes threads.  Sum of `kN` values over them, the same bits in every
// thread; scratch: kN * kLanes / 32 floats (block rows only), which the next
// but one call may reuse after another barrier.
template <int kLanes, int kN>
__device__ __forceinline__ void row_sum(float (&v)[kN], float* scratch) {
#pragma unroll
  for (int o = (kLanes < 32 ? kLanes : 32) / 2; o > 0; o >>= 1)
#pragma unroll
    for (int i = 0; i < kN; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
  if constexpr (kLanes > 32) {
    if ((threadIdx.x & 31) == 0)
#pragma unroll
      for (int i = 0; i < kN; ++i) scratch[i * (kLanes / 32) + (threadIdx.x >> 5)] = v[i];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      float s = 0.f;
      if constexpr (kLanes == 64) {
        s = scratch[2 * i] + scratch[2 * i + 1];
      } else {
#pragma unroll
        for (int k = 0; k < kLanes / 32; k += 4) {
          const float4 q = *reinterpret_cast<const float4*>(scratch + i * (kLanes / 32) + k);
          s += (q.x + q.y) + (q.z + q.w);
        }
      }
      v[i] = s;
    }
  }
}

// ---- forward ---------------------------------------------------------------

struct ForwardArgs {
  const void* x;
  void* y;
  const void *w, *b;
  float *mean, *rstd;
  int64_t M, N;
  int wt;
  float eps;
};

// The whole row in registers: kVec packs of W elements per thread, read once;
// the variance is summed around the mean.  Blocks of 256 threads hold
// 256 / kLanes short rows, longer ones a block each.
template <typename T, int W, int kLanes, int kVec>
__global__ void __launch_bounds__(kLanes < 256 ? 256 : kLanes) norm_forward_kernel(const ForwardArgs a) {
  constexpr int kRows = kLanes < 256 ? (kLanes > 32 ? 1 : 256 / kLanes) : 1;
  __shared__ __align__(16) float scratch[2][kLanes > 32 ? kLanes / 32 : 1];
  const int lane = threadIdx.x % kLanes;
  const int64_t m = static_cast<int64_t>(blockIdx.x) * kRows + threadIdx.x / kLanes;
  const bool live = m < a.M;
  const int64_t N = a.N;
  const T* x = static_cast<const T*>(a.x) + (live ? m : 0) * N;
  Pack<T, W> p[kVec];
  float s[1] = {0.f};
#pragma unroll
  for (int i = 0; i < kVec; ++i) {
    const int64_t n = static_cast<int64_t>(lane + i * kLanes) * W;
    if (n < N) p[i] = load_pack<T, W>(x + n);
  }
#pragma unroll
  for (int i = 0; i < kVec; ++i) {
    const int64_t n = static_cast<int64_t>(lane + i * kLanes) * W;
    if (n < N)
#pragma unroll
      for (int k = 0; k < W; ++k) s[0] += to_float(p[i].v[k]);
  }
  row_sum<kLanes, 1>(s, scratch[0]);
  const float mu = s[0] / static_cast<float>(N);
  s[0] = 0.f;
#pragma unroll
  for (int i = 0; i < kVec; ++i) {
    const int64_t n = static_cast<int64_t>(lane + i * kLanes) * W;
    if (n < N)
#pragma unroll
      for (int k = 0; k < W; ++k) {
        const float d = to_float(p[i].v[k]) - mu;
        s[0] += d * d;
      }
  }
  row_sum<kLanes, 1>(s, scratch[1]);
  const float r = 1.0f / sqrtf(s[0] / static_cast<float>(N) + a.eps);
  if (!live) return;
  T* y = static_cast<T*>(a.y) + m * N;
#pragma unroll
  for (int i = 0; i < kVec; ++i) {
    const int64_t n = static_cast<int64_t>(lane + i * kLanes) * W;
    if (n >= N) continue;
    float f[W], q[W];
#pragma unroll
    for (int k = 0; k < W; ++k) f[k] = (to_float(p[i].v[k]) - mu) * r;
    if (a.w != nullptr) {
      load_param<W>(a.w, a.wt, n, q);
#pragma unroll
      for (int k = 0; k < W; ++k) f[k] *= q[k];
    }
    if (a.b != nullptr) {
      load_param<W>(a.b, a.wt, n, q);
#pragma unroll
      for (int k = 0; k < W; ++k) f[k] += q[k];
    }
#pragma unroll
    for (int k = 0; k < W; ++k) p[i].v[k] = from_float<T>(f[k]);
    store_pack<T, W>(y + n, p[i]);
  }
  if (lane == 0) {
    if (a.mean != nullptr) a.mean[m] = mu;
    if (a.rstd != nullptr) a.rstd[m] = r;
  }
}

// Rows that do not fit the registers of a block: three passes over the row,
// the later ones from L1 / L2.
constexpr int kLongThreads = 1024;
template <typename T>
__global__ void __launch_bounds__(kLongThreads) norm_forward_long_kernel(const ForwardArgs a) {
  __shared__ __align__(16) float scratch[2][kLongThreads / 32];
  const int64_t m = blockIdx.x, N = a.N;
  const T* x = static_cast<const T*>(a.x) + m * N;
  T* y = static_cast<T*>(a.y) + m * N;
  float s[1] = {0.f};
  for (int64_t n = threadIdx.x; n < N; n += kLongThreads) s[0] += to_float(x[n]);
  row_sum<kLongThreads, 1>(s, scratch[0]);
  const float mu = s[0] / static_cast<float>(N);
  s[0] = 0.f;
  for (int64_t n = threadIdx.x; n < N; n += kLongThreads) {
    const float d = to_float(x[n]) - mu;
    s[0] += d * d;
  }
  row_sum<kLongThreads, 1>(s, scratch[1]);
  const float r = 1.0f / sqrtf(s[0] / static_cast<float>(N) + a.eps);
  for (int64_t n = threadIdx.x; n < N; n += kLongThreads) {
    float v = (to_float(x[n]) - mu) * r;
    if (a.w != nullptr) v *= load_any(a.w, a.wt, n);
    if (a.b != nullptr) v += load_any(a.b, a.wt, n);
    y[n] = from_float<T>(v);
  }
  if (threadIdx.x == 0) {
    if (a.mean != nullptr) a.mean[m] = mu;
    if (a.rstd != nullptr) a.rstd[m] = r;
  }
}

template <typename T, int W, int kLanes, int kVec>
cudaError_t launch_forward(const ForwardArgs& a, cudaStream_t s) {
  constexpr int kRows = kLanes > 32 ? 1 : 256 / kLanes;
  norm_forward_kernel<T, W, kLanes, kVec>
      <<<static_cast<unsigned>(ceil_div(a.M, kRows)), kLanes > 32 ? kLanes : 256, 0, s>>>(a);
  return cudaGetLastError();
}

// The fewest threads that hold a row with 32 elements each (8 in rows of up
// to 256): fewer partial sums to exchange, and enough rows in flight per SM.
template <typename T, int W>
cudaError_t forward_sized(const ForwardArgs& a, cudaStream_t s) {
  if (a.N <= 64) return launch_forward<T, W, 8, 8 / W>(a, s);
  if (a.N <= 256) return launch_forward<T, W, 32, 8 / W>(a, s);
  if (a.N <= 1024) return launch_forward<T, W, 32, 32 / W>(a, s);
  if (a.N <= 4096) return launch_forward<T, W, 128, 32 / W>(a, s);
  if (a.N <= 8192) return launch_forward<T, W, 256, 32 / W>(a, s);
  if (a.N <= 16384) return launch_forward<T, W, 512, 32 / W>(a, s);
  if (a.N <= 32768) return launch_forward<T, W, 1024, 32 / W>(a, s);
  norm_forward_long_kernel<T><<<static_cast<unsigned>(a.M), kLongThreads, 0, s>>>(a);
  return cudaGetLastError();
}

template <typename T>
cudaError_t forward(const ForwardArgs& a, cudaStream_t s) {
  ProfScope ps(K_LAYER_NORM, s);
  constexpr int kW = 16 / sizeof(T);
  return a.N % kW == 0 ? forward_sized<T, kW>(a, s) : forward_sized<T, 1>(a, s);
}

// ---- backward --------------------------------------------------------------

struct BackwardArgs {
  const void *g, *x;
  const float *mean, *rstd;
  const void* w;
  void* gx;                // or NULL
  float* partial;          // [2][blocks][N], or NULL: sums of g h and of g over a block's rows
  DevStatus* st;
  int64_t M, N;
  int wt;
};

// Short rows: kLanes lanes of a warp per row, rows dealt out in turn, the
// next row's loads issued before this row's arithmetic; every lane sums its
// own columns' gradients over its rows, the block adds them up at the end.
template <typename T, int W, int kLanes, int kVec>
__global__ void __launch_bounds__(256) norm_backward_short_kernel(const BackwardArgs a) {
  constexpr int kSlots = 256 / kLanes;
  constexpr int kElems = kVec * W;
  __shared__ float sums[kSlots][kLanes * kElems];
  const int lane = threadIdx.x % kLanes, slot = threadIdx.x / kLanes;
  const int64_t N = a.N, step = static_cast<int64_t>(gridDim.x) * kSlots;
  const T* x = static_cast<const T*>(a.x);
  const T* g = static_cast<const T*>(a.g);
  float w[kElems], aw[kElems], ab[kElems];
#pragma unroll
  for (int i = 0; i < kVec; ++i) {
    const int64_t n = static_cast<int64_t>(lane + i * kLanes) * W;
    float q[W];
#pragma unroll
    for (int k = 0; k < W; ++k) q[k] = n < N ? 1.f : 0.f;
    if (a.w != nullptr && n < N) load_param<W>(a.w, a.wt, n, q);
#pragma unroll
    for (int k = 0; k < W; ++k) {
      w[i * W + k] = q[k];
      aw[i * W + k] = ab[i * W + k] = 0.f;
    }
  }
  Pack<T, W> px[kVec], pg[kVec];
  float mu = 0.f, r = 0.f;
  auto fetch = [&](int64_t m) {
    if (m >= a.M) return;
    mu = a.mean[m];
    r = a.rstd[m];
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
      const int64_t n = static_cast<int64_t>(lane + i * kLanes) * W;
      if (n < N) {
        px[i] = load_pack<T, W>(x + m * N + n);
        pg[i] = load_pack<T, W>(g + m * N + n);
      }
    }
  };
  int64_t m = static_cast<int64_t>(blockIdx.x) * kSlots + slot;
  // every lane of a warp makes the same number of turns
  const int64_t first = static_cast<int64_t>(blockIdx.x) * kSlots + (threadIdx.x & ~31) / kLanes;
  fetch(m);
  for (int64_t turn = first; turn < a.M; turn += step, m += step) {
    const bool live = m < a.M;
    float h[kElems], gv[kElems];
    const float cmu = mu, cr = r;
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
      const bool in = live && static_cast<int64_t>(lane + i * kLanes) * W < N;
#pragma unroll
      for (int k = 0; k < W; ++k) {
        h[i * W + k] = in ? (to_float(px[i].v[k]) - cmu) * cr : 0.f;
        gv[i * W + k] = in ? to_float(pg[i].v[k]) : 0.f;
      }
    }
    fetch(m + step);
    float s[2] = {0.f, 0.f};
#pragma unroll
    for (int e = 0; e < kElems; ++e) {
      aw[e] += gv[e] * h[e];
      ab[e] += gv[e];
      gv[e] *= w[e];
      s[0] += gv[e];
      s[1] += gv[e] * h[e];
    }
    if (a.gx == nullptr) continue;
    row_sum<kLanes, 2>(s, nullptr);
    const float c1 = s[0] / static_cast<float>(N), c2 = s[1] / static_cast<float>(N);
    if (!live) continue;
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
      const int64_t n = static_cast<int64_t>(lane + i * kLanes) * W;
      if (n >= N) continue;
      Pack<T, W> o;
#pragma unroll
      for (int k = 0; k < W; ++k) o.v[k] = from_float<T>(cr * (gv[i * W + k] - c1 - h[i * W + k] * c2));
      store_pack<T, W>(static_cast<T*>(a.gx) + m * N + n, o);
    }
  }
  if (a.partial == nullptr) return;
#pragma unroll
  for (int v = 0; v < 2; ++v) {
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kVec; ++i)
#pragma unroll
      for (int k = 0; k < W; ++k)
        sums[slot][(lane + i * kLanes) * W + k] = v == 0 ? aw[i * W + k] : ab[i * W + k];
    __syncthreads();
    for (int n = threadIdx.x; n < N; n += 256) {
      float t = 0.f;
      for (int k = 0; k < kSlots; ++k) t += sums[k][n];
      a.partial[(static_cast<int64_t>(v) * gridDim.x + blockIdx.x) * N + n] = t;
    }
  }
}

// Longer rows: a block per row slice of up to kLanes * 16 columns, a cluster
// of blocks per row when one does not cover it.  Every block walks over rows
// in turn; bulk copies bring the x and g slices of the next rows into a ring
// of shared-memory stages while this row is worked on; each thread keeps the
// gradient sums of its 16 columns in registers over all its rows.  Rows that
// do not start on 16 bytes are copied from the boundary below them and read
// element by element.
constexpr int kElems = 16;
constexpr int kMaxStages = 8;

struct RingLayout {
  int cols;         // columns per block
  int slot_bytes;   // bytes of one slice in a stage
  int stages;
};

template <typename T, int W, int kLanes>
__global__ void __launch_bounds__(kLanes, 512 / kLanes) norm_backward_ring_kernel(const BackwardArgs a, const RingLayout L) {
  extern __shared__ __align__(128) uint8_t ring[];
  __shared__ uint64_t full[kMaxStages];
  __shared__ __align__(16) float scratch[2][2 * (kLanes / 32)];
  __shared__ float2 peer[2][8];    // the cluster's slice sums of a row, by rank
  __shared__ int abort_flag;
  constexpr int kVec = kElems / W;
  const int tid = threadIdx.x;
  const int ranks = static_cast<int>(gridDim.y), rank = static_cast<int>(blockIdx.y);
  const int64_t N = a.N, n0 = static_cast<int64_t>(rank) * L.cols;
  const int cols = static_cast<int>(min(static_cast<int64_t>(L.cols), N - n0));
  const int64_t row_step = gridDim.x;
  const int64_t rows = blockIdx.x < a.M ? (a.M - blockIdx.x + row_step - 1) / row_step : 0;
  if (tid == 0) {
    for (int i = 0; i < L.stages; ++i) mbar_init(&full[i], 1);
    abort_flag = 0;
    fence_mbar_init();
    if (blockIdx.x == 0 && rank == 0) *a.st = DevStatus{0, 0, 0, 0};
  }
  __syncthreads();

  // Slice of row number i (of this block's rows): the bytes from the 16-byte
  // boundary below it to the one above its end, or below where that would be
  // past the end of the matrix; the elements not covered are read directly.
  using u64 = unsigned long long;
  const u64 end_bytes = static_cast<u64>(a.M) * N * sizeof(T);
  auto start_byte = [&](int64_t i) {
    return static_cast<u64>(((blockIdx.x + i * row_step) * N + n0) * static_cast<int64_t>(sizeof(T)));
  };
  auto slice_end = [&](u64 b) { return min((b + cols * sizeof(T) + 15ull) & ~15ull, end_bytes & ~15ull); };
  auto issue = [&](int64_t i) {   // thread 0
    const u64 b = start_byte(i), lo = b & ~15ull, hi = slice_end(b);
    const uint32_t bytes = hi > lo ? static_cast<uint32_t>(hi - lo) : 0u;
    const int s = static_cast<int>(i % L.stages);
    uint8_t* slot = ring + static_cast<size_t>(s) * 2 * L.slot_bytes;
    mbar_arrive_expect_tx(&full[s], 2 * bytes);
    if (bytes != 0) {
      bulk_load(slot, static_cast<const uint8_t*>(a.x) + lo, bytes, &full[s]);
      bulk_load(slot + L.slot_bytes, static_cast<const uint8_t*>(a.g) + lo, bytes, &full[s]);
    }
  };
  if (tid == 0)
    for (int64_t i = 0; i < L.stages && i < rows; ++i) issue(i);

  float w[kElems], aw[kElems], ab[kElems];
#pragma unroll
  for (int i = 0; i < kVec; ++i) {
    const int c = (tid + i * kLanes) * W;
    float q[W];
#pragma unroll
    for (int k = 0; k < W; ++k) q[k] = c < cols ? 1.f : 0.f;
    if (a.w != nullptr && c < cols) load_param<W>(a.w, a.wt, n0 + c, q);
#pragma unroll
    for (int k = 0; k < W; ++k) {
      w[i * W + k] = q[k];
      aw[i * W + k] = ab[i * W + k] = 0.f;
    }
  }

  const float inv_n = 1.0f / static_cast<float>(N);
  float mu = 0.f, r = 0.f;
  if (rows > 0) {
    mu = a.mean[blockIdx.x];
    r = a.rstd[blockIdx.x];
  }
  int s = 0;
  uint32_t phase = 0;
  for (int64_t i = 0; i < rows; ++i) {
    const int64_t m = blockIdx.x + i * row_step;
    const float cmu = mu, cr = r;
    if (i + 1 < rows) {
      mu = a.mean[m + row_step];
      r = a.rstd[m + row_step];
    }
    mbar_wait(&full[s], phase, &abort_flag, a.st, 30);
    const u64 b = start_byte(i);
    const uint8_t* xs = ring + static_cast<size_t>(s) * 2 * L.slot_bytes + (b & 15);
    const uint8_t* gs = xs + L.slot_bytes;
    float h[kElems], gv[kElems];
    const int have = W == 1 ? static_cast<int>((slice_end(b) - min(slice_end(b), b)) / sizeof(T)) : cols;
#pragma unroll
    for (int v = 0; v < kVec; ++v) {
      const int c = (tid + v * kLanes) * W;
      Pack<T, W> px, pg;
      if (c < cols) {
        if (W == 1 && c >= have) {   // the last elements of the matrix
          px.v[0] = static_cast<const T*>(a.x)[m * N + n0 + c];
          pg.v[0] = static_cast<const T*>(a.g)[m * N + n0 + c];
        } else {
          px = load_pack<T, W>(reinterpret_cast<const T*>(xs) + c);
          pg = load_pack<T, W>(reinterpret_cast<const T*>(gs) + c);
        }
      }
#pragma unroll
      for (int k = 0; k < W; ++k) {
        h[v * W + k] = c < cols ? (to_float(px.v[k]) - cmu) * cr : 0.f;
        gv[v * W + k] = c < cols ? to_float(pg.v[k]) : 0.f;
      }
    }
    float t[2] = {0.f, 0.f};
#pragma unroll
    for (int e = 0; e < kElems; ++e) {
      aw[e] += gv[e] * h[e];
      ab[e] += gv[e];
      gv[e] *= w[e];
      t[0] += gv[e];
      t[1] += gv[e] * h[e];
    }
    row_sum<kLanes, 2>(t, scratch[i & 1]);   // its barrier: every thread has read the stage
    if (tid == 0 && i + L.stages < rows) issue(i + L.stages);
    if (++s == L.stages) {
      s = 0;
      phase ^= 1;
    }
    if (a.gx == nullptr) continue;
    if (ranks > 1) {
      // each block sends its sums to all, and adds them in the order of the ranks
      if (tid < ranks) {
        const uint32_t dst = mapa_shared(&peer[i & 1][rank], tid);
        asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(dst), "f"(t[0]), "f"(t[1]) : "memory");
      }
      cluster_sync();
      t[0] = t[1] = 0.f;
      for (int q = 0; q < ranks; ++q) {
        t[0] += peer[i & 1][q].x;
        t[1] += peer[i & 1][q].y;
      }
    }
    const float c1 = t[0] * inv_n, c2 = t[1] * inv_n;
    T* gx = static_cast<T*>(a.gx) + m * N + n0;
#pragma unroll
    for (int v = 0; v < kVec; ++v) {
      const int c = (tid + v * kLanes) * W;
      if (c >= cols) continue;
      Pack<T, W> o;
#pragma unroll
      for (int k = 0; k < W; ++k) o.v[k] = from_float<T>(cr * (gv[v * W + k] - c1 - h[v * W + k] * c2));
      store_pack<T, W>(gx + c, o);
    }
  }
  if (ranks > 1 && a.gx != nullptr) cluster_sync();   // no block leaves while a peer may write to it
  if (a.partial == nullptr) return;
  float* pw = a.partial + static_cast<int64_t>(blockIdx.x) * N + n0;
  float* pb = pw + static_cast<int64_t>(gridDim.x) * N;
#pragma unroll
  for (int v = 0; v < kVec; ++v) {
    const int c = (tid + v * kLanes) * W;
    if (c >= cols) continue;
#pragma unroll
    for (int k = 0; k < W; ++k) {
      pw[c + k] = aw[v * W + k];
      pb[c + k] = ab[v * W + k];
    }
  }
}

// Rows beyond a cluster's reach: passes over global memory.
template <typename T>
__global__ void __launch_bounds__(kLongThreads) norm_backward_long_kernel(const BackwardArgs a) {
  __shared__ __align__(16) float scratch[2 * (kLongThreads / 32)];
  const int64_t m = blockIdx.x, N = a.N;
  const T* g = static_cast<const T*>(a.g) + m * N;
  const T* x = static_cast<const T*>(a.x) + m * N;
  T* gx = static_cast<T*>(a.gx) + m * N;
  const float mu = a.mean[m], r = a.rstd[m];
  float s[2] = {0.f, 0.f};
  for (int64_t n = threadIdx.x; n < N; n += kLongThreads) {
    const float gw = to_float(g[n]) * (a.w != nullptr ? load_any(a.w, a.wt, n) : 1.f);
    s[0] += gw;
    s[1] += gw * ((to_float(x[n]) - mu) * r);
  }
  row_sum<kLongThreads, 2>(s, scratch);
  const float c1 = s[0] / static_cast<float>(N), c2 = s[1] / static_cast<float>(N);
  for (int64_t n = threadIdx.x; n < N; n += kLongThreads) {
    const float gw = to_float(g[n]) * (a.w != nullptr ? load_any(a.w, a.wt, n) : 1.f);
    gx[n] = from_float<T>(r * (gw - c1 - ((to_float(x[n]) - mu) * r) * c2));
  }
}
template <typename T>
__global__ void __launch_bounds__(256) norm_grad_long_kernel(const BackwardArgs a, int64_t rows) {
  const int64_t n = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x, N = a.N;
  if (n >= N) return;
  const int64_t c = blockIdx.y, m0 = c * rows, m1 = min(m0 + rows, a.M);
  float sw = 0.f, sb = 0.f;
  for (int64_t m = m0; m < m1; ++m) {
    const float gv = to_float(static_cast<const T*>(a.g)[m * N + n]);
    sw += gv * ((to_float(static_cast<const T*>(a.x)[m * N + n]) - a.mean[m]) * a.rstd[m]);
    sb += gv;
  }
  a.partial[c * N + n] = sw;
  a.partial[(gridDim.y + c) * N + n] = sb;
}

// gw[n], gb[n]: the blocks' partial sums added up in a fixed order, 32
// columns per block (blockIdx.y: gw or gb), 32 threads per column.
__global__ void __launch_bounds__(1024) norm_grad_sum_kernel(const float* partial, int blocks, int64_t N, int wt,
                                                             void* gw, void* gb) {
  __shared__ float sums[32][33];
  const int lane = threadIdx.x & 31, part = threadIdx.x >> 5;
  void* out = blockIdx.y == 0 ? gw : gb;
  if (out == nullptr) return;
  const int64_t n = static_cast<int64_t>(blockIdx.x) * 32 + lane;
  const float* p = partial + static_cast<int64_t>(blockIdx.y) * blocks * N + n;
  float s = 0.f;
  if (n < N)
#pragma unroll 4
    for (int c = part; c < blocks; c += 32) s += p[static_cast<int64_t>(c) * N];
  sums[lane][part] = s;
  __syncthreads();
  // warp `part` adds column `part`'s 32 sums
  s = sums[part][lane];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  const int64_t col = static_cast<int64_t>(blockIdx.x) * 32 + part;
  if (lane == 0 && col < N) store_any(out, wt, col, s);
}

constexpr int kShortRow = 512;         // columns up to which a warp takes a row
constexpr int kSliceCols = 8192;       // columns a block of the ring kernel covers
constexpr int kMaxCluster = 8;
constexpr int kRingBytes = 200 * 1024; // shared memory per SM given to the ring
constexpr int kMaxBlocks = 1216;       // eight blocks of each of 152 SMs

int sm_count() {
  int dev = 0, sms = 152;
  cudaGetDevice(&dev);
  cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  return sms;
}

// Rows of partial sums the workspace has room for.
int64_t partial_rows(int64_t M, int64_t N) {
  const int64_t per_block = N <= kShortRow ? 8 : 1;
  return std::max<int64_t>(1, std::min<int64_t>(kMaxBlocks, ceil_div(M, per_block)));
}

struct Shape {
  const BackwardArgs& a;
  int sms;
  int blocks;    // out: rows of partial sums
  cudaStream_t s;
};

template <typename T, int W, int kLanes, int kVec>
cudaError_t launch_short(Shape& h) {
  auto kernel = norm_backward_short_kernel<T, W, kLanes, kVec>;
  const int per_sm = std::min(4, cached_blocks_per_sm(reinterpret_cast<const void*>(kernel), 256, 0));
  h.blocks = static_cast<int>(std::min<int64_t>(
      {ceil_div(h.a.M, 256 / kLanes), static_cast<int64_t>(h.sms) * per_sm, partial_rows(h.a.M, h.a.N)}));
  ProfScope ps(K_LAYER_NORM_BWD, h.s);
  kernel<<<h.blocks, 256, 0, h.s>>>(h.a);
  return cudaGetLastError();
}

template <typename T, int W, int kLanes>
cudaError_t launch_ring(Shape& h) {
  auto kernel = norm_backward_ring_kernel<T, W, kLanes>;
  const int64_t N = h.a.N;
  RingLayout L;
  const int ranks = static_cast<int>(ceil_div(N, kSliceCols));
  // slices start on 16 bytes of an aligned row
  L.cols = static_cast<int>(round_up(ceil_div(N, ranks), 8));
  L.slot_bytes = static_cast<int>(round_up(L.cols * static_cast<int64_t>(sizeof(T)) + 16, 128));
  const int per_sm = 512 / kLanes;
  L.stages = std::min(kMaxStages, kRingBytes / per_sm / (2 * L.slot_bytes));
  const int smem = L.stages * 2 * L.slot_bytes;
  if (!ensure_smem_attr(reinterpret_cast<const void*>(kernel), smem)) return cudaGetLastError();
  const int64_t resident = std::max(1, h.sms * per_sm / ranks);
  h.blocks = static_cast<int>(std::min<int64_t>({h.a.M, resident, partial_rows(h.a.M, N)}));
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(h.blocks), static_cast<unsigned>(ranks));
  cfg.blockDim = dim3(kLanes);
  cfg.dynamicSmemBytes = static_cast<size_t>(smem);
  cfg.stream = h.s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 1;
  attr[0].val.clusterDim.y = static_cast<unsigned>(ranks);
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  ProfScope ps(K_LAYER_NORM_BWD, h.s);
  return cudaLaunchKernelEx(&cfg, kernel, h.a, L);
}

template <typename T, int W>
cudaError_t backward_sized(Shape& h) {
  const int64_t N = h.a.N;
  if (N <= 64) return launch_short<T, W, 8, 8 / W>(h);
  if (N <= 256) return launch_short<T, W, 32, 8 / W>(h);
  if (N <= kShortRow) return launch_short<T, W, 32, 16 / W>(h);
  if (N <= 1024) return launch_ring<T, W, 64>(h);
  if (N <= 2048) return launch_ring<T, W, 128>(h);
  if (N <= 4096) return launch_ring<T, W, 256>(h);
  if (N <= static_cast<int64_t>(kSliceCols) * kMaxCluster) return launch_ring<T, W, 512>(h);
  if (h.a.gx != nullptr) {
    ProfScope ps(K_LAYER_NORM_BWD, h.s);
    norm_backward_long_kernel<T><<<static_cast<unsigned>(h.a.M), kLongThreads, 0, h.s>>>(h.a);
    if (cudaError_t e = cudaGetLastError()) return e;
  }
  if (h.a.partial == nullptr) return cudaSuccess;
  h.blocks = static_cast<int>(std::min<int64_t>(ceil_div(h.a.M, 16), partial_rows(h.a.M, N)));
  ProfScope ps(K_LAYER_NORM_BWD, h.s);
  norm_grad_long_kernel<T><<<dim3(static_cast<unsigned>(ceil_div(N, 256)), h.blocks), 256, 0, h.s>>>(
      h.a, ceil_div(h.a.M, h.blocks));
  return cudaGetLastError();
}

template <typename T>
cudaError_t backward(const BackwardArgs& a, void* gw, void* gb, cudaStream_t s) {
  constexpr int kW = 16 / sizeof(T);
  Shape h{a, sm_count(), 0, s};
  if (cudaError_t e = a.N % kW == 0 ? backward_sized<T, kW>(h) : backward_sized<T, 1>(h)) return e;
  if (a.partial == nullptr) return cudaSuccess;
  ProfScope ps(K_LAYER_NORM_GRAD_SUM, s);
  norm_grad_sum_kernel<<<dim3(static_cast<unsigned>(ceil_div(a.N, 32)), 2), 1024, 0, s>>>(a.partial, h.blocks, a.N,
                                                                                         a.wt, gw, gb);
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
  const ForwardArgs a{x, y, w, b, mean, rstd, M, N, wt, eps};
  if (xt == DT_F16) return cuda_status(forward<__half>(a, s));
  if (xt == DT_BF16) return cuda_status(forward<__nv_bfloat16>(a, s));
  return cuda_status(forward<float>(a, s));
}

size_t i8lt_layer_norm_backward_workspace_size(int64_t M, int64_t N) {
  if (M < 0 || N <= 0 || M > INT32_MAX / 2 || N > INT32_MAX / 2) return 0;
  return 256 + static_cast<size_t>(round_up(partial_rows(M, N) * N * 8, 256));
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
  if (ws == nullptr || ws_bytes < i8lt_layer_norm_backward_workspace_size(M, N)) return I8LT_ERR_WORKSPACE;
  if ((reinterpret_cast<uintptr_t>(ws) & 255u) != 0) return I8LT_ERR_MISALIGNED;
  if (int d = check_device()) return d;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (M == 0) {
    const size_t bytes = static_cast<size_t>(N) * (wt == DT_F32 ? 4 : 2);
    if (gw != nullptr && cudaMemsetAsync(gw, 0, bytes, s) != cudaSuccess) return I8LT_ERR_CUDA;
    if (gb != nullptr && cudaMemsetAsync(gb, 0, bytes, s) != cudaSuccess) return I8LT_ERR_CUDA;
    return I8LT_OK;
  }
  float* partial = grads ? reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + 256) : nullptr;
  const BackwardArgs a{g, x, mean, rstd, w, gx, partial, static_cast<DevStatus*>(ws), M, N, wt};
  if (xt == DT_F16) return cuda_status(backward<__half>(a, gw, gb, s));
  if (xt == DT_BF16) return cuda_status(backward<__nv_bfloat16>(a, gw, gb, s));
  return cuda_status(backward<float>(a, gw, gb, s));
}

}  // extern "C"
