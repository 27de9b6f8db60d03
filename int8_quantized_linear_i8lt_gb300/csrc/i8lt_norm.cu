// Layer norm over the last dimension, forward and backward:
//   mean = sum_n x / N, rstd = 1 / sqrt(sum_n (x - mean)^2 / N + eps),
//   h = (x - mean) * rstd, y = h * w + b;
//   gx = rstd * (g w - mean_n(g w) - h * mean_n(g w h)),
//   gw = sum_m g h, gb = sum_m g.
// The forward has no workspace, so no status word: should a wait run out, its
// block's row and those after it are NaN.
// Statistics and sums are fp32; each output is rounded once.  Both
// directions are bound by HBM: the forward reads x and writes y, the backward
// reads x and g and writes gx, each once; everything between stays in
// registers and shared memory.
#include <algorithm>
#include <cmath>
#include <mutex>
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

// ---- packs -----------------------------------------------------------------
//
// A thread reads and writes packs of W consecutive elements: 16 bytes, or a
// single element in rows that are not 16-byte aligned.  Pack i of thread
// `lane` of kLanes starts at column (lane + i * kLanes) * W.

template <typename T, int W>
struct alignas(W == 1 ? sizeof(T) : 16) Pack {
  T v[W];
};
template <typename T, int W>
__device__ __forceinline__ Pack<T, W> load_pack(const T* p) {
  return *reinterpret_cast<const Pack<T, W>*>(p);
}
// Both halves of a 16-bit pair widen and narrow at once.
template <typename T, int W>
__device__ __forceinline__ void widen(const Pack<T, W>& p, float* f) {
  if constexpr (W == 1 || sizeof(T) == 4) {
#pragma unroll
    for (int k = 0; k < W; ++k) f[k] = to_float(p.v[k]);
  } else {
#pragma unroll
    for (int k = 0; k < W; k += 2) {
      const uint32_t u = *reinterpret_cast<const uint32_t*>(p.v + k);
      if constexpr (std::is_same<T, __half>::value) {
        const float2 q = __half22float2(*reinterpret_cast<const __half2*>(&u));
        f[k] = q.x;
        f[k + 1] = q.y;
      } else {
        f[k] = __uint_as_float(u << 16);
        f[k + 1] = __uint_as_float(u & 0xffff0000u);
      }
    }
  }
}
template <typename T, int W>
__device__ __forceinline__ void store_floats(T* dst, const float* f) {
  Pack<T, W> p;
  if constexpr (W == 1 || sizeof(T) == 4) {
#pragma unroll
    for (int k = 0; k < W; ++k) p.v[k] = from_float<T>(f[k]);
  } else {
#pragma unroll
    for (int k = 0; k < W; k += 2) {
      if constexpr (std::is_same<T, __half>::value)
        *reinterpret_cast<__half2*>(p.v + k) = __floats2half2_rn(f[k], f[k + 1]);
      else
        *reinterpret_cast<__nv_bfloat162*>(p.v + k) = __floats2bfloat162_rn(f[k], f[k + 1]);
    }
  }
  *reinterpret_cast<Pack<T, W>*>(dst) = p;
}
// W elements of a parameter vector of runtime type, widened; `none` for a
// vector that is absent.
template <int W>
__device__ __forceinline__ void load_param(const void* p, int dt, int64_t i, float none, float* f) {
  if (p == nullptr) {
#pragma unroll
    for (int k = 0; k < W; ++k) f[k] = none;
  } else if constexpr (W == 1) {
    f[0] = load_any(p, dt, i);
  } else if (dt == DT_F32) {
#pragma unroll
    for (int k = 0; k < W; k += 4)
      *reinterpret_cast<float4*>(f + k) = __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(p) + i + k));
  } else {
    using U = typename std::conditional<W == 8, uint4, uint2>::type;
    const U u = __ldg(reinterpret_cast<const U*>(static_cast<const uint16_t*>(p) + i));
    const uint32_t* q = reinterpret_cast<const uint32_t*>(&u);
#pragma unroll
    for (int k = 0; k < W / 2; ++k) {
      if (dt == DT_BF16) {
        f[2 * k] = __uint_as_float(q[k] << 16);
        f[2 * k + 1] = __uint_as_float(q[k] & 0xffff0000u);
      } else {
        const float2 h = __half22float2(*reinterpret_cast<const __half2*>(q + k));
        f[2 * k] = h.x;
        f[2 * k + 1] = h.y;
      }
    }
  }
}

// A row is shared by kLanes threads: kLanes <= 32 lanes of a warp, or a block
// of kLanes threads.  The sum of a value over them, the same bits in every
// thread; scratch: kLanes / 32 floats (block rows only), free again after the
// block's next barrier.
template <int kLanes>
__device__ __forceinline__ float row_sum(float v, float* scratch) {
#pragma unroll
  for (int o = (kLanes < 32 ? kLanes : 32) / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if constexpr (kLanes > 32) {
    if ((threadIdx.x & 31) == 0) scratch[threadIdx.x >> 5] = v;
    __syncthreads();
    v = 0.f;
    if constexpr (kLanes == 64) {
      v = scratch[0] + scratch[1];
    } else {
#pragma unroll
      for (int k = 0; k < kLanes / 32; k += 4) {
        const float4 q = *reinterpret_cast<const float4*>(scratch + k);
        v += (q.x + q.y) + (q.z + q.w);
      }
    }
  }
  return v;
}

// ---- the ring --------------------------------------------------------------
//
// Rows of more than 512 (backward: 256) elements: every block walks over rows,
// or over the same slice of rows, in turn; bulk copies bring the next rows
// into a ring of shared-memory stages while this row is worked on, so that
// the bytes in flight do not depend on how many rows a block's registers
// hold.
// Rows of a length that is no multiple of 16 bytes are worked on in the same
// packs, counted from the boundary below the row's start ("shifted": x, g, y
// and gx lie alike): with a row step that is a multiple of W, all rows of a
// block start equally far behind a boundary, so that a thread keeps its
// columns.  16384 x 5001 bf16 takes 93 us forward and 115 us backward so;
// element by element it took 74 and 70 us more.
constexpr int kMaxStages = 8;
constexpr int kRingBytes = 200 * 1024;   // shared memory per SM given to the rings

struct RingLayout {
  int cols;         // columns per block
  int slot_bytes;   // bytes of one slice of one matrix in a stage
  unsigned stages;
};

// A wait that runs out raises `abort`: nothing more is issued, and the block
// leaves once the copies under way have landed.
struct RingSync {
  uint64_t full[kMaxStages];
  int64_t issued;   // rows
  int abort;
};

template <typename T, int kMats>
struct Ring {
  const uint8_t* mat[kMats];
  uint8_t* base;
  RingSync* y;
  RingLayout L;
  int64_t N, n0, step, rows;
  unsigned long long end;   // bytes of a matrix
  int cols, shift;          // shift: elements from the boundary to a row

  __device__ __forceinline__ int64_t row(int64_t i) const { return blockIdx.x + i * step; }
  __device__ __forceinline__ unsigned long long start(int64_t i) const {
    return static_cast<unsigned long long>((row(i) * N - shift + n0) * static_cast<int64_t>(sizeof(T)));
  }
  // the end of the copy of a slice that starts at byte b: the boundary above
  // its end, or the last one inside the matrix
  __device__ __forceinline__ unsigned long long stop(unsigned long long b) const {
    return min((b + cols * sizeof(T) + 15ull) & ~15ull, end & ~15ull);
  }
  __device__ __forceinline__ void issue(int64_t i) {   // one thread, row after row
    if (*static_cast<volatile int*>(&y->abort)) return;
    y->issued = i + 1;
    const unsigned long long b = start(i), e = stop(b);
    const uint32_t bytes = e > b ? static_cast<uint32_t>(e - b) : 0u;
    const int s = static_cast<int>(static_cast<unsigned>(i) % L.stages);
    mbar_arrive_expect_tx(&y->full[s], kMats * bytes);
    if (bytes != 0)
#pragma unroll
      for (int k = 0; k < kMats; ++k)
        bulk_load(base + (static_cast<size_t>(s) * kMats + k) * L.slot_bytes, mat[k] + b, bytes, &y->full[s]);
  }
  __device__ __forceinline__ void wind_down(DevStatus* st) {   // the same thread, at the end
    if (!*static_cast<volatile int*>(&y->abort)) return;
    for (int64_t i = max(y->issued - static_cast<int64_t>(L.stages), static_cast<int64_t>(0)); i < y->issued; ++i)
      mbar_wait_out(&y->full[static_cast<unsigned>(i) % L.stages], static_cast<unsigned>(i) / L.stages & 1, st, 35);
  }
};

// Zeros behind the slices of all stages (the copies never write there).
template <typename T, int kMats>
__device__ __forceinline__ void zero_tails(const Ring<T, kMats>& r, int threads) {
  const int tail = (r.L.slot_bytes - r.cols * static_cast<int>(sizeof(T))) / 16;
  for (int i = threadIdx.x; i < tail * static_cast<int>(r.L.stages) * kMats; i += threads)
    *reinterpret_cast<uint4*>(r.base + (i / tail + 1) * r.L.slot_bytes - (i % tail + 1) * 16) = make_uint4(0, 0, 0, 0);
}

// A shifted row: its first element's place in the first pack, its end, and
// which packs reach over either.
template <int W, bool kShift>
struct Shift {
  int first, end;   // the row's places, counted from the boundary
  __device__ __forceinline__ Shift(int64_t row, int64_t N)
      : first(kShift ? static_cast<int>(row * N % W) : 0), end(static_cast<int>(N) + first) {}
  __device__ __forceinline__ bool edge(int c) const { return kShift && (c < W || c + W > end); }
  __device__ __forceinline__ bool in(int c) const { return c >= first && c < end; }
  __device__ __forceinline__ void clear(int c, float* f) const {   // what the pack at c holds of other rows
#pragma unroll
    for (int k = 0; k < W; ++k)
      if (!in(c + k)) f[k] = 0.f;
  }
  // the pack at place c of a parameter vector, and of a row whose boundary is o
  __device__ __forceinline__ void param(const void* p, int dt, int c, float none, float* f) const {
    if constexpr (!kShift) {
      load_param<W>(p, dt, c, none, f);
    } else {
#pragma unroll
      for (int k = 0; k < W; ++k) f[k] = p == nullptr ? none : in(c + k) ? load_any(p, dt, c + k - first) : 0.f;
    }
  }
  template <typename T>
  __device__ __forceinline__ void store(T* o, int c, const float* f) const {
    if (!edge(c)) {
      store_floats<T, W>(o + c, f);
      return;
    }
#pragma unroll
    for (int k = 0; k < W; ++k)
      if (in(c + k)) o[c + k] = from_float<T>(f[k]);
  }
};
// The last elements of a matrix of shifted rows, which no copy of 16 bytes
// covers, into the stage of its last row.  All threads of the block call it.
template <typename T, int kMats>
__device__ __forceinline__ void last_elements(const Ring<T, kMats>& r, int64_t i, int64_t M, int stage) {
  const int left = static_cast<int>((r.end & 15) / sizeof(T));
  if (left == 0 || r.row(i) != M - 1) return;
  const unsigned long long b = r.start(i), at = r.end & ~15ull;
  const int tid = threadIdx.x;
  if (at >= b && at < b + static_cast<unsigned long long>(r.cols) * sizeof(T) && tid < left * kMats) {
    const int k = tid / left, e = tid % left;
    reinterpret_cast<T*>(r.base + (static_cast<size_t>(stage) * kMats + k) * r.L.slot_bytes + (at - b))[e] =
        reinterpret_cast<const T*>(r.mat[k] + at)[e];
  }
  __syncthreads();
}

__device__ __forceinline__ void ring_setup(RingSync& y, unsigned stages) {
  for (unsigned i = 0; i < stages; ++i) mbar_init(&y.full[i], 1);
  y.issued = 0;
  y.abort = 0;
  fence_mbar_init();
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

// One row per kLanes threads (lanes of a warp for short rows, a block for rows
// of 8192 to 16384), held in registers; the variance is summed around the
// mean.  The block form has no ring, but several blocks per SM: 4096 x 11008
// bf16 takes 50 us (3.6 TB/s) so, 83 us in three passes over the ring.  Bound
// by the latency of a row: its loads, two sums over the block, its stores.
template <typename T, int W, int kLanes, int kE>
__global__ void __launch_bounds__(kLanes > 32 ? kLanes : 256) norm_forward_row_kernel(const ForwardArgs a) {
  constexpr int kRows = kLanes > 32 ? 1 : 256 / kLanes;
  __shared__ __align__(16) float scratch[2][kLanes > 32 ? kLanes / 32 : 1];
  const int lane = threadIdx.x % kLanes, N = static_cast<int>(a.N);
  const int64_t m = static_cast<int64_t>(blockIdx.x) * kRows + threadIdx.x / kLanes;
  const bool live = m < a.M;
  const T* x = static_cast<const T*>(a.x) + (live ? m : 0) * N;
  float v[kE];
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < kE / W; ++i) {
    const int c = (lane + i * kLanes) * W;
    if (c < N) widen<T, W>(load_pack<T, W>(x + c), v + i * W);
  }
#pragma unroll
  for (int i = 0; i < kE / W; ++i)
    if ((lane + i * kLanes) * W < N)
#pragma unroll
      for (int k = 0; k < W; ++k) s += v[i * W + k];
  const float mu = row_sum<kLanes>(s, scratch[0]) / static_cast<float>(N);
  s = 0.f;
#pragma unroll
  for (int i = 0; i < kE / W; ++i)
    if ((lane + i * kLanes) * W < N)
#pragma unroll
      for (int k = 0; k < W; ++k) {
        v[i * W + k] -= mu;
        s += v[i * W + k] * v[i * W + k];
      }
  const float r = 1.0f / sqrtf(row_sum<kLanes>(s, scratch[1]) / static_cast<float>(N) + a.eps);
  if (!live) return;
  T* y = static_cast<T*>(a.y) + m * N;
#pragma unroll
  for (int i = 0; i < kE / W; ++i) {
    const int c = (lane + i * kLanes) * W;
    if (c >= N) continue;
    float w[W], b[W];
    load_param<W>(a.w, a.wt, c, 1.f, w);
    load_param<W>(a.b, a.wt, c, 0.f, b);
#pragma unroll
    for (int k = 0; k < W; ++k) v[i * W + k] = fmaf(v[i * W + k] * r, w[k], b[k]);
    store_floats<T, W>(y + c, v + i * W);
  }
  if (lane == 0) {
    if (a.mean != nullptr) a.mean[m] = mu;
    if (a.rstd != nullptr) a.rstd[m] = r;
  }
}

// Rows of up to 8192 elements (shifted: 16384): 32 elements, and their w and
// b, in each thread's registers (16 in rows of up to 1024).  Bound by HBM:
// 16384 x 8192 bf16 takes 88 us, 6.1 TB/s.
template <typename T, int W, int kLanes, int kE, bool kShift>
__global__ void __launch_bounds__(kLanes, 512 / kLanes) norm_forward_ring_kernel(const ForwardArgs a,
                                                                                const RingLayout L) {
  extern __shared__ __align__(128) uint8_t stages[];
  __shared__ RingSync y;
  __shared__ __align__(16) float scratch[2][kLanes / 32];
  const int tid = threadIdx.x;
  const Shift<W, kShift> shift(blockIdx.x, a.N);
  const int end = shift.end;
  Ring<T, 1> ring{{static_cast<const uint8_t*>(a.x)}, stages, &y, L, a.N, 0, gridDim.x,
                  (a.M - blockIdx.x + gridDim.x - 1) / gridDim.x,
                  static_cast<unsigned long long>(a.M) * a.N * sizeof(T), end, shift.first};
  if (tid == 0) {
    ring_setup(y, L.stages);
    for (int64_t i = 0; i < L.stages && i < ring.rows; ++i) ring.issue(i);
  }
  __syncthreads();
  float w[kE], b[kE], v[kE];
#pragma unroll
  for (int i = 0; i < kE / W; ++i) {
    const int c = (tid + i * kLanes) * W;
    if (c < end) {
      shift.param(a.w, a.wt, c, 1.f, w + i * W);
      shift.param(a.b, a.wt, c, 0.f, b + i * W);
    }
  }
  const float inv_n = 1.0f / static_cast<float>(a.N);
  float lost = 0.f;   // NaN once a wait of this thread ran out: this row's and all further sums are NaN
  unsigned s = 0;
  uint32_t phase = 0;
  for (int64_t i = 0; i < ring.rows; ++i) {
    if (!mbar_wait(&y.full[s], phase, &y.abort, nullptr, 31)) lost = NAN;
    float t = lost;
    if constexpr (kShift) last_elements(ring, i, a.M, s);
    const T* x = reinterpret_cast<const T*>(stages + s * L.slot_bytes);
#pragma unroll
    for (int e = 0; e < kE / W; ++e) {
      const int c = (tid + e * kLanes) * W;
      // (a branch per pack, which keeps the loads apart: without it, on zeros
      // behind the row, 16384 x 8192 bf16 took 99 us instead of 90)
      if (c < end) {
        widen<T, W>(load_pack<T, W>(x + c), v + e * W);
        if (shift.edge(c)) shift.clear(c, v + e * W);
      } else {
#pragma unroll
        for (int k = 0; k < W; ++k) v[e * W + k] = 0.f;
      }
#pragma unroll
      for (int k = 0; k < W; ++k) t += v[e * W + k];
    }
    const float mu = row_sum<kLanes>(t, scratch[0]) * inv_n;   // its barrier: every thread has read the stage
    if (tid == 0 && i + L.stages < ring.rows) ring.issue(i + L.stages);
    if (++s == L.stages) {
      s = 0;
      phase ^= 1;
    }
    t = 0.f;
#pragma unroll
    for (int e = 0; e < kE / W; ++e) {
      const int c = (tid + e * kLanes) * W;
      if (c >= end) continue;
#pragma unroll
      for (int k = 0; k < W; ++k) v[e * W + k] -= mu;
      if (shift.edge(c)) shift.clear(c, v + e * W);
#pragma unroll
      for (int k = 0; k < W; ++k) t += v[e * W + k] * v[e * W + k];
    }
    const float r = 1.0f / sqrtf(row_sum<kLanes>(t, scratch[1]) * inv_n + a.eps);
    const int64_t m = ring.row(i);
    T* out = static_cast<T*>(a.y) + m * a.N - shift.first;
#pragma unroll
    for (int e = 0; e < kE / W; ++e) {
      const int c = (tid + e * kLanes) * W;
      if (c >= end) continue;
#pragma unroll
      for (int k = 0; k < W; ++k) v[e * W + k] = fmaf(v[e * W + k] * r, w[e * W + k], b[e * W + k]);
      shift.store(out, c, v + e * W);
    }
    if (tid == 0) {
      if (a.mean != nullptr) a.mean[m] = mu;
      if (a.rstd != nullptr) a.rstd[m] = r;
    }
  }
  if (tid == 0) ring.wind_down(nullptr);
}

// Longer rows: three passes over the row's stage in shared memory, w and b
// from L2 (registers do not hold them).  Bound by these passes: 4096 x 28672
// bf16 takes 135 us, 3.5 TB/s; shifted, where w and b are read singly, 4096 x
// 21003 takes 191 us.
constexpr int kWideThreads = 1024;
template <typename T, int W, bool kShift>
__global__ void __launch_bounds__(kWideThreads) norm_forward_wide_kernel(const ForwardArgs a, const RingLayout L) {
  extern __shared__ __align__(128) uint8_t stages[];
  __shared__ RingSync y;
  __shared__ __align__(16) float scratch[2][kWideThreads / 32];
  const int tid = threadIdx.x;
  const Shift<W, kShift> shift(blockIdx.x, a.N);
  const int end = shift.end;
  Ring<T, 1> ring{{static_cast<const uint8_t*>(a.x)}, stages, &y, L, a.N, 0, gridDim.x,
                  (a.M - blockIdx.x + gridDim.x - 1) / gridDim.x,
                  static_cast<unsigned long long>(a.M) * a.N * sizeof(T), end, shift.first};
  if (tid == 0) {
    ring_setup(y, L.stages);
    for (int64_t i = 0; i < L.stages && i < ring.rows; ++i) ring.issue(i);
  }
  __syncthreads();
  const float inv_n = 1.0f / static_cast<float>(a.N);
  float lost = 0.f;   // NaN once a wait of this thread ran out: this row's and all further sums are NaN
  unsigned s = 0;
  uint32_t phase = 0;
  for (int64_t i = 0; i < ring.rows; ++i) {
    if (!mbar_wait(&y.full[s], phase, &y.abort, nullptr, 31)) lost = NAN;
    float t = lost, v[W];
    if constexpr (kShift) last_elements(ring, i, a.M, s);
    const T* x = reinterpret_cast<const T*>(stages + s * L.slot_bytes);
#pragma unroll 4
    for (int c = tid * W; c < end; c += kWideThreads * W) {
      widen<T, W>(load_pack<T, W>(x + c), v);
      if (shift.edge(c)) shift.clear(c, v);
#pragma unroll
      for (int k = 0; k < W; ++k) t += v[k];
    }
    const float mu = row_sum<kWideThreads>(t, scratch[0]) * inv_n;
    // every thread is past the stage of the row before this one
    if (tid == 0 && i > 0 && i - 1 + L.stages < ring.rows) ring.issue(i - 1 + L.stages);
    t = 0.f;
#pragma unroll 4
    for (int c = tid * W; c < end; c += kWideThreads * W) {
      widen<T, W>(load_pack<T, W>(x + c), v);
#pragma unroll
      for (int k = 0; k < W; ++k) v[k] -= mu;
      if (shift.edge(c)) shift.clear(c, v);
#pragma unroll
      for (int k = 0; k < W; ++k) t += v[k] * v[k];
    }
    const float r = 1.0f / sqrtf(row_sum<kWideThreads>(t, scratch[1]) * inv_n + a.eps);
    const int64_t m = ring.row(i);
    T* out = static_cast<T*>(a.y) + m * a.N - shift.first;
#pragma unroll 4
    for (int c = tid * W; c < end; c += kWideThreads * W) {
      float w[W], b[W];
      shift.param(a.w, a.wt, c, 1.f, w);
      shift.param(a.b, a.wt, c, 0.f, b);
      widen<T, W>(load_pack<T, W>(x + c), v);
#pragma unroll
      for (int k = 0; k < W; ++k) v[k] = fmaf((v[k] - mu) * r, w[k], b[k]);
      shift.store(out, c, v);
    }
    if (tid == 0) {
      if (a.mean != nullptr) a.mean[m] = mu;
      if (a.rstd != nullptr) a.rstd[m] = r;
    }
    if (++s == L.stages) {
      s = 0;
      phase ^= 1;
    }
  }
  if (tid == 0) ring.wind_down(nullptr);
}

// Rows that do not fit shared memory twice: three passes over global memory
// (the second and third mostly from L2).
template <typename T>
__global__ void __launch_bounds__(kWideThreads) norm_forward_long_kernel(const ForwardArgs a) {
  __shared__ __align__(16) float scratch[2][kWideThreads / 32];
  const int64_t m = blockIdx.x, N = a.N;
  const T* x = static_cast<const T*>(a.x) + m * N;
  T* y = static_cast<T*>(a.y) + m * N;
  float t = 0.f;
  for (int64_t n = threadIdx.x; n < N; n += kWideThreads) t += to_float(x[n]);
  const float mu = row_sum<kWideThreads>(t, scratch[0]) / static_cast<float>(N);
  t = 0.f;
  for (int64_t n = threadIdx.x; n < N; n += kWideThreads) {
    const float d = to_float(x[n]) - mu;
    t += d * d;
  }
  const float r = 1.0f / sqrtf(row_sum<kWideThreads>(t, scratch[1]) / static_cast<float>(N) + a.eps);
  for (int64_t n = threadIdx.x; n < N; n += kWideThreads) {
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

int sm_count() {
  int dev = 0, sms = 152;
  cudaGetDevice(&dev);
  cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  return sms;
}

// Stages of `mats` slices of `cols` elements, for per_sm blocks per SM.
// width: the elements that the block's threads read of a slice.
RingLayout ring_layout(int64_t cols, int64_t width, int elem, int mats, int per_sm) {
  RingLayout L;
  L.cols = static_cast<int>(cols);
  L.slot_bytes = static_cast<int>(width * elem);
  L.stages = static_cast<unsigned>(std::min(kMaxStages, kRingBytes / per_sm / (mats * L.slot_bytes)));
  return L;
}

template <typename T, int W, int kLanes, int kE>
cudaError_t launch_forward_row(const ForwardArgs& a, cudaStream_t s) {
  constexpr int kThreads = kLanes > 32 ? kLanes : 256;
  norm_forward_row_kernel<T, W, kLanes, kE>
      <<<static_cast<unsigned>(ceil_div(a.M, kThreads / kLanes)), kThreads, 0, s>>>(a);
  return cudaGetLastError();
}

// Blocks (clusters) that take the rows in turn: of shifted rows each takes
// one, or they are a multiple of the pack.
int64_t row_blocks(int64_t M, int64_t most, int W, bool shifted) {
  if (M <= std::max<int64_t>(most, W)) return M;
  return shifted ? std::max<int64_t>(W, most / W * W) : most;
}

template <typename T, int W, int kLanes, int kE, bool kShift>
cudaError_t launch_forward_ring(const ForwardArgs& a, cudaStream_t s) {
  auto kernel = norm_forward_ring_kernel<T, W, kLanes, kE, kShift>;
  constexpr int per_sm = 512 / kLanes;
  const int64_t width = a.N + (kShift ? W - 1 : 0);
  const RingLayout L = ring_layout(width, round_up(width, 64), sizeof(T), 1, per_sm);
  const int smem = static_cast<int>(L.stages) * L.slot_bytes;
  if (!ensure_smem_attr(reinterpret_cast<const void*>(kernel), smem)) return cudaGetLastError();
  kernel<<<static_cast<unsigned>(row_blocks(a.M, sm_count() * per_sm, W, kShift)), kLanes, smem, s>>>(a, L);
  return cudaGetLastError();
}

// kW: elements in 16 bytes; kShift: rows are no multiple of that.
template <typename T, int kW, bool kShift>
cudaError_t forward_sized(const ForwardArgs& a, cudaStream_t s) {
  constexpr int W = kShift ? 1 : kW;   // of the kernels without shifted packs
  const int64_t width = a.N + (kShift ? kW - 1 : 0);
  if (a.N <= 64) return launch_forward_row<T, W, 8, 8>(a, s);
  if (a.N <= 256) return launch_forward_row<T, W, 32, 8>(a, s);
  if (a.N <= 512) return launch_forward_row<T, W, 32, 16>(a, s);
  if (width <= 1024) return launch_forward_ring<T, kW, 64, 16, kShift>(a, s);
  if (width <= 2048) return launch_forward_ring<T, kW, 64, 32, kShift>(a, s);
  if (width <= 4096) return launch_forward_ring<T, kW, 128, 32, kShift>(a, s);
  if (width <= 8192) return launch_forward_ring<T, kW, 256, 32, kShift>(a, s);
  if (width <= 16384) {
    if constexpr (kShift) return launch_forward_ring<T, kW, 512, 32, true>(a, s);
    else return launch_forward_row<T, kW, 512, 32>(a, s);
  }
  if (round_up(width, 64) * static_cast<int64_t>(sizeof(T)) <= kRingBytes / 2) {   // two rows
    auto kernel = norm_forward_wide_kernel<T, kW, kShift>;
    const RingLayout L = ring_layout(width, round_up(width, 64), sizeof(T), 1, 1);
    const int smem = static_cast<int>(L.stages) * L.slot_bytes;
    if (!ensure_smem_attr(reinterpret_cast<const void*>(kernel), smem)) return cudaGetLastError();
    kernel<<<static_cast<unsigned>(row_blocks(a.M, sm_count(), kW, kShift)), kWideThreads, smem, s>>>(a, L);
    return cudaGetLastError();
  }
  norm_forward_long_kernel<T><<<static_cast<unsigned>(a.M), kWideThreads, 0, s>>>(a);
  return cudaGetLastError();
}

template <typename T>
cudaError_t forward(const ForwardArgs& a, cudaStream_t s) {
  ProfScope ps(K_LAYER_NORM, s);
  constexpr int kW = 16 / sizeof(T);
  return a.N % kW == 0 ? forward_sized<T, kW, false>(a, s) : forward_sized<T, kW, true>(a, s);
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
// Bound by the latency of a row: 32768 x 118 f32 takes 16 us, 2.9 TB/s.
template <typename T, int W, int kLanes>
__global__ void __launch_bounds__(256, 2) norm_backward_short_kernel(const BackwardArgs a) {
  constexpr int kE = 8, kSlots = 256 / kLanes, kVec = kE / W;
  __shared__ float sums[kSlots][kLanes * kE];
  const int lane = threadIdx.x % kLanes, slot = threadIdx.x / kLanes, N = static_cast<int>(a.N);
  const int64_t step = static_cast<int64_t>(gridDim.x) * kSlots;
  if (blockIdx.x == 0 && threadIdx.x == 0) *a.st = DevStatus{0, 0, 0, 0};
  float w[kE], aw[kE], ab[kE];
  Pack<T, W> px[kVec], pg[kVec];
#pragma unroll
  for (int i = 0; i < kVec; ++i) {
    const int c = (lane + i * kLanes) * W;
#pragma unroll
    for (int k = 0; k < W; ++k) {
      px[i].v[k] = pg[i].v[k] = from_float<T>(0.f);
      w[i * W + k] = aw[i * W + k] = ab[i * W + k] = 0.f;
    }
    if (c < N) load_param<W>(a.w, a.wt, c, 1.f, w + i * W);
  }
  float mu = 0.f, r = 0.f;
  auto fetch = [&](int64_t m) {
    if (m >= a.M) return;
    mu = a.mean[m];
    r = a.rstd[m];
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
      const int c = (lane + i * kLanes) * W;
      if (c < N) {
        px[i] = load_pack<T, W>(static_cast<const T*>(a.x) + m * N + c);
        pg[i] = load_pack<T, W>(static_cast<const T*>(a.g) + m * N + c);
      }
    }
  };
  int64_t m = static_cast<int64_t>(blockIdx.x) * kSlots + slot;
  // every lane of a warp makes the same number of turns; a lane group without
  // a row of its own repeats what it holds and keeps nothing of it
  const int64_t first = static_cast<int64_t>(blockIdx.x) * kSlots + (threadIdx.x & ~31) / kLanes;
  fetch(m);
  for (int64_t turn = first; turn < a.M; turn += step, m += step) {
    const bool live = m < a.M;
    float h[kE], g[kE];
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
      widen<T, W>(px[i], h + i * W);
      widen<T, W>(pg[i], g + i * W);
    }
    const float cmu = mu, cr = r;
    fetch(m + step);
    float s0 = 0.f, s1 = 0.f;
#pragma unroll
    for (int e = 0; e < kE; ++e) {
      h[e] = (h[e] - cmu) * cr;
      if (live) {
        aw[e] += g[e] * h[e];
        ab[e] += g[e];
      }
      g[e] *= w[e];
      s0 += g[e];
      s1 += g[e] * h[e];
    }
    if (a.gx == nullptr) continue;
    const float c1 = row_sum<kLanes>(s0, nullptr) / static_cast<float>(N);
    const float c2 = row_sum<kLanes>(s1, nullptr) / static_cast<float>(N);
    if (!live) continue;
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
      const int c = (lane + i * kLanes) * W;
      if (c >= N) continue;
#pragma unroll
      for (int k = 0; k < W; ++k) g[i * W + k] = cr * (g[i * W + k] - c1 - h[i * W + k] * c2);
      store_floats<T, W>(static_cast<T*>(a.gx) + m * N + c, g + i * W);
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

// Sums kN values over a warp with kN - 1 + 5 - log2(kN) shuffles: each step
// halves the values a lane carries before it halves the lanes.  Value v's sum
// ends in the lanes with lane / (32 / kN) == v.
template <int kN>
__device__ __forceinline__ float warp_sums(float (&v)[kN]) {
  const int lane = threadIdx.x & 31;
  int n = kN;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    if (n > 1) {
      n >>= 1;
#pragma unroll
      for (int i = 0; i < kN / 2; ++i) {
        if (i >= n) break;
        const bool upper = (lane & o) != 0;
        const float send = upper ? v[i] : v[i + n];
        v[i] = (upper ? v[i + n] : v[i]) + __shfl_xor_sync(0xffffffffu, send, o);
      }
    } else {
      v[0] += __shfl_xor_sync(0xffffffffu, v[0], o);
    }
  }
  return v[0];
}

// A block's two sums of columns, place c of which is the thread's element
// W * i + k with c = (tid + i * kLanes) * W + k, to consecutive global memory:
// places [skip, skip + n) of `cols`, through shared memory (the stages, no
// longer needed): a thread's own stores hit a sector per element, and 8192 x
// 4096 f16 took 52 us instead of 44.
template <int W, int kLanes, int kVec>
__device__ __forceinline__ void store_sums(float* buf, int cols, int skip, int n, const float* s0, const float* s1,
                                           float* out, int64_t stride) {
  const int pitch = (cols + W - 1) / W * W;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kVec; ++i) {
    const int c = (threadIdx.x + i * kLanes) * W;
    if (c >= cols) continue;
#pragma unroll
    for (int k = 0; k < W; k += 4) {
      *reinterpret_cast<float4*>(buf + c + k) = *reinterpret_cast<const float4*>(s0 + i * W + k);
      *reinterpret_cast<float4*>(buf + pitch + c + k) = *reinterpret_cast<const float4*>(s1 + i * W + k);
    }
  }
  __syncthreads();
  for (int c = threadIdx.x; c < n; c += kLanes) {
    out[c] = buf[skip + c];
    out[stride + c] = buf[pitch + skip + c];
  }
}

// Rows of up to 8192 elements through the ring, a block per row: 16 elements
// in each thread's registers, with w and the gradient sums of their columns
// over all the block's rows.  Bound by HBM on many rows (16384 x 8192 bf16:
// 129 us, 6.2 TB/s), by the blocks' start, last row and sums on fewer
// (8192 x 4096 f16: 38 us, 5.3 TB/s).  With 8 elements per thread and twice
// the warps the former took 38 us more; reading each stage twice, for the sums
// and for gx, as in the kernel for longer rows, 21 us more.
template <typename T, int W, int kLanes, int kE, bool kShift>
__global__ void __launch_bounds__(kLanes, 512 / kLanes) norm_backward_ring_kernel(const BackwardArgs a,
                                                                                 const RingLayout L) {
  extern __shared__ __align__(128) uint8_t stages[];
  constexpr int kWarps = kLanes / 32, kVec = kE / W;
  __shared__ RingSync y;
  __shared__ __align__(16) float2 scratch[2][kWarps];
  const int tid = threadIdx.x;
  const Shift<W, kShift> shift(blockIdx.x, a.N);
  const int cols = shift.end;
  Ring<T, 2> ring{{static_cast<const uint8_t*>(a.x), static_cast<const uint8_t*>(a.g)},
                  stages, &y, L, a.N, 0, gridDim.x,
                  (a.M - blockIdx.x + gridDim.x - 1) / gridDim.x,
                  static_cast<unsigned long long>(a.M) * a.N * sizeof(T), cols, shift.first};
  const int rows = static_cast<int>(ring.rows);
  zero_tails(ring, kLanes);
  if (tid == 0) {
    ring_setup(y, L.stages);
    if (blockIdx.x == 0) *a.st = DevStatus{0, 0, 0, 0};
    for (int i = 0; i < static_cast<int>(L.stages) && i < rows; ++i) ring.issue(i);
  }
  __syncthreads();

  __align__(16) float w[kE], aw[kE], ab[kE];
#pragma unroll
  for (int i = 0; i < kVec; ++i) {
    const int c = (tid + i * kLanes) * W;
#pragma unroll
    for (int k = 0; k < W; ++k) w[i * W + k] = aw[i * W + k] = ab[i * W + k] = 0.f;
    if (c < cols) shift.param(a.w, a.wt, c, 1.f, w + i * W);
  }
  const float inv_n = 1.0f / static_cast<float>(a.N);
  const bool want_x = a.gx != nullptr;
  const float *mean = a.mean + blockIdx.x, *rstd = a.rstd + blockIdx.x;
  T* out = static_cast<T*>(a.gx) + (want_x ? blockIdx.x * a.N - shift.first : 0);
  float mu = mean[0], r = rstd[0];
  unsigned s = 0;
  uint32_t phase = 0;
  for (int i = 0; i < rows; ++i) {
    const float cmu = mu, cr = r;
    if (i + 1 < rows) {
      mean += gridDim.x;
      rstd += gridDim.x;
      mu = *mean;
      r = *rstd;
    }
    mbar_wait(&y.full[s], phase, &y.abort, a.st, 30);
    float h[kE], g[kE], t0 = 0.f, t1 = 0.f;
    if constexpr (kShift) last_elements(ring, i, a.M, s);
    const T* xs = reinterpret_cast<const T*>(stages + 2 * s * L.slot_bytes);
    const T* gs = reinterpret_cast<const T*>(stages + (2 * s + 1) * L.slot_bytes);
#pragma unroll
    for (int e = 0; e < kVec; ++e) {
      const int c = (tid + e * kLanes) * W;
      // with the zeros behind the row: a branch per pack cost 16384 x 8192 bf16
      // 43 us more
      widen<T, W>(load_pack<T, W>(xs + c), h + e * W);
      widen<T, W>(load_pack<T, W>(gs + c), g + e * W);
      if (shift.edge(c)) {
        shift.clear(c, h + e * W);
        shift.clear(c, g + e * W);
      }
#pragma unroll
      for (int k = e * W; k < (e + 1) * W; ++k) {
        h[k] = (h[k] - cmu) * cr;
        aw[k] += g[k] * h[k];
        ab[k] += g[k];
        g[k] *= w[k];
        t0 += g[k];
        t1 += g[k] * h[k];
      }
    }
    float v[2] = {t0, t1};
    const float t = warp_sums<2>(v);
    if ((tid & 15) == 0) reinterpret_cast<float*>(&scratch[i & 1][tid >> 5])[(tid >> 4) & 1] = t;
    __syncthreads();   // every thread has read the stage
    if (tid == 0 && i + static_cast<int>(L.stages) < rows) ring.issue(i + L.stages);
    if (++s == L.stages) {
      s = 0;
      phase ^= 1;
    }
    if (!want_x) continue;
    t0 = t1 = 0.f;
    if constexpr (kWarps == 2) {
      t0 = scratch[i & 1][0].x + scratch[i & 1][1].x;
      t1 = scratch[i & 1][0].y + scratch[i & 1][1].y;
    } else {
#pragma unroll
      for (int k = 0; k < kWarps; k += 2) {
        const float4 q = *reinterpret_cast<const float4*>(&scratch[i & 1][k]);
        t0 += q.x + q.z;
        t1 += q.y + q.w;
      }
    }
    const float c1 = -cr * (t0 * inv_n), c2 = -cr * (t1 * inv_n);
#pragma unroll
    for (int e = 0; e < kVec; ++e) {
      const int c = (tid + e * kLanes) * W;
#pragma unroll
      for (int k = e * W; k < (e + 1) * W; ++k) g[k] = fmaf(h[k], c2, fmaf(g[k], cr, c1));
      if (c < cols) shift.store(out, c, g + e * W);
    }
    out += gridDim.x * a.N;
  }
  grid_dependents_launch();
  if (tid == 0) ring.wind_down(a.st);
  if (a.partial == nullptr) return;
  store_sums<W, kLanes, kVec>(reinterpret_cast<float*>(stages), cols, shift.first, static_cast<int>(a.N), aw, ab,
                              a.partial + static_cast<int64_t>(blockIdx.x) * a.N,
                              static_cast<int64_t>(gridDim.x) * a.N);
}

// Longer rows: a cluster of blocks per row, each on a slice of it.  kRows
// rows are worked on between two barriers: their stages are read twice, for
// the rows' two sums and for gx, so that registers hold only w and the
// gradient sums of the thread's columns.  The blocks send each other their
// sums without waiting: gx follows one step later.  Bound by instruction
// issue and the steps' barriers: 4096 x 12288 bf16 takes 84 us, 3.6 TB/s,
// 4096 x 28672 184 us, 3.8 TB/s.
template <typename T, int W, int kLanes, int kE, int kRows, bool kShift>
__global__ void __launch_bounds__(kLanes, 512 / kLanes) norm_backward_cluster_kernel(const BackwardArgs a,
                                                                                 const RingLayout L) {
  extern __shared__ __align__(128) uint8_t stages[];
  constexpr int kWarps = kLanes / 32, kVec = kE / W, kSums = 2 * kRows;
  __shared__ RingSync y;
  __shared__ uint64_t sent[4];
  __shared__ float scratch[2][kSums][kWarps];
  __shared__ __align__(16) float peer[4][8][kSums];   // the cluster's slice sums of a step, by rank
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int ranks = static_cast<int>(gridDim.y), rank = static_cast<int>(blockIdx.y);
  const int64_t n0 = static_cast<int64_t>(rank) * L.cols;
  const Shift<W, kShift> shift(blockIdx.x, a.N);
  const int first = static_cast<int>(n0);   // n0, like the slices, in places from the boundary
  const int cols = min(L.cols, shift.end - first);
  Ring<T, 2> ring{{static_cast<const uint8_t*>(a.x), static_cast<const uint8_t*>(a.g)},
                  stages, &y, L, a.N, n0, gridDim.x,
                  (a.M - blockIdx.x + gridDim.x - 1) / gridDim.x,
                  static_cast<unsigned long long>(a.M) * a.N * sizeof(T), cols, shift.first};
  const int64_t rows = ring.rows, steps = (rows + kRows - 1) / kRows;
  zero_tails(ring, kLanes);
  if (tid == 0) {
    for (int i = 0; i < 4; ++i) mbar_init(&sent[i], 1);
    ring_setup(y, L.stages);
    if (blockIdx.x == 0 && rank == 0) *a.st = DevStatus{0, 0, 0, 0};
    for (int64_t i = 0; i < L.stages && i < rows; ++i) ring.issue(i);
  }
  __syncthreads();
  if (ranks > 1) cluster_sync();   // the peers' barriers are ready

  __align__(16) float w[kE], aw[kE], ab[kE];
#pragma unroll
  for (int i = 0; i < kVec; ++i) {
    const int c = (tid + i * kLanes) * W;
#pragma unroll
    for (int k = 0; k < W; ++k) w[i * W + k] = aw[i * W + k] = ab[i * W + k] = 0.f;
    if (c < cols) shift.param(a.w, a.wt, first + c, 1.f, w + i * W);
  }
  auto read_pack = [&](const T* slice, int c, float* f) {
    widen<T, W>(load_pack<T, W>(slice + c), f);
    if (c < cols && shift.edge(first + c)) shift.clear(first + c, f);
  };
  const float inv_n = 1.0f / static_cast<float>(a.N);
  const bool want_x = a.gx != nullptr;
  const int lag = ranks > 1 && want_x ? 1 : 0;
  int64_t armed = 0;   // steps whose sums the peers were told to send (lane 0 of warp 0)
  for (int64_t i = 0; i < steps + lag; ++i) {
    if (i < steps) {
      float sums[kSums];
#pragma unroll
      for (int q = 0; q < kRows; ++q) {
        sums[2 * q] = sums[2 * q + 1] = 0.f;
        const int64_t row = i * kRows + q;
        if (row >= rows) continue;
        const int s = static_cast<int>(static_cast<unsigned>(row) % L.stages);
        mbar_wait(&y.full[s], static_cast<unsigned>(row) / L.stages & 1, &y.abort, a.st, 30);
        if constexpr (kShift) last_elements(ring, row, a.M, s);
        if (!want_x) continue;
        const float mu = __ldg(a.mean + ring.row(row)), r = __ldg(a.rstd + ring.row(row));
        const T* xs = reinterpret_cast<const T*>(stages + 2 * s * L.slot_bytes);
        const T* gs = reinterpret_cast<const T*>(stages + (2 * s + 1) * L.slot_bytes);
#pragma unroll
        for (int e = 0; e < kVec; ++e) {
          float x[W], g[W];
          read_pack(xs, (tid + e * kLanes) * W, x);
          read_pack(gs, (tid + e * kLanes) * W, g);
#pragma unroll
          for (int k = 0; k < W; ++k) {
            g[k] *= w[e * W + k];
            sums[2 * q] += g[k];
            sums[2 * q + 1] += g[k] * (x[k] - mu);
          }
        }
        sums[2 * q + 1] *= r;
      }
      if (want_x) {
        const float t = warp_sums<kSums>(sums);
        if ((lane & (32 / kSums - 1)) == 0) scratch[i & 1][lane / (32 / kSums)][warp] = t;
      }
    }
    __syncthreads();
    // every thread is done with the rows of step i - 1 - lag
    if (tid == 0 && i > lag)
      for (int q = 0; q < kRows; ++q) {
        const int64_t next = (i - 1 - lag) * kRows + q + L.stages;
        if (next < rows) ring.issue(next);
      }
    // The totals of a step: value v in the lanes with lane / (32 / kSums) == v.
    float total = 0.f;
    const int v = lane / (32 / kSums), sub = lane & (32 / kSums - 1);
    if (want_x && i < steps) {
      for (int k = sub; k < kWarps; k += 32 / kSums) total += scratch[i & 1][v][k];
#pragma unroll
      for (int o = 16 / kSums; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
    }
    if (lag != 0 && i < steps && warp == 0 && !*static_cast<volatile int*>(&y.abort)) {
      if (lane == 0) armed = i + 1;
      if (lane == 0) mbar_arrive_expect_tx(&sent[i & 3], 4u * kSums * ranks);
      // lane group v sends value v, lane `sub` of it to rank sub
      if (sub < ranks)
        asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.b32 [%0], %1, [%2];" ::"r"(
                         mapa_shared(&peer[i & 3][rank][v], sub)),
                     "r"(__float_as_uint(total)), "r"(mapa_shared(&sent[i & 3], sub))
                     : "memory");
    }
    const int64_t j = i - lag;
    if (j < 0) continue;
    if (lag != 0) {
      mbar_wait(&sent[j & 3], static_cast<uint32_t>(j >> 2) & 1, &y.abort, a.st, 32);
      total = 0.f;
      for (int k = 0; k < ranks; ++k) total += peer[j & 3][k][v];
    }
#pragma unroll
    for (int q = 0; q < kRows; ++q) {
      const int64_t row = j * kRows + q;
      if (row >= rows) break;
      const int s = static_cast<int>(static_cast<unsigned>(row) % L.stages);
      const float mu = __ldg(a.mean + ring.row(row)), r = __ldg(a.rstd + ring.row(row));
      const float c1 = -r * inv_n * __shfl_sync(0xffffffffu, total, 2 * q * (32 / kSums));
      const float c2 = -r * inv_n * __shfl_sync(0xffffffffu, total, (2 * q + 1) * (32 / kSums));
      const T* xs = reinterpret_cast<const T*>(stages + 2 * s * L.slot_bytes);
      const T* gs = reinterpret_cast<const T*>(stages + (2 * s + 1) * L.slot_bytes);
      T* out = static_cast<T*>(a.gx) + ring.row(row) * a.N - shift.first;
#pragma unroll
      for (int e = 0; e < kVec; ++e) {
        const int c = (tid + e * kLanes) * W;
        float x[W], g[W];
        read_pack(xs, c, x);
        read_pack(gs, c, g);
#pragma unroll
        for (int k = 0; k < W; ++k) {
          x[k] = (x[k] - mu) * r;
          aw[e * W + k] += g[k] * x[k];
          ab[e * W + k] += g[k];
          g[k] = fmaf(x[k], c2, fmaf(g[k] * w[e * W + k], r, c1));
        }
        if (want_x && c < cols) shift.store(out, first + c, g);
      }
    }
  }
  if (tid == 0) {
    ring.wind_down(a.st);
    if (*static_cast<volatile int*>(&y.abort))   // the peers' sums under way, of two steps at most
      for (int64_t i = max(armed - 2, static_cast<int64_t>(0)); i < armed; ++i)
        mbar_wait_out(&sent[i & 3], static_cast<uint32_t>(i >> 2) & 1, a.st, 36);
  }
  __syncwarp();
  if (ranks > 1) cluster_sync();   // no block leaves while a peer may write to it
  if (a.partial == nullptr) return;
  // this slice's places [0, cols) are the columns from first - shift.first on,
  // those of the row among them
  const int skip = max(0, shift.first - first);
  store_sums<W, kLanes, kVec>(reinterpret_cast<float*>(stages), cols, skip, cols - skip, aw, ab,
                              a.partial + static_cast<int64_t>(blockIdx.x) * a.N + (first + skip - shift.first),
                              static_cast<int64_t>(gridDim.x) * a.N);
}

// Rows beyond a cluster's reach: passes over global memory.
template <typename T>
__global__ void __launch_bounds__(kWideThreads) norm_backward_long_kernel(const BackwardArgs a) {
  __shared__ __align__(16) float scratch[2][kWideThreads / 32];
  if (blockIdx.x == 0 && threadIdx.x == 0) *a.st = DevStatus{0, 0, 0, 0};
  const int64_t m = blockIdx.x, N = a.N;
  const T* g = static_cast<const T*>(a.g) + m * N;
  const T* x = static_cast<const T*>(a.x) + m * N;
  T* gx = static_cast<T*>(a.gx) + m * N;
  const float mu = a.mean[m], r = a.rstd[m];
  float s0 = 0.f, s1 = 0.f;
  for (int64_t n = threadIdx.x; n < N; n += kWideThreads) {
    const float gw = to_float(g[n]) * (a.w != nullptr ? load_any(a.w, a.wt, n) : 1.f);
    s0 += gw;
    s1 += gw * ((to_float(x[n]) - mu) * r);
  }
  const float c1 = row_sum<kWideThreads>(s0, scratch[0]) / static_cast<float>(N);
  const float c2 = row_sum<kWideThreads>(s1, scratch[1]) / static_cast<float>(N);
  for (int64_t n = threadIdx.x; n < N; n += kWideThreads) {
    const float gw = to_float(g[n]) * (a.w != nullptr ? load_any(a.w, a.wt, n) : 1.f);
    gx[n] = from_float<T>(r * (gw - c1 - ((to_float(x[n]) - mu) * r) * c2));
  }
}
template <typename T>
__global__ void __launch_bounds__(256) norm_grad_long_kernel(const BackwardArgs a, int64_t rows) {
  if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) *a.st = DevStatus{0, 0, 0, 0};
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
// columns per block (blockIdx.y: gw or gb), 32 threads per column.  Bound by
// latency: 304 sums of 4096 columns add 5 us to the kernel before.
__global__ void __launch_bounds__(1024) norm_grad_sum_kernel(const float* partial, int blocks, int64_t N, int wt,
                                                             void* gw, void* gb) {
  __shared__ float sums[32][33];
  const int lane = threadIdx.x & 31, part = threadIdx.x >> 5;
  void* out = blockIdx.y == 0 ? gw : gb;
  if (out == nullptr) return;
  grid_dependency_wait();
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

constexpr int kShortRow = 256;         // columns up to which a warp takes a row
constexpr int kSliceCols = 8192;       // largest slice of a row per block of the ring kernel
constexpr int kMaxCluster = 8;
constexpr int kSms = 152;

// Rows of partial sums the workspace has room for, and so the most blocks (or
// clusters) of a launch: those that fit the SMs at once in the length's class.
// Shifted rows take at least a pack's 8, as far as there are rows.
int64_t partial_rows(int64_t M, int64_t N) {
  const int64_t per_sm = N <= kShortRow ? 4 : N <= 1024 ? 8 : N <= 2048 ? 4 : N <= 4096 ? 2 : 1;
  return std::max<int64_t>(1, std::min<int64_t>(kSms * per_sm, N <= kShortRow ? ceil_div(M, 8) : M));
}

struct Shape {
  const BackwardArgs& a;
  int sms;
  int blocks;    // out: rows of partial sums
  cudaStream_t s;
};

template <typename T, int W, int kLanes>
cudaError_t launch_short(Shape& h) {
  auto kernel = norm_backward_short_kernel<T, W, kLanes>;
  const int per_sm = std::min(4, cached_blocks_per_sm(reinterpret_cast<const void*>(kernel), 256, 0));
  h.blocks = static_cast<int>(std::min<int64_t>(
      {ceil_div(h.a.M, 256 / kLanes), static_cast<int64_t>(h.sms) * per_sm, partial_rows(h.a.M, h.a.N)}));
  ProfScope ps(K_LAYER_NORM_BWD, h.s);
  kernel<<<h.blocks, 256, 0, h.s>>>(h.a);
  return cudaGetLastError();
}

template <typename T, int W, int kLanes, int kE, bool kShift>
cudaError_t launch_ring(Shape& h) {
  constexpr int per_sm = 512 / kLanes;
  const RingLayout L = ring_layout(h.a.N, kLanes * kE, sizeof(T), 2, per_sm);
  auto kernel = norm_backward_ring_kernel<T, W, kLanes, kE, kShift>;
  const int smem = static_cast<int>(L.stages) * 2 * L.slot_bytes;
  if (!ensure_smem_attr(reinterpret_cast<const void*>(kernel), smem)) return cudaGetLastError();
  h.blocks = static_cast<int>(row_blocks(
      h.a.M, std::min<int64_t>(static_cast<int64_t>(h.sms) * per_sm, partial_rows(h.a.M, h.a.N)), W, kShift));
  ProfScope ps(K_LAYER_NORM_BWD, h.s);
  kernel<<<h.blocks, kLanes, smem, h.s>>>(h.a, L);
  return cudaGetLastError();
}

// Clusters of a kernel resident at once, asked for once per (kernel, device,
// shared memory, cluster size).
template <typename Query>
int cached_clusters(const void* fn, int smem, int ranks, Query query) {
  struct Entry {
    const void* fn;
    int dev, smem, ranks, n;
  };
  static Entry cache[64];
  static int used = 0;
  static std::mutex mu;
  int dev = 0;
  cudaGetDevice(&dev);
  std::lock_guard<std::mutex> lock(mu);
  for (int i = 0; i < used; ++i)
    if (cache[i].fn == fn && cache[i].dev == dev && cache[i].smem == smem && cache[i].ranks == ranks)
      return cache[i].n;
  const int n = query();
  if (n == 0) cudaGetLastError();
  if (used < 64) cache[used++] = Entry{fn, dev, smem, ranks, n};
  return n;
}

// Two rows per step where the ring holds the rows of a step, of the one
// before it and of the next.
template <typename T, int W, bool kShift, int kLanes>
cudaError_t launch_cluster(Shape& h, int64_t width) {
  constexpr int kE = 16, per_sm = 512 / kLanes;
  const int64_t least = ceil_div(width, kLanes * kE);
  const int64_t cols = round_up(ceil_div(width, least), 8);   // slices of whole packs
  const int ranks = static_cast<int>(ceil_div(width, cols));
  const RingLayout L = ring_layout(cols, kLanes * kE, sizeof(T), 2, per_sm);
  auto kernel = L.stages >= 6u ? norm_backward_cluster_kernel<T, W, kLanes, kE, 2, kShift>
                               : norm_backward_cluster_kernel<T, W, kLanes, kE, 1, kShift>;
  const int smem = static_cast<int>(L.stages) * 2 * L.slot_bytes;
  if (!ensure_smem_attr(reinterpret_cast<const void*>(kernel), smem)) return cudaGetLastError();
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(1, static_cast<unsigned>(ranks));
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
  // as many clusters as fit at once (a processor group whose SMs are no
  // multiple of the cluster leaves some idle): one more would wait for a
  // whole pass of the others
  const int resident = cached_clusters(reinterpret_cast<const void*>(kernel), smem, ranks, [&] {
    int n = 0;
    cudaLaunchConfig_t q = cfg;
    q.gridDim.x = static_cast<unsigned>(std::max(1, h.sms * per_sm / ranks));
    return cudaOccupancyMaxActiveClusters(&n, kernel, &q) == cudaSuccess ? n : 0;
  });
  h.blocks = static_cast<int>(row_blocks(
      h.a.M, std::min<int64_t>(std::max(1, std::min(resident, h.sms * per_sm / ranks)), partial_rows(h.a.M, h.a.N)), W,
      kShift));
  cfg.gridDim.x = static_cast<unsigned>(h.blocks);
  ProfScope ps(K_LAYER_NORM_BWD, h.s);
  return cudaLaunchKernelEx(&cfg, kernel, h.a, L);
}

template <typename T, int kW, bool kShift>
cudaError_t backward_sized(Shape& h) {
  constexpr int W = kShift ? 1 : kW;
  const int64_t N = h.a.N, width = N + (kShift ? kW - 1 : 0);
  if (N <= 64) return launch_short<T, W, 8>(h);
  if (N <= kShortRow) return launch_short<T, W, 32>(h);
  if (width <= 512) return launch_ring<T, kW, 64, 8, kShift>(h);
  if (width <= 1024) return launch_ring<T, kW, 64, 16, kShift>(h);
  if (width <= 2048) return launch_ring<T, kW, 128, 16, kShift>(h);
  if (width <= 4096) return launch_ring<T, kW, 256, 16, kShift>(h);
  if (width <= 6144) return launch_ring<T, kW, 384, 16, kShift>(h);
  if (width <= kSliceCols) return launch_ring<T, kW, 512, 16, kShift>(h);
  // two blocks per SM, of other clusters, where eight of their slices hold a
  // row: 4096 x 12288 bf16 took 94 us so and 109 us with one of twice the size
  if (width <= kMaxCluster * kSliceCols / 2) return launch_cluster<T, kW, kShift, 256>(h, width);
  if (width <= kMaxCluster * kSliceCols) return launch_cluster<T, kW, kShift, 512>(h, width);
  if (h.a.gx != nullptr) {
    ProfScope ps(K_LAYER_NORM_BWD, h.s);
    norm_backward_long_kernel<T><<<static_cast<unsigned>(h.a.M), kWideThreads, 0, h.s>>>(h.a);
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
  if (cudaError_t e = a.N % kW == 0 ? backward_sized<T, kW, false>(h) : backward_sized<T, kW, true>(h)) return e;
  if (a.partial == nullptr) return cudaSuccess;
  ProfScope ps(K_LAYER_NORM_GRAD_SUM, s);
  // started while the backward kernel's last blocks run
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(ceil_div(a.N, 32)), 2);
  cfg.blockDim = dim3(1024);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, norm_grad_sum_kernel, static_cast<const float*>(a.partial), h.blocks, a.N, a.wt, gw,
                            gb);
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
    if (cudaMemsetAsync(ws, 0, sizeof(DevStatus), s) != cudaSuccess) return I8LT_ERR_CUDA;
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
