// Low-rank adapters of many requests at once beside a shared projection.
// Token m uses adapter e = index[m] (none outside [0, E)):
//   t[m] = x[m] A[e]^T,            y[m]  = base[m] + scale[e] t[m] B[e]^T,
//   u[m] = scale[e] g[m] B[e],     gx[m] = addend[m] + u[m] A[e],
//   gA[e] = sum_m u[m]^T x[m],     gB[e] = scale[e] sum_m g[m]^T t[m],
// with A [E, r, K], B [E, N, r].  Every sum is fp32.  t and u are rounded to
// the 16-bit compute type (each is the operand of a second product, as the
// 16-bit activations are of the layers' own products); y, gx, gA and gB are
// rounded once.
#include <algorithm>

#include "i8lt.h"
#include "i8lt_internal.h"

namespace i8lt {
namespace {

constexpr int kThreads = 256;
constexpr int kTile = 128;   // tokens per tile of the plan

// The plan: tokens sorted by adapter, those without one (group E) last, and
// tiles of at most kTile tokens of one group.  Group e's tiles take the slots
// from offset[e] / kTile + e: ranges that never overlap, because
// floor((o + n) / T) + 1 >= floor(o / T) + ceil(n / T), so no group needs
// the tile counts of the others.  Slots without a tile hold a count of 0.
struct Tile {
  int group, start, count;
  int row0;       // first token when the tile's tokens are consecutive, else -1
};
struct Plan {
  int* offset;    // [E + 2]
  int* perm;      // [M] token at each sorted place
  Tile* tiles;    // [slots]
  int64_t slots;
  size_t bytes;
};

Plan plan_layout(void* base, int64_t M, int64_t E) {
  Plan p;
  auto* b = static_cast<uint8_t*>(base);
  p.slots = M / kTile + E + 1;
  size_t off = 0;
  p.offset = reinterpret_cast<int*>(b + off);
  off += round_up((E + 2) * 4, 256);
  p.perm = reinterpret_cast<int*>(b + off);
  off += round_up(M * 4, 256);
  p.tiles = reinterpret_cast<Tile*>(b + off);
  off += round_up(p.slots * static_cast<int64_t>(sizeof(Tile)), 256);
  p.bytes = off;
  return p;
}

// One warp per group: counts the tokens of the groups before it, then places
// its own in order (a stable sort, the same on every run) and fills its slots.
__global__ void __launch_bounds__(kThreads) adapter_plan_kernel(const int32_t* index, int M, int E, int* offset,
                                                                int* perm, Tile* tiles) {
  const int e = (blockIdx.x * kThreads + threadIdx.x) >> 5, lane = threadIdx.x & 31;
  if (e > E) return;
  auto group = [&](int m) {
    const int i = index != nullptr ? index[m] : 0;
    return i >= 0 && i < E ? i : E;
  };
  int before = 0;
  for (int m = lane; m < M; m += 32) before += group(m) < e;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) before += __shfl_xor_sync(0xffffffffu, before, o);
  int n = 0;
  for (int m0 = 0; m0 < M; m0 += 32) {
    const int m = m0 + lane;
    const bool mine = m < M && group(m) == e;
    const unsigned who = __ballot_sync(0xffffffffu, mine);
    if (mine) perm[before + n + __popc(who & ((1u << lane) - 1))] = m;
    n += __popc(who);
  }
  __syncwarp();
  if (lane == 0) {
    offset[e] = before;
    if (e == E) offset[E + 1] = M;
  }
  const int slot0 = before / kTile + e, slot1 = (before + n) / kTile + e + 1;
  for (int s = slot0 + lane; s < slot1; s += 32) {
    const int start = before + (s - slot0) * kTile;
    const int count = max(0, min(kTile, before + n - start));
    int row0 = -1;
    if (count > 0 && perm[start + count - 1] - perm[start] == count - 1) row0 = perm[start];
    tiles[s] = Tile{e, start, count, row0};
  }
}

// out[m, j] = (scaled ? scale[e] : 1) * sum_c X[m, c] W(e, j, c) for the
// tokens of one tile slot; W(e, j, c) at e R C + (w_rank_major ? j C + c :
// c R + j).  One warp per (token, j) in turn.
template <typename T>
__global__ void __launch_bounds__(kThreads) shrink_kernel(const T* X, int64_t C, const T* W, int R, bool w_rank_major,
                                                          int E, const float* scale, const Tile* tiles,
                                                          const int* perm, T* out) {
  const Tile t = tiles[blockIdx.x];
  const int lane = threadIdx.x & 31;
  for (int i = threadIdx.x >> 5; i < t.count * R; i += kThreads / 32) {
    const int64_t m = perm[t.start + i / R];
    const int j = i % R;
    float s = 0.f;
    if (t.group < E) {
      const T* w = W + static_cast<int64_t>(t.group) * R * C + (w_rank_major ? j * C : j);
      const int64_t step = w_rank_major ? 1 : R;
      for (int64_t c = lane; c < C; c += 32) s += to_float(X[m * C + c]) * to_float(w[c * step]);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
      if (scale != nullptr) s *= scale[t.group];
    }
    if (lane == 0) out[m * R + j] = from_float<T>(s);
  }
}

// out[m, c] = addend[m, c] + (scaled ? scale[e] : 1) * sum_j X[m, j] W(e, j, c).
template <typename T>
__global__ void __launch_bounds__(kThreads) expand_kernel(const T* X, int R, const T* W, int64_t C, bool w_rank_major,
                                                          int E, const float* scale, const Tile* tiles,
                                                          const int* perm, const T* addend, T* out) {
  const Tile t = tiles[blockIdx.x];
  const int64_t c = static_cast<int64_t>(blockIdx.y) * kThreads + threadIdx.x;
  if (c >= C) return;
  for (int i = 0; i < t.count; ++i) {
    const int64_t m = perm[t.start + i];
    float s = 0.f;
    if (t.group < E) {
      const T* w = W + static_cast<int64_t>(t.group) * R * C + (w_rank_major ? c : c * R);
      const int64_t step = w_rank_major ? C : 1;
      for (int j = 0; j < R; ++j) s += to_float(X[m * R + j]) * to_float(w[j * step]);
      if (scale != nullptr) s *= scale[t.group];
    }
    if (addend != nullptr) s += to_float(addend[m * C + c]);
    out[m * C + c] = from_float<T>(s);
  }
}

// grad(e, j, c) = (scaled ? scale[e] : 1) * sum over the tokens of group e of
// P[m, j] X[m, c], stored as W above.
template <typename T>
__global__ void __launch_bounds__(kThreads) grad_kernel(const T* P, int R, const T* X, int64_t C, bool w_rank_major,
                                                        const float* scale, const int* offset, const int* perm,
                                                        T* grad) {
  const int64_t c = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
  if (c >= C) return;
  const int j = blockIdx.y;
  const int64_t e = blockIdx.z;
  float s = 0.f;
  for (int i = offset[e]; i < offset[e + 1]; ++i) {
    const int64_t m = perm[i];
    s += to_float(P[m * R + j]) * to_float(X[m * C + c]);
  }
  if (scale != nullptr) s *= scale[e];
  grad[e * R * C + (w_rank_major ? j * C + c : c * R + j)] = from_float<T>(s);
}

struct Problem {
  int64_t M, K, N, E;
  int R;
  const float* scale;
  Plan plan;
  cudaStream_t s;
};

template <typename T>
cudaError_t shrink(const Problem& p, const void* X, int64_t C, const void* W, bool rank_major, const float* scale,
                   void* out) {
  ProfScope ps(K_ADAPTERS, p.s);
  shrink_kernel<T><<<static_cast<unsigned>(p.plan.slots), kThreads, 0, p.s>>>(
      static_cast<const T*>(X), C, static_cast<const T*>(W), p.R, rank_major, static_cast<int>(p.E), scale,
      p.plan.tiles, p.plan.perm, static_cast<T*>(out));
  return cudaGetLastError();
}

template <typename T>
cudaError_t expand(const Problem& p, const void* X, const void* W, int64_t C, bool rank_major, const float* scale,
                   const void* addend, void* out) {
  ProfScope ps(K_ADAPTERS, p.s);
  const dim3 grid(static_cast<unsigned>(p.plan.slots), static_cast<unsigned>(ceil_div(C, kThreads)));
  expand_kernel<T><<<grid, kThreads, 0, p.s>>>(static_cast<const T*>(X), p.R, static_cast<const T*>(W), C, rank_major,
                                               static_cast<int>(p.E), scale, p.plan.tiles, p.plan.perm,
                                               static_cast<const T*>(addend), static_cast<T*>(out));
  return cudaGetLastError();
}

template <typename T>
cudaError_t grad(const Problem& p, const void* P, const void* X, int64_t C, bool rank_major, const float* scale,
                 void* out) {
  ProfScope ps(K_ADAPTERS_GRAD, p.s);
  const dim3 grid(static_cast<unsigned>(ceil_div(C, kThreads)), static_cast<unsigned>(p.R),
                  static_cast<unsigned>(p.E));
  grad_kernel<T><<<grid, kThreads, 0, p.s>>>(static_cast<const T*>(P), p.R, static_cast<const T*>(X), C, rank_major,
                                             scale, p.plan.offset, p.plan.perm, static_cast<T*>(out));
  return cudaGetLastError();
}

template <typename T>
cudaError_t forward(const Problem& p, const void* x, const void* A, const void* B, const void* base, void* y,
                    void* t) {
  if (cudaError_t e = shrink<T>(p, x, p.K, A, true, nullptr, t)) return e;
  return expand<T>(p, t, B, p.N, false, p.scale, base, y);
}

template <typename T>
cudaError_t backward(const Problem& p, const void* g, const void* x, const void* t, const void* A, const void* B,
                     const void* addend, void* gx, void* gA, void* gB, void* u) {
  if (gx != nullptr || gA != nullptr) {
    if (cudaError_t e = shrink<T>(p, g, p.N, B, false, p.scale, u)) return e;
  }
  if (gx != nullptr) {
    if (cudaError_t e = expand<T>(p, u, A, p.K, true, nullptr, addend, gx)) return e;
  }
  if (gA != nullptr) {
    if (cudaError_t e = grad<T>(p, u, x, p.K, true, nullptr, gA)) return e;
  }
  if (gB != nullptr) return grad<T>(p, t, g, p.N, false, p.scale, gB);
  return cudaSuccess;
}

constexpr int64_t kMaxRank = 128, kMaxAdapters = 65535;

bool valid_sizes(int64_t M, int64_t K, int64_t N, int64_t E, int64_t r) {
  return M >= 0 && K > 0 && N > 0 && E > 0 && r > 0 && r <= kMaxRank && E <= kMaxAdapters && M <= INT32_MAX / 2 &&
         K <= (1 << 23) && N <= (1 << 23);
}

bool aligned256(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 255u) == 0; }

}  // namespace
}  // namespace i8lt

using namespace i8lt;

extern "C" {

size_t i8lt_adapter_plan_bytes(int64_t M, int64_t E) {
  if (!valid_sizes(M, 1, 1, E, 1)) return 0;
  return plan_layout(nullptr, M, E).bytes;
}

int i8lt_adapter_plan(const int32_t* index, int64_t M, int64_t E, void* plan, size_t plan_bytes, void* stream) {
  if (!valid_sizes(M, 1, 1, E, 1)) return I8LT_ERR_INVALID_ARG;
  if (plan == nullptr || plan_bytes < i8lt_adapter_plan_bytes(M, E)) return I8LT_ERR_WORKSPACE;
  if (!aligned256(plan) || (reinterpret_cast<uintptr_t>(index) & 3u) != 0) return I8LT_ERR_MISALIGNED;
  if (int d = check_device()) return d;
  const Plan p = plan_layout(plan, M, E);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  ProfScope ps(K_ADAPTER_PLAN, s);
  adapter_plan_kernel<<<static_cast<unsigned>(ceil_div((E + 1) * 32, kThreads)), kThreads, 0, s>>>(
      index, static_cast<int>(M), static_cast<int>(E), p.offset, p.perm, p.tiles);
  return cuda_status(cudaGetLastError());
}

size_t i8lt_adapters_workspace_size(int64_t M, int64_t K, int64_t N, int64_t E, int64_t r) {
  if (!valid_sizes(M, K, N, E, r)) return 0;
  return 256 + static_cast<size_t>(round_up(M * r * 2, 256));
}

int i8lt_adapters_forward(const void* x, int dt, int64_t M, int64_t K, const void* A, const void* B, int64_t E,
                          int64_t r, int64_t N, const float* scale, const void* plan, const void* base, void* y,
                          void* t, void* ws, size_t ws_bytes, void* stream) {
  if (dt != DT_F16 && dt != DT_BF16) return I8LT_ERR_UNSUPPORTED_DTYPE;
  if (!valid_sizes(M, K, N, E, r)) return I8LT_ERR_INVALID_ARG;
  if (A == nullptr || B == nullptr || plan == nullptr) return I8LT_ERR_INVALID_ARG;
  if (M > 0 && (x == nullptr || y == nullptr || t == nullptr)) return I8LT_ERR_INVALID_ARG;
  if (!aligned16(x) || !aligned16(A) || !aligned16(B) || !aligned16(base) || !aligned16(y) || !aligned16(t) ||
      !aligned256(plan) || !aligned256(ws))
    return I8LT_ERR_MISALIGNED;
  if (ws == nullptr || ws_bytes < i8lt_adapters_workspace_size(M, K, N, E, r)) return I8LT_ERR_WORKSPACE;
  if (int d = check_device()) return d;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (cudaMemsetAsync(ws, 0, sizeof(DevStatus), s) != cudaSuccess) return I8LT_ERR_CUDA;
  if (M == 0) return I8LT_OK;
  const Problem p{M, K, N, E, static_cast<int>(r), scale, plan_layout(const_cast<void*>(plan), M, E), s};
  return cuda_status(dt == DT_F16 ? forward<__half>(p, x, A, B, base, y, t)
                                  : forward<__nv_bfloat16>(p, x, A, B, base, y, t));
}

int i8lt_adapters_backward(const void* g, const void* x, const void* t, int dt, int64_t M, int64_t K, const void* A,
                           const void* B, int64_t E, int64_t r, int64_t N, const float* scale, const void* plan,
                           const void* addend, void* gx, void* gA, void* gB, void* ws, size_t ws_bytes,
                           void* stream) {
  if (dt != DT_F16 && dt != DT_BF16) return I8LT_ERR_UNSUPPORTED_DTYPE;
  if (!valid_sizes(M, K, N, E, r)) return I8LT_ERR_INVALID_ARG;
  if (gx == nullptr && gA == nullptr && gB == nullptr) return I8LT_ERR_INVALID_ARG;
  if (A == nullptr || B == nullptr || plan == nullptr) return I8LT_ERR_INVALID_ARG;
  if (M > 0 && (g == nullptr || (x == nullptr && gA != nullptr) || (t == nullptr && gB != nullptr)))
    return I8LT_ERR_INVALID_ARG;
  if (!aligned16(g) || !aligned16(x) || !aligned16(t) || !aligned16(A) || !aligned16(B) || !aligned16(addend) ||
      !aligned16(gx) || !aligned16(gA) || !aligned16(gB) || !aligned256(plan) || !aligned256(ws))
    return I8LT_ERR_MISALIGNED;
  if (ws == nullptr || ws_bytes < i8lt_adapters_workspace_size(M, K, N, E, r)) return I8LT_ERR_WORKSPACE;
  if (int d = check_device()) return d;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (cudaMemsetAsync(ws, 0, sizeof(DevStatus), s) != cudaSuccess) return I8LT_ERR_CUDA;
  if (M == 0) {   // no tokens: the weight gradients are zeros
    if (gA != nullptr && cudaMemsetAsync(gA, 0, static_cast<size_t>(E * r * K) * 2, s) != cudaSuccess)
      return I8LT_ERR_CUDA;
    if (gB != nullptr && cudaMemsetAsync(gB, 0, static_cast<size_t>(E * r * N) * 2, s) != cudaSuccess)
      return I8LT_ERR_CUDA;
    return I8LT_OK;
  }
  const Problem p{M, K, N, E, static_cast<int>(r), scale, plan_layout(const_cast<void*>(plan), M, E), s};
  void* u = static_cast<uint8_t*>(ws) + 256;
  return cuda_status(dt == DT_F16 ? backward<__half>(p, g, x, t, A, B, addend, gx, gA, gB, u)
                                  : backward<__nv_bfloat16>(p, g, x, t, A, B, addend, gx, gA, gB, u));
}

}  // extern "C"
