// Block-scaled FP8 linear layer (sm_103a): E4M3 codes with one fp32 scale per
// 128 columns of a row (tokens) and per 128 x 128 block (weight), multiplied
// on the FP8 tensor cores; one weight, or one per expert with the tokens of
// an expert in consecutive rows.
//
//   quantising a block:  a = max |x|, r = fp32(448 / a) (0 for a < 2^-100),
//                        code = E4M3(fp32(x r)), scale = fp32(a fp32(1/448))
//   forward   y[m, n] = sum_b sx[m, b] sw[n / 128, b] sum_(k in b) qx[m, k] qw[n, k] + bias[n]
//   backward gx[m, k] = sum_b sg[m, b] sw[b, k / 128] sum_(n in b) qg[m, n] qw[n, k]
//
// Both products are D[m, r] = sum_b s[m, b] w[r / 128, b] sum_(c in b) X[m, c] W(r, c)
// with R outputs and a reduction over C; the backward reads the same weight
// codes as an MN-major operand, so no transposed copy is kept.
#include <cuda_fp8.h>

#include <algorithm>
#include <atomic>
#include <cstring>

#include "i8lt.h"
#include "i8lt_internal.h"

namespace i8lt {
namespace {

constexpr int kBlk = 128;            // columns (of a weight: and rows) per scale
constexpr float kE4M3Max = 448.0f;
constexpr float kTinyMax = 0x1p-100f;   // blocks below it are blocks of zeros: 448 / a could overflow
constexpr int kMaxExperts = I8LT_FP8_MAX_EXPERTS;

int64_t code_ld(int64_t C) { return round_up(C, 16); }

// ---------------------------------------------------------------------------
// quantising
// ---------------------------------------------------------------------------

__device__ __forceinline__ uint32_t abs_bits(float x) { return __float_as_uint(x) & 0x7fffffffu; }
// 448 / a, and 0 for a block of zeros (for a NaN, too: NaN * 0 stays NaN).
__device__ __forceinline__ float code_scale(float a) { return a >= kTinyMax ? __fdiv_rn(kE4M3Max, a) : 0.f; }
__device__ __forceinline__ float block_scale(float a) { return __fmul_rn(a, 1.0f / kE4M3Max); }
__device__ __forceinline__ uint32_t encode4(float a, float b, float c, float d) {
  const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
  const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
  return lo | (hi << 16);
}

// Rows.  A thread takes 16 consecutive columns, 8 threads a block of 128, a
// warp 512 columns of a row, a thread block a range of rows of them; the
// maximum is taken over the bits of |x|, so that a NaN stands above all.
// kSum: also the columns' sums over the block's rows (of the values before
// they are rounded), partial [row ranges][C], for the bias gradient.
// Bound by HBM: 2 bytes read and 1 written per element, two rows under way.
// 16384 x 8192 bf16: 70 us, 5.8 TB/s (with one row under way and a division
// per item of work 92); 16384 x 28672 with the sums 285 us, 5.0 TB/s, at 78
// registers a thread (a pass of its own for the sums: 245 us on top of 275).
template <typename T, bool kSum>
__global__ void __launch_bounds__(256) fp8_quantize_kernel(const T* __restrict__ x, int64_t M, int C, int ld, bool vec,
                                                           int rows, uint8_t* __restrict__ codes,
                                                           float* __restrict__ scales, float* __restrict__ partial,
                                                           DevStatus* st) {
  grid_dependents_launch();
  if (st != nullptr && blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) *st = DevStatus{0, 0, 0, 0};
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int c = blockIdx.x * 512 + lane * 16;
  const int64_t m0 = static_cast<int64_t>(blockIdx.y) * rows, m1 = min(M, m0 + rows);
  const bool whole = vec && c + 16 <= C;
  float sum[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) sum[i] = 0.f;
  auto load = [&](int64_t m, float (&f)[16]) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float (&g)[8] = *reinterpret_cast<float (*)[8]>(f + 8 * h);
      load8_float(x + m * C + c + 8 * h, C - c - 8 * h, whole || (vec && c + 8 * h + 8 <= C), g);
    }
  };
  auto quantize = [&](int64_t m, float (&f)[16]) {
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 16; ++i) top = max(top, abs_bits(f[i]));
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
    const float a = __uint_as_float(top), r = code_scale(a);
    if constexpr (kSum) {
#pragma unroll
      for (int i = 0; i < 16; ++i) sum[i] += f[i];
    }
    if (c < ld) {
#pragma unroll
      for (int i = 0; i < 16; ++i) f[i] = __fmul_rn(f[i], r);
      uint4 q;
      q.x = encode4(f[0], f[1], f[2], f[3]);
      q.y = encode4(f[4], f[5], f[6], f[7]);
      q.z = encode4(f[8], f[9], f[10], f[11]);
      q.w = encode4(f[12], f[13], f[14], f[15]);
      *reinterpret_cast<uint4*>(codes + m * ld + c) = q;
      if ((lane & 7) == 0) scales[static_cast<int64_t>(c / kBlk) * M + m] = block_scale(a);
    }
  };
  int64_t m = m0 + warp;
  for (; m + 8 < m1; m += 16) {
    float f[16], g[16];
    load(m, f);
    load(m + 8, g);
    quantize(m, f);
    quantize(m + 8, g);
  }
  if (m < m1) {
    float f[16];
    load(m, f);
    quantize(m, f);
  }
  if constexpr (kSum) {
    __shared__ float4 sums[8][4][32];
#pragma unroll
    for (int i = 0; i < 4; ++i) sums[warp][i][lane] = make_float4(sum[4 * i], sum[4 * i + 1], sum[4 * i + 2], sum[4 * i + 3]);
    __syncthreads();
    // column k of the 512: part (k / 4) % 4 of lane k / 16
    for (int k = threadIdx.x; k < 512; k += 256) {
      const int col = blockIdx.x * 512 + k;
      if (col >= C) continue;
      float s = 0.f;
#pragma unroll
      for (int w = 0; w < 8; ++w) s += reinterpret_cast<const float*>(&sums[w][(k >> 2) & 3][k >> 4])[k & 3];
      partial[static_cast<int64_t>(blockIdx.y) * C + col] = s;
    }
  }
}

// Row ranges of the kernel above: about eight thread blocks an SM, of 16 rows
// at least.
constexpr int64_t kQuantizeBlocks = 152 * 8;
int64_t quantize_rows(int64_t M, int64_t C) {
  const int64_t ranges = std::max<int64_t>(1, kQuantizeBlocks / ceil_div(C, 512));
  return std::max<int64_t>(16, ceil_div(M, ranges));
}
int64_t quantize_ranges(int64_t M, int64_t C) { return std::max<int64_t>(1, ceil_div(M, quantize_rows(M, C))); }

// Weights: one thread block per block of 128 x 128 (once per weight).
template <typename T>
__global__ void __launch_bounds__(256) fp8_quantize_weight_kernel(const T* __restrict__ W, int N, int K, int ld,
                                                                  uint8_t* __restrict__ codes,
                                                                  float* __restrict__ scales) {
  __shared__ uint32_t top_s;
  const int kb = static_cast<int>(gridDim.x), nb = static_cast<int>(gridDim.y);
  const int k0 = blockIdx.x * kBlk, n0 = blockIdx.y * kBlk;
  const T* w = W + static_cast<int64_t>(blockIdx.z) * N * K;
  if (threadIdx.x == 0) top_s = 0;
  __syncthreads();
  const int k = k0 + (threadIdx.x & 127);
  uint32_t top = 0;
  for (int i = threadIdx.x >> 7; i < kBlk; i += 2)
    if (k < K && n0 + i < N) top = max(top, abs_bits(to_float(w[static_cast<int64_t>(n0 + i) * K + k])));
  top = __reduce_max_sync(0xffffffffu, top);
  if ((threadIdx.x & 31) == 0) atomicMax(&top_s, top);
  __syncthreads();
  const float a = __uint_as_float(top_s), r = code_scale(a);
  if (threadIdx.x == 0)
    scales[(static_cast<int64_t>(blockIdx.z) * nb + blockIdx.y) * kb + blockIdx.x] = block_scale(a);
  uint8_t* q = codes + static_cast<int64_t>(blockIdx.z) * N * ld;
  for (int i = threadIdx.x >> 7; i < kBlk; i += 2) {
    const int n = n0 + i;
    if (k < ld && n < N) {
      const float f = k < K ? to_float(w[static_cast<int64_t>(n) * K + k]) : 0.f;
      q[static_cast<int64_t>(n) * ld + k] = __nv_cvt_float_to_fp8(__fmul_rn(f, r), __NV_SATFINITE, __NV_E4M3);
    }
  }
}

template <typename T>
__global__ void __launch_bounds__(256) fp8_dequantize_weight_kernel(const uint8_t* __restrict__ codes,
                                                                    const float* __restrict__ scales, int64_t rows,
                                                                    int N, int K, int ld, T* __restrict__ out) {
  const int kb = (K + kBlk - 1) / kBlk, nb = (N + kBlk - 1) / kBlk;
  const int64_t total = rows * K, step = static_cast<int64_t>(gridDim.x) * 256;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < total; i += step) {
    const int64_t row = i / K;
    const int k = static_cast<int>(i - row * K);
    const int64_t e = row / N;
    const int n = static_cast<int>(row - e * N);
    const float s = scales[(e * nb + n / kBlk) * kb + k / kBlk];
    const __half v(__nv_cvt_fp8_to_halfraw(codes[row * ld + k], __NV_E4M3));
    out[i] = from_float<T>(__fmul_rn(__half2float(v), s));
  }
}

// ---------------------------------------------------------------------------
// products
// ---------------------------------------------------------------------------

constexpr uint16_t kNaN16 = 0x7fff;   // in fp16 and in bf16
struct Product {
  CUtensorMap tmX;           // codes of the tokens [M, ld(C)], box 128 columns x a tile's tokens
  CUtensorMap tmW;           // codes of the weight [E][N, ld(K)], box of a block and up to 128 outputs
  CUtensorMap tmOut;         // out, box 32 outputs x 32 rows (wide kernel, rows on 16 bytes)
  const float* xs;           // scales of the tokens [ceil(C / 128)][M]
  const float* ws;           // scales of the weight [E][ceil(N / 128)][ceil(K / 128)]
  const int32_t* offsets;    // [E + 1] row ranges of the experts, or NULL: one weight for all rows
  const void* bias;          // [R], or NULL
  void* out;                 // [M, R]
  DevStatus* st;
  unsigned long long limit;  // of a wait, ns
  int hold;                  // fetches after which a CTA waits for what never comes (the test of the waits), else INT_MAX
  const float* partial;      // sums of the tokens' columns over row ranges, or NULL
  void* grad_bias;           // [C]
  int M, R, C, E;
  int nb, kb;                // blocks of the weight along N and K
  int stages, split;         // few tokens, small products: stages, CTAs that share a tile's reduction
  int bias_dt;               // of bias or grad_bias
  int ranges;                // of partial
  bool bf16;                 // type of out: bf16, else fp16
  bool vec;                  // rows of out start on 16 bytes
  bool zero_rest;            // rows of no expert are written as zeros (else left as they are)
};

__device__ __forceinline__ bool wait_for(const Product& p, uint64_t* bar, uint32_t parity, volatile int* abort, int where) {
  return mbar_wait_limit(bar, parity, abort, p.st, where, 0, p.limit);
}

// After a wait that ran out: NaN in the outputs that are not to come, `rows`
// rows from row0 on and `count` outputs from r on, by a warp.
__device__ __forceinline__ void lose_rows(const Product& p, int row0, int rows, int r, int count, int lane) {
  uint16_t* out = static_cast<uint16_t*>(p.out) + static_cast<int64_t>(row0) * p.R + r;
  for (int row = 0; row < rows; ++row)
    for (int c = lane; c < min(count, p.R - r); c += 32) out[static_cast<int64_t>(row) * p.R + c] = kNaN16;
}

constexpr int kTileBytes = 128 * 128;
enum { kWhereFetch = 1, kWhereProduct = 2, kWhereOut = 3 };

// of several experts: their first rows and first token tiles
struct Groups {
  int begin[kMaxExperts + 1];        // begin[E]: the end of the last expert's rows
  int tile[kMaxExperts + 1];
};
__device__ __forceinline__ void umma_fp8(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}

// The row ranges of the experts, by one warp.  They are data: each start is
// taken as at least the one before it and at most M, so that no range leaves
// the tokens or overlaps another one whatever the values are.
__device__ __forceinline__ void plan_groups(const Product& p, Groups& g, int tile_m, int lane) {
  int first = 0, tiles = 0;
  // begin[e] = min(M, max(0, offsets[0 .. e]))
  for (int e0 = 0; e0 <= p.E; e0 += 32) {
    const int e = e0 + lane;
    int b = e <= p.E ? min(max(p.offsets[e], 0), p.M) : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int up = __shfl_up_sync(0xffffffffu, b, o);
      if (lane >= o) b = max(b, up);
    }
    b = max(b, first);
    first = __shfl_sync(0xffffffffu, b, 31);
    if (e <= p.E) g.begin[e] = b;
  }
  __syncwarp();
  for (int e0 = 0; e0 <= p.E; e0 += 32) {
    const int e = e0 + lane;
    int t = e < p.E ? (g.begin[e + 1] - g.begin[e] + tile_m - 1) / tile_m : 0;
    const int own = t;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int up = __shfl_up_sync(0xffffffffu, t, o);
      if (lane >= o) t += up;
    }
    if (e <= p.E) g.tile[e] = tiles + t - own;
    tiles += __shfl_sync(0xffffffffu, t, 31);
  }
}

struct Tile {
  int e, m0, end, r0;   // expert, first row, end of the expert's rows, first output
};
// Tile t: runs of 8 token tiles for each tile of outputs, so that tiles at
// work together share tokens and weights in L2.
template <int kTileR>
__device__ __forceinline__ Tile tile_at(const Product& p, const Groups& g, int t, int num_m, int num_r, int tile_m) {
  constexpr int kRun = 8;
  const int run = t / (kRun * num_r), first = run * kRun, in = t - run * (kRun * num_r);
  const int width = min(kRun, num_m - first);
  const int rt = width == kRun ? in / kRun : in / width, mt = first + in - rt * width;
  Tile x;
  x.r0 = rt * kTileR;
  if (p.offsets == nullptr) {
    x.e = 0;
    x.m0 = mt * tile_m;
    x.end = p.M;
    return x;
  }
  int lo = 0, hi = p.E;   // the last expert whose first tile is at most mt (experts without rows share it)
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (g.tile[mid] <= mt) lo = mid;
    else hi = mid;
  }
  x.e = lo;
  x.m0 = g.begin[lo] + (mt - g.tile[lo]) * tile_m;
  x.end = g.begin[lo + 1];
  return x;
}

__device__ __forceinline__ uint32_t pack16(bool bf16, float a, float b) {
  if (bf16) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&v);
  }
  const __half2 v = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&v);
}

__device__ __forceinline__ float bias_at(const Product& p, int r) {
  if (p.bias == nullptr || r >= p.R) return 0.f;
  return p.bias_dt == DT_F32    ? static_cast<const float*>(p.bias)[r]
         : p.bias_dt == DT_BF16 ? to_float(static_cast<const __nv_bfloat16*>(p.bias)[r])
                                : to_float(static_cast<const __half*>(p.bias)[r]);
}

// Zeros in the rows of no expert, by warp `w` of `count`.
__device__ __forceinline__ void zero_rest(const Product& p, const Groups& g, int64_t w, int64_t count, int lane) {
  const int64_t head = g.begin[0], rest = head + p.M - g.begin[p.E];
  uint16_t* out = static_cast<uint16_t*>(p.out);
  for (int64_t i = w; i < rest; i += count) {
    uint16_t* row = out + (i < head ? i : i - head + g.begin[p.E]) * p.R;
    for (int c = lane; c < p.R; c += 32) row[c] = 0;
  }
}

// grad_bias from the sums of the row ranges, in their order, by thread `i` of
// `count`.
__device__ __forceinline__ void sum_bias(const Product& p, int64_t i, int64_t count) {
  for (int64_t c = i; c < p.C; c += count) {
    float s = 0.f;
#pragma unroll 8
    for (int k = 0; k < p.ranges; ++k) s += p.partial[static_cast<int64_t>(k) * p.C + c];
    if (p.bias_dt == DT_F32) static_cast<float*>(p.grad_bias)[c] = s;
    else if (p.bias_dt == DT_BF16) static_cast<__nv_bfloat16*>(p.grad_bias)[c] = __float2bfloat16_rn(s);
    else static_cast<__half*>(p.grad_bias)[c] = __float2half_rn(s);
  }
}
__global__ void __launch_bounds__(256) fp8_sum_bias_kernel(const __grid_constant__ Product p) {
  sum_bias(p, static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x, static_cast<int64_t>(gridDim.x) * 256);
}

// 32 outputs from output r on of up to 32 rows, from a warp's shared memory
// (rows of 64 bytes, 16-byte chunks permuted): whole sectors at a time, or, with
// rows off 16-byte boundaries, a row at a time.
__device__ __forceinline__ void write_rows(const Product& p, int row0, int rows, int r, const uint8_t* out_s, int lane) {
  uint16_t* out = static_cast<uint16_t*>(p.out) + static_cast<int64_t>(row0) * p.R + r;
  if (p.vec) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int row = i * 8 + (lane >> 2), c = lane & 3;
      const uint4 v = ld_shared_v4(out_s + row * 64 + ((c ^ ((row >> 1) & 3)) << 4));
      if (row < rows && r + 8 * c < p.R) *reinterpret_cast<uint4*>(out + static_cast<int64_t>(row) * p.R + 8 * c) = v;
    }
  } else {
    for (int row = 0; row < rows; ++row) {
      const uint8_t* src = out_s + row * 64 + (((lane >> 3) ^ ((row >> 1) & 3)) << 4) + (lane & 7) * 2;
      if (r + lane < p.R) out[static_cast<int64_t>(row) * p.R + lane] = *reinterpret_cast<const uint16_t*>(src);
    }
  }
}

constexpr uint32_t kSwizzle64B = 4;

__device__ __forceinline__ void tmem_ld_wait(uint32_t (&a)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;\n" ::: "memory");
#pragma unroll
  for (int i = 0; i < 32; ++i) asm volatile("" : "+r"(a[i]));
}
// two fp32 sums += two products
__device__ __forceinline__ void fma2(uint64_t& acc, uint32_t lo, uint32_t hi, uint64_t scale2) {
  asm("{\n .reg .b64 d;\n mov.b64 d, {%1, %2};\n fma.rn.f32x2 %0, d, %3, %0;\n}" : "+l"(acc) : "r"(lo), "r"(hi), "l"(scale2));
}
__device__ __forceinline__ uint64_t splat2(float f) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %1};" : "=l"(r) : "r"(__float_as_uint(f)));
  return r;
}
__device__ __forceinline__ float2 unpack2(uint64_t v) {
  uint32_t a, b;
  asm("mov.b64 {%0, %1}, %2;" : "=r"(a), "=r"(b) : "l"(v));
  return make_float2(__uint_as_float(a), __uint_as_float(b));
}
__device__ __forceinline__ float4 ld_cluster4(uint32_t a) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(a)
               : "memory");
  return v;
}

// The sum of the same place in every CTA of the cluster, in the order of the
// ranks, with all loads under way.
constexpr int kMaxSplit = 8;
__device__ __forceinline__ float4 cluster_sum(const float* src, int split) {
  float4 part[kMaxSplit];
#pragma unroll
  for (int k = 0; k < kMaxSplit; ++k)
    if (k < split) part[k] = ld_cluster4(mapa_shared(src, static_cast<uint32_t>(k)));
  float4 v = part[0];
#pragma unroll
  for (int k = 1; k < kMaxSplit; ++k)
    if (k < split) {
      v.x += part[k].x;
      v.y += part[k].y;
      v.z += part[k].z;
      v.w += part[k].w;
    }
  return v;
}

// After a wait that ran out: NaN for a CTA's part of its cluster's sums, by its
// epilogue's threads, once nothing more writes to its shared memory.
__device__ __forceinline__ void lose_sums(uint8_t* smem, int count) {
  for (int i = static_cast<int>(threadIdx.x) - 64; i < count; i += 128) reinterpret_cast<float*>(smem)[i] = __int_as_float(0x7fffffff);
}

constexpr int kEpiWarps = 4;         // warps 2 to 5: lanes 32 (w % 4) of the accumulators

// ---- few tokens -----------------------------------------------------------

// Tiles of 128 outputs x kN tokens, kN = 16, 32 or 64: the weight is the first
// operand, an accumulator has kN columns, and the 256 columns of TMEM that a
// CTA takes hold two groups of 128 / kN blocks of the reduction: one hand-over
// between the thread that multiplies and the warps that add for so many blocks
// (one a block costs 400 ns a block, three times what its 16 KB of weight take
// to arrive).  A thread has one output of every token; the scales of a group's
// blocks and tokens lie across the warp's registers, four a lane, fetched a
// group ahead.  Bound by HBM: each weight is read once.  16 tokens, 8192 ->
// 28672: 43 us with the quantizing kernel, 5.5 TB/s (35 us at the rate of a
// copy; the first data arrive 5 us after the start, half of it the launch);
// 128 rows of 64 experts, 4096 -> 2048: 72 us for the 429 MB of the experts that
// have rows.  One token, 4096 -> 11008: 18 us, of which 6.6 are HBM's.
// The weight does not depend on the kernel before, so its first stages are on
// their way while the tokens are being quantized.  With few tiles a cluster of
// `split` CTAs shares a tile: each has a part of the reduction, and the parts
// are added in the order of the ranks.
constexpr int kFewThreads = 192;
template <int kN>
constexpr int few_stages() { return kN == 64 ? 4 : 5; }   // two CTAs an SM
template <int kN>
struct FewShared {
  uint64_t full[few_stages<kN>()], empty[few_stages<kN>()];
  uint64_t acc_full[2], acc_empty[2];   // of a group
  uint64_t last;                        // all products have completed
  uint32_t tmem;
  int abort;
};
template <int kN>
constexpr int few_smem() {
  return 1024 + few_stages<kN>() * (kTileBytes + kN * 128) + static_cast<int>(sizeof(FewShared<kN>));
}

template <bool kT, int kN>
__global__ void __launch_bounds__(kFewThreads, 2) fp8_product_few_kernel(const __grid_constant__ Product p) {
  constexpr int kGroup = 128 / kN;             // blocks
  constexpr int kStageBytes = kTileBytes + kN * 128, kFewStages = few_stages<kN>();
  static_assert(kFewStages * kStageBytes >= kN * 128 * 4, "the sums of a tile fit the stages");
  extern __shared__ uint8_t smem_raw[];
  __shared__ Groups groups;
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  FewShared<kN>& y = *reinterpret_cast<FewShared<kN>*>(smem + kFewStages * kStageBytes);
  volatile int* abort = &y.abort;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = p.split > 1 ? static_cast<int>(cluster_ctarank()) : 0;
  const int first = static_cast<int>(blockIdx.x) / p.split, step = static_cast<int>(gridDim.x) / p.split;

  if (threadIdx.x == 0) {
    for (int i = 0; i < kFewStages; ++i) {
      mbar_init(&y.full[i], 1);
      mbar_init(&y.empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&y.acc_full[i], 1);
      mbar_init(&y.acc_empty[i], kEpiWarps);
    }
    mbar_init(&y.last, 1);
    y.abort = 0;
    fence_mbar_init();
    tma_prefetch_desc(&p.tmX);
    tma_prefetch_desc(&p.tmW);
  }
  if (warp == 1) {
    tmem_alloc(&y.tmem, 256);
    tmem_relinquish();
  }
  if (warp == 2 && p.offsets != nullptr) plan_groups(p, groups, kN, lane);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = y.tmem;
  const int num_m = p.offsets == nullptr ? (p.M + kN - 1) / kN : groups.tile[p.E];
  const int num_r = (p.R + 127) / 128;
  const int tiles = num_m * num_r, all = (p.C + kBlk - 1) / kBlk;
  // this CTA's blocks of a reduction: every `split`th, so that the CTAs of a
  // cluster read neighbouring memory at a time
  const int split = p.split, count = (all - rank + split - 1) / split;

  if (warp == 0) {
    if (lane == 0) {
      auto fetch_w = [&](int s, const Tile& x, int b) {
        uint8_t* wd = smem + s * kStageBytes;
        mbar_arrive_expect_tx(&y.full[s], kStageBytes);
        if (kT) tma_load_3d(wd, &p.tmW, x.r0, b * kBlk, x.e, &y.full[s]);
        else tma_load_3d(wd, &p.tmW, b * kBlk, x.r0, x.e, &y.full[s]);
      };
      int it = 0, ahead = 0;
      bool ok = true;
      if (first < tiles) {
        const Tile x = tile_at<128>(p, groups, first, num_m, num_r, kN);
        ahead = min(kFewStages, count);
        for (int s = 0; s < ahead; ++s) fetch_w(s, x, rank + s * split);
      }
      grid_dependency_wait();
      asm volatile("fence.proxy.async;" ::: "memory");
      for (int t = first; t < tiles && ok; t += step) {
        const Tile x = tile_at<128>(p, groups, t, num_m, num_r, kN);
        for (int b = 0; b < count; ++b, ++it) {
          const int s = it % kFewStages;
          if ((it == max(p.hold, ahead) && !wait_for(p, &y.last, 0, abort, kWhereFetch)) ||
              !wait_for(p, &y.empty[s], ((it / kFewStages) & 1) ^ 1, abort, kWhereFetch)) {
            ok = false;   // not before the fetches ahead have their tokens: those stages are empty
            break;
          }
          if (it >= ahead) fetch_w(s, x, rank + b * split);
          tma_load_2d(smem + s * kStageBytes + kTileBytes, &p.tmX, (rank + b * split) * kBlk, x.m0, &y.full[s]);
        }
      }
      // what is under way lands before the block may end
      for (int j = max(0, it - kFewStages); j < it; ++j)
        mbar_wait_out(&y.full[j % kFewStages], (j / kFewStages) & 1, p.st, kWhereFetch);
    }
  } else if (warp == 1) {
    if (lane == 0) {
      const uint32_t idesc = make_idesc_f16(128, kN, kT, false);   // E4M3 has the format number of fp16
      const uint32_t base = smem_u32(smem);
      int it = 0, grp = 0;
      bool ok = true;
      for (int t = first; t < tiles && ok; t += step) {
        for (int b = 0; b < count && ok; b += kGroup, ++grp) {
          const int a = grp & 1;
          if (!wait_for(p, &y.acc_empty[a], ((grp >> 1) & 1) ^ 1, abort, kWhereProduct)) {
            ok = false;
            break;
          }
          for (int g = 0; g < min(kGroup, count - b); ++g, ++it) {
            const int s = it % kFewStages;
            if (!wait_for(p, &y.full[s], (it / kFewStages) & 1, abort, kWhereProduct)) {
              ok = false;
              break;
            }
            tc_fence_after();
            const uint32_t wa = base + s * kStageBytes, xa = wa + kTileBytes;
#pragma unroll
            for (int k = 0; k < 4; ++k)
              umma_fp8(tmem + a * 128 + g * kN,
                       kT ? make_sdesc(wa + 4096 * k, kTileBytes, 1024, kSwizzle128B)
                          : make_sdesc(wa + 32 * k, 16, 1024, kSwizzle128B),
                       make_sdesc(xa + 32 * k, 16, 1024, kSwizzle128B), idesc, k > 0 ? 1u : 0u);
            umma_commit(&y.empty[s]);
          }
          if (ok) umma_commit(&y.acc_full[a]);
        }
      }
      umma_commit(&y.last);
      mbar_wait_out(&y.last, 0, p.st, kWhereProduct);
    }
  } else {
    const int quad = warp & 3;
    const uint32_t lanes = tmem + (static_cast<uint32_t>(quad * 32) << 16);
    grid_dependency_wait();
    if (p.offsets != nullptr && p.zero_rest)
      zero_rest(p, groups, blockIdx.x * kEpiWarps + quad, gridDim.x * kEpiWarps, lane);
    if (p.partial != nullptr)
      sum_bias(p, (static_cast<int64_t>(blockIdx.x) * kEpiWarps + quad) * 32 + lane, static_cast<int64_t>(gridDim.x) * kEpiWarps * 32);
    int grp = 0, t = first;
    bool ok = true;
    for (; t < tiles; t += step) {
      const Tile x = tile_at<128>(p, groups, t, num_m, num_r, kN);
      const int r = x.r0 + quad * 32 + lane;
      const float* ws = p.ws + static_cast<int64_t>(x.e) * p.nb * p.kb + (kT ? x.r0 / kBlk : x.r0 / kBlk * p.kb);
      const int wstep = kT ? p.kb : 1;
      const float bias = bias_at(p, r);
      float acc[kN];
#pragma unroll
      for (int i = 0; i < kN; ++i) acc[i] = 0.f;
      // the scales of a group: block g, token j at place g kN + j of 128, four a lane
      float xv[4], wv[4];
      auto fetch = [&](int b) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int at = i * 32 + lane, blk = rank + min(b + at / kN, count - 1) * split;
          xv[i] = p.xs[static_cast<int64_t>(blk) * p.M + min(x.m0 + at % kN, p.M - 1)];
          wv[i] = ws[static_cast<int64_t>(blk) * wstep];
        }
      };
      if (count > 0) fetch(0);
      for (int b = 0; b < count; b += kGroup, ++grp) {
        const int a = grp & 1;
        float s[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) s[i] = xv[i] * wv[i];
        if (b + kGroup < count) fetch(b + kGroup);
        if (!__all_sync(0xffffffffu, wait_for(p, &y.acc_full[a], (grp >> 1) & 1, abort, kWhereOut))) {
          ok = false;
          break;
        }
        tc_fence_after();
        uint32_t d[2][32];
        tmem_ld32_nowait(lanes + a * 128, d[0]);
#pragma unroll
        for (int c = 0; c < 4; ++c) {   // 32 columns: 32 / kN blocks, or a part of one
          tmem_ld_wait(d[c & 1]);
          if (c < 3) {
            tmem_ld32_nowait(lanes + a * 128 + 32 * (c + 1), d[(c + 1) & 1]);
          } else {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&y.acc_empty[a]);
          }
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            const float scale = __shfl_sync(0xffffffffu, s[c], i);
            // columns of blocks past the last hold an older group's products
            if (b + (32 * c + i) / kN < count)
              acc[(32 * c + i) % kN] = fmaf(__uint_as_float(d[c & 1][i]), scale, acc[(32 * c + i) % kN]);
          }
        }
      }
      if (!ok) break;
      if (split > 1) {
        // all of this CTA's products have completed: its stages hold the sums now, [token][output]
        float* dst = reinterpret_cast<float*>(smem) + quad * 32 + lane;
#pragma unroll
        for (int i = 0; i < kN; ++i) dst[i * 128] = acc[i];
      } else if (r < p.R) {
        uint16_t* dst = static_cast<uint16_t*>(p.out) + static_cast<int64_t>(x.m0) * p.R + r;
#pragma unroll
        for (int i = 0; i < kN; ++i)
          if (x.m0 + i < x.end) dst[static_cast<int64_t>(i) * p.R] = static_cast<uint16_t>(pack16(p.bf16, acc[i] + bias, 0.f));
      }
    }
    if (split == 1)   // the tiles that a wait that ran out cut off
      for (; t < tiles; t += step) {
        const Tile x = tile_at<128>(p, groups, t, num_m, num_r, kN);
        lose_rows(p, x.m0, min(kN, x.end - x.m0), x.r0 + quad * 32, 32, lane);
      }
  }
  if (split > 1) {
    // one tile a cluster; every rank adds up its share of the tokens, a warp
    // four outputs a lane
    __syncthreads();
    if (warp >= 2 && *abort) lose_sums(smem, kN * 128);
    cluster_sync();
    if (warp >= 2 && first < tiles) {
      const Tile x = tile_at<128>(p, groups, first, num_m, num_r, kN);
      const int r = x.r0 + 4 * lane;
      for (int i = rank * kEpiWarps + warp - 2; i < min(kN, x.end - x.m0); i += split * kEpiWarps) {
        if (r >= p.R) continue;
        const float* src = reinterpret_cast<const float*>(smem) + i * 128 + 4 * lane;
        const float4 v = cluster_sum(src, split);
        const uint32_t q[2] = {pack16(p.bf16, v.x + bias_at(p, r), v.y + bias_at(p, r + 1)),
                               pack16(p.bf16, v.z + bias_at(p, r + 2), v.w + bias_at(p, r + 3))};
        uint16_t* dst = static_cast<uint16_t*>(p.out) + static_cast<int64_t>(x.m0 + i) * p.R + r;
        if (p.vec) {
          *reinterpret_cast<uint2*>(dst) = make_uint2(q[0], q[1]);
        } else {
#pragma unroll
          for (int k = 0; k < 4; ++k)
            if (r + k < p.R) dst[k] = static_cast<uint16_t>(q[k >> 1] >> (16 * (k & 1)));
        }
      }
    }
    cluster_sync();   // no CTA leaves while another reads its sums
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, 256);
}

// ---- small products -------------------------------------------------------

constexpr int kThreads = 192;
constexpr int kStoreBytes = 2048;    // per epilogue warp: 32 rows of 32 outputs on their way out
constexpr int kMaxStages = 8;
constexpr int kTileR = 64;           // outputs of a tile
struct Shared {
  uint64_t full[kMaxStages], empty[kMaxStages];
  uint64_t acc_full[2], acc_empty[2];
  uint64_t last;                     // all products have completed
  uint32_t tmem;
  int abort;
  float bias[kEpiWarps][kTileR];
};
constexpr int small_smem(int stages) {
  return 1024 + stages * (128 + kTileR) * 128 + kEpiWarps * kStoreBytes + static_cast<int>(sizeof(Shared));
}

// Tiles of 128 tokens x 64 outputs, two CTAs an SM.  Warp 0 fetches, warp 1
// multiplies: one accumulator in TMEM per 128 columns of the reduction, two of
// them in turn.  Warps 2 to 5 add each, times its two scales, to the sums that
// they hold in registers: a thread has one token and kTileR outputs, so the
// product of the scales is one number.  The weight does not depend on the
// kernel before, so its first stages are on their way while the tokens are
// being quantized.  With few tiles a cluster of `split` CTAs shares a tile:
// each has a part of the reduction, and the parts are added in the order of
// the ranks.  Bound by latency: 777 tokens, 1100 -> 519: 13 us, of which 5 are
// the launch and the first data, and 3 the cluster's sums.
template <bool kT>
__global__ void __launch_bounds__(kThreads, 2) fp8_product_kernel(const __grid_constant__ Product p) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ Groups groups;
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  constexpr int kTileM = 128, x_bytes = kTileBytes, stage_bytes = x_bytes + kTileR * 128;
  const int stages = p.stages;
  Shared& y = *reinterpret_cast<Shared*>(smem + stages * stage_bytes + kEpiWarps * kStoreBytes);
  volatile int* abort = &y.abort;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = p.split > 1 ? static_cast<int>(cluster_ctarank()) : 0;
  const int first = static_cast<int>(blockIdx.x) / p.split, step = static_cast<int>(gridDim.x) / p.split;

  if (threadIdx.x == 0) {
    for (int i = 0; i < stages; ++i) {
      mbar_init(&y.full[i], 1);
      mbar_init(&y.empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&y.acc_full[i], 1);
      mbar_init(&y.acc_empty[i], kEpiWarps);
    }
    mbar_init(&y.last, 1);
    y.abort = 0;
    fence_mbar_init();
    tma_prefetch_desc(&p.tmX);
    tma_prefetch_desc(&p.tmW);
  }
  if (warp == 1) {
    tmem_alloc(&y.tmem, 2 * kTileR);
    tmem_relinquish();
  }
  if (warp == 2 && p.offsets != nullptr) plan_groups(p, groups, kTileM, lane);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = y.tmem;
  const int num_m = p.offsets == nullptr ? (p.M + kTileM - 1) / kTileM : groups.tile[p.E];
  const int num_r = (p.R + kTileR - 1) / kTileR;
  const int tiles = num_m * num_r, all = (p.C + kBlk - 1) / kBlk;
  const int b0 = all * rank / p.split, b1 = all * (rank + 1) / p.split;   // this CTA's blocks of a reduction

  if (warp == 0) {
    if (lane == 0) {
      auto fetch_w = [&](int s, const Tile& x, int b) {
        uint8_t* wd = smem + s * stage_bytes + x_bytes;
        mbar_arrive_expect_tx(&y.full[s], stage_bytes);
        if (kT) tma_load_3d(wd, &p.tmW, x.r0, b * kBlk, x.e, &y.full[s]);
        else tma_load_3d(wd, &p.tmW, b * kBlk, x.r0, x.e, &y.full[s]);
      };
      int it = 0, ahead = 0;
      bool ok = true;
      if (first < tiles) {
        const Tile x = tile_at<kTileR>(p, groups, first, num_m, num_r, kTileM);
        ahead = min(stages, b1 - b0);
        for (int s = 0; s < ahead; ++s) fetch_w(s, x, b0 + s);
      }
      grid_dependency_wait();
      asm volatile("fence.proxy.async;" ::: "memory");
      for (int t = first; t < tiles && ok; t += step) {
        const Tile x = tile_at<kTileR>(p, groups, t, num_m, num_r, kTileM);
        for (int b = b0; b < b1; ++b, ++it) {
          const int s = it % stages;
          if ((it == max(p.hold, ahead) && !wait_for(p, &y.last, 0, abort, kWhereFetch)) ||
              !wait_for(p, &y.empty[s], ((it / stages) & 1) ^ 1, abort, kWhereFetch)) {
            ok = false;   // not before the fetches ahead have their tokens: those stages are empty
            break;
          }
          if (it >= ahead) fetch_w(s, x, b);
          tma_load_2d(smem + s * stage_bytes, &p.tmX, b * kBlk, x.m0, &y.full[s]);
        }
      }
      // what is under way lands before the block may end
      for (int j = max(0, it - stages); j < it; ++j) mbar_wait_out(&y.full[j % stages], (j / stages) & 1, p.st, kWhereFetch);
    }
  } else if (warp == 1) {
    if (lane == 0) {
      const uint32_t idesc = make_idesc_f16(128, kTileR, false, kT);   // E4M3 has the format number of fp16
      const uint32_t base = smem_u32(smem);
      int it = 0;
      bool ok = true;
      for (int t = first; t < tiles && ok; t += step) {
        for (int b = b0; b < b1; ++b, ++it) {
          const int s = it % stages, a = it & 1;
          if (!wait_for(p, &y.full[s], (it / stages) & 1, abort, kWhereProduct) ||
              !wait_for(p, &y.acc_empty[a], ((it >> 1) & 1) ^ 1, abort, kWhereProduct)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t xa = base + s * stage_bytes, wa = xa + x_bytes;
#pragma unroll
          for (int k = 0; k < 4; ++k)
            umma_fp8(tmem + a * kTileR, make_sdesc(xa + 32 * k, 16, 1024, kSwizzle128B),
                     kT ? make_sdesc(wa + 2048 * k, kTileR * 128, 512, kSwizzle64B)
                        : make_sdesc(wa + 32 * k, 16, 1024, kSwizzle128B),
                     idesc, k > 0 ? 1u : 0u);
          umma_commit(&y.acc_full[a]);
          umma_commit(&y.empty[s]);
        }
      }
      umma_commit(&y.last);
      mbar_wait_out(&y.last, 0, p.st, kWhereProduct);
    }
  } else {
    const int quad = warp & 3;
    const uint32_t lanes = tmem + (static_cast<uint32_t>(quad * 32) << 16);
    float* bias_s = y.bias[quad];
    uint8_t* out_s = smem + stages * stage_bytes + quad * kStoreBytes;
    grid_dependency_wait();
    if (p.offsets != nullptr && p.zero_rest)
      zero_rest(p, groups, blockIdx.x * kEpiWarps + quad, gridDim.x * kEpiWarps, lane);
    if (p.partial != nullptr)
      sum_bias(p, (static_cast<int64_t>(blockIdx.x) * kEpiWarps + quad) * 32 + lane, static_cast<int64_t>(gridDim.x) * kEpiWarps * 32);
    const int wstep = kT ? p.kb : 1;
    int it = 0, t = first;
    bool ok = true;
    for (; t < tiles; t += step) {
      const Tile x = tile_at<kTileR>(p, groups, t, num_m, num_r, kTileM);
      const int last = min(x.end, x.m0 + kTileM), row0 = x.m0 + quad * 32, m = row0 + lane;
      const bool any = row0 < last;   // a warp without tokens hands the accumulators on
      const float* xs = p.xs + static_cast<int64_t>(b0) * p.M + min(m, p.M - 1);
      const float* ws = p.ws + static_cast<int64_t>(x.e) * p.nb * p.kb + (kT ? x.r0 / kBlk : x.r0 / kBlk * p.kb) +
                        static_cast<int64_t>(b0) * wstep;
      uint64_t acc[kTileR / 2];
#pragma unroll
      for (int i = 0; i < kTileR / 2; ++i) acc[i] = 0;
      float bias[kTileR / 32];   // used at the tile's end
#pragma unroll
      for (int i = 0; i < kTileR / 32; ++i) bias[i] = any ? bias_at(p, x.r0 + lane + 32 * i) : 0.f;
      // the scales are fetched two blocks ahead and multiplied when they are used
      float x1 = 0.f, w1 = 0.f, x2 = 0.f, w2 = 0.f;
      if (any && b0 < b1) {
        x1 = xs[0];
        w1 = ws[0];
        if (b0 + 1 < b1) {
          x2 = xs[p.M];
          w2 = ws[wstep];
        }
      }
      for (int b = 0; b < b1 - b0; ++b, ++it) {
        const int a = it & 1;
        if (!__all_sync(0xffffffffu, wait_for(p, &y.acc_full[a], (it >> 1) & 1, abort, kWhereOut))) {
          ok = false;
          break;
        }
        if (any) {
          tc_fence_after();
          uint32_t d[32];
          tmem_ld32_nowait(lanes + a * kTileR, d);
          const uint64_t scale = splat2(x1 * w1);
          x1 = x2;
          w1 = w2;
          if (b + 2 < b1 - b0) {
            x2 = xs[static_cast<int64_t>(b + 2) * p.M];
            w2 = ws[static_cast<int64_t>(b + 2) * wstep];
          }
#pragma unroll
          for (int c = 0; c < kTileR / 32; ++c) {
            tmem_ld_wait(d);
#pragma unroll
            for (int i = 0; i < 16; ++i) fma2(acc[16 * c + i], d[2 * i], d[2 * i + 1], scale);
            if (c + 1 < kTileR / 32) tmem_ld32_nowait(lanes + a * kTileR + 32 * (c + 1), d);
          }
          tc_fence_before();
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&y.acc_empty[a]);
      }
      if (!ok) break;
      if (p.split > 1) {
        // all of this CTA's products have completed: its stages hold the sums
        // now, one row of the tile after another, 16-byte chunks permuted
        const int row = quad * 32 + lane;
        if (row < kTileM) {
          float4* dst = reinterpret_cast<float4*>(smem) + row * (kTileR / 4);
#pragma unroll
          for (int i = 0; i < kTileR / 4; ++i) {
            const float2 lo = unpack2(acc[2 * i]), hi = unpack2(acc[2 * i + 1]);
            dst[i ^ (row & 7)] = make_float4(lo.x, lo.y, hi.x, hi.y);
          }
        }
      } else if (any) {
        __syncwarp();
#pragma unroll
        for (int i = 0; i < kTileR / 32; ++i) bias_s[lane + 32 * i] = bias[i];
        __syncwarp();
        // through shared memory, 32 outputs of 32 rows at a time, so that rows
        // are written in whole sectors
#pragma unroll
        for (int h = 0; h < kTileR / 32; ++h) {
          if (x.r0 + 32 * h >= p.R) break;
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const float4 lo = *reinterpret_cast<const float4*>(bias_s + 32 * h + 8 * c);
            const float4 hi = *reinterpret_cast<const float4*>(bias_s + 32 * h + 8 * c + 4);
            const float bv[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
            uint32_t q[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const float2 v = unpack2(acc[16 * h + 4 * c + k]);
              q[k] = pack16(p.bf16, v.x + bv[2 * k], v.y + bv[2 * k + 1]);
            }
            st_shared_v4(out_s + lane * 64 + ((c ^ ((lane >> 1) & 3)) << 4), make_uint4(q[0], q[1], q[2], q[3]));
          }
          __syncwarp();
          const int r = x.r0 + 32 * h;
          write_rows(p, row0, min(32, last - row0), r, out_s, lane);
          __syncwarp();
        }
        __syncwarp();
      }
    }
    if (p.split == 1)   // the tiles that a wait that ran out cut off
      for (; t < tiles; t += step) {
        const Tile x = tile_at<kTileR>(p, groups, t, num_m, num_r, kTileM);
        const int row0 = x.m0 + quad * 32;
        lose_rows(p, row0, min(32, min(x.end, x.m0 + kTileM) - row0), x.r0, kTileR, lane);
      }
  }
  if (p.split > 1) {
    // one tile a cluster; every rank adds up its share of the tile, 4 outputs
    // at a time
    __syncthreads();
    if (warp >= 2 && *abort) lose_sums(smem, kTileM * kTileR);
    cluster_sync();
    if (warp >= 2 && first < tiles) {
      const Tile x = tile_at<kTileR>(p, groups, first, num_m, num_r, kTileM);
      const int rows = min(kTileM, x.end - x.m0), count = rows * (kTileR / 4);
      for (int g = rank * (kEpiWarps * 32) + static_cast<int>(threadIdx.x) - 64; g < count; g += p.split * kEpiWarps * 32) {
        const int row = g / (kTileR / 4), i = g % (kTileR / 4), r = x.r0 + 4 * i;
        if (r >= p.R) continue;
        const float* src = reinterpret_cast<const float*>(smem) + 4 * (row * (kTileR / 4) + (i ^ (row & 7)));
        const float4 v = cluster_sum(src, p.split);
        const uint32_t q[2] = {pack16(p.bf16, v.x + bias_at(p, r), v.y + bias_at(p, r + 1)),
                               pack16(p.bf16, v.z + bias_at(p, r + 2), v.w + bias_at(p, r + 3))};
        uint16_t* dst = static_cast<uint16_t*>(p.out) + static_cast<int64_t>(x.m0 + row) * p.R + r;
        if (p.vec) {
          *reinterpret_cast<uint2*>(dst) = make_uint2(q[0], q[1]);
        } else {
#pragma unroll
          for (int k = 0; k < 4; ++k)
            if (r + k < p.R) dst[k] = static_cast<uint16_t>(q[k >> 1] >> (16 * (k & 1)));
        }
      }
    }
    cluster_sync();   // no CTA leaves while another reads its sums
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, 2 * kTileR);
}

// ---- many tokens ----------------------------------------------------------

constexpr int kWideThreads = 384;
constexpr int kWideEpiWarps = 8;          // warps 4 to 11
constexpr int kWideStages = 4;
constexpr int kWideStageBytes = 3 * kTileBytes;
constexpr int kWideCols = 128;            // outputs of an epilogue warp
constexpr int kWideStoreBytes = 2048;     // per epilogue warp: 32 rows of 32 outputs
// Registers a thread: 168 at launch (384 x 168 = 64512); of those the first
// four warps keep 40 and the epilogue's take 232 (128 x 40 + 256 x 232 = 64512).
constexpr int kWideRegs = 40, kWideEpiRegs = 232;
static_assert(128 * kWideRegs + 256 * kWideEpiRegs <= kWideThreads * 168, "register split");
constexpr int kScaleRing = 8;             // blocks whose scales are in shared memory
constexpr int kScaleAhead = 6;            // ... of which so many are on their way
struct WideShared {
  uint64_t full[kWideStages], empty[kWideStages];
  uint64_t acc_full[2];                   // an accumulator is there, and the scales of its block and the next
  uint64_t acc_empty[2];                  // it has been read
  uint64_t scale_read[2];                 // the next block's scales have been read
  uint64_t last;
  uint32_t tmem;
  int abort;
  float bias[kWideEpiWarps][kWideCols];
  float xs[kScaleRing][128], ws[kScaleRing][2];
};
constexpr int kWideSmemBytes = 1024 + kWideStages * kWideStageBytes + kWideEpiWarps * kWideStoreBytes + static_cast<int>(sizeof(WideShared));

// whether the phase has completed, without waiting for it
__device__ __forceinline__ bool mbar_test(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n .reg .pred p;\n"
      " mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n"
      " selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}
__device__ __forceinline__ void cp_async4(void* dst, const float* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int kPending>
__device__ __forceinline__ void cp_async_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(kPending) : "memory"); }

template <int kRegs>
__device__ __forceinline__ void keep_registers() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegs)); }
template <int kRegs>
__device__ __forceinline__ void take_registers() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegs)); }
// Tiles of 128 tokens x 256 outputs; two accumulators in turn fill TMEM, and
// eight warps keep the sums in registers (128 outputs a thread).
// What bounds it is how fast an accumulator is handed back: a block's product
// takes 512 clocks, its loads from TMEM and multiply-adds 750, of which 420 are
// the 128 packed multiply-adds of each scheduler (3.3 clocks each) and the rest
// latencies of barriers and shared memory that its two warps do not hide.  So
// the epilogue keeps a load under way at all times, asks for the next
// accumulator before it needs it and has its scales one block early; two
// threads multiply in turn, each for one accumulator, since a wait costs over a
// tenth of a block's product even when there is nothing to wait for; and warp 3
// brings the scales to shared memory, blocks and tiles ahead.  Writing a tile
// out takes 5000 clocks more, of which the tensor cores fill two blocks' worth.
// 4096 tokens, 4096 -> 11008: 162 us, 2.3 PFLOP/s; 16384 tokens, 8192 -> 28672:
// 3.1 ms forward, 3.0 ms backward, 2.5 PFLOP/s at 1.5 to 1.6 GHz under the power
// limit (59 % and 65 % of twice the 16-bit rate).
template <bool kT>
__global__ void __launch_bounds__(kWideThreads, 1) fp8_product_wide_kernel(const __grid_constant__ Product p) {
  constexpr int kTileM = 128, kTileR = 256;
  extern __shared__ uint8_t smem_raw[];
  __shared__ Groups groups;
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* store = smem + kWideStages * kWideStageBytes;
  WideShared& y = *reinterpret_cast<WideShared*>(store + kWideEpiWarps * kWideStoreBytes);
  volatile int* abort = &y.abort;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int first = blockIdx.x, step = gridDim.x;

  if (threadIdx.x == 0) {
    for (int i = 0; i < kWideStages; ++i) {
      mbar_init(&y.full[i], 1);
      mbar_init(&y.empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&y.acc_full[i], 2);
      mbar_init(&y.acc_empty[i], kWideEpiWarps);
      mbar_init(&y.scale_read[i], kWideEpiWarps);
    }
    mbar_init(&y.last, 2);
    y.abort = 0;
    fence_mbar_init();
    tma_prefetch_desc(&p.tmX);
    tma_prefetch_desc(&p.tmW);
    if (p.vec) tma_prefetch_desc(&p.tmOut);
  }
  if (warp == 1) {
    tmem_alloc(&y.tmem, 512);
    tmem_relinquish();
  }
  if (warp == 4 && p.offsets != nullptr) plan_groups(p, groups, kTileM, lane);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = y.tmem;
  const int num_m = p.offsets == nullptr ? (p.M + kTileM - 1) / kTileM : groups.tile[p.E];
  const int num_r = (p.R + kTileR - 1) / kTileR;
  const int tiles = num_m * num_r, blocks = (p.C + kBlk - 1) / kBlk;

  if (warp < 4) {
    keep_registers<kWideRegs>();
    const int total = first < tiles ? ((tiles - 1 - first) / step + 1) * blocks : 0;   // of all of this CTA's tiles
    if (warp == 0 && lane == 0) {
      grid_dependency_wait();
      asm volatile("fence.proxy.async;" ::: "memory");
      int it = 0;
      bool ok = true;
      for (int t = first; t < tiles && ok; t += step) {
        const Tile x = tile_at<kTileR>(p, groups, t, num_m, num_r, kTileM);
        // by tiles: a test of every fetch costs 0.5 % of 4096 tokens, 4096 -> 11008
        if (it >= p.hold && !wait_for(p, &y.last, 0, abort, kWhereFetch)) break;
        for (int b = 0; b < blocks; ++b, ++it) {
          const int s = it % kWideStages;
          if (!wait_for(p, &y.empty[s], ((it / kWideStages) & 1) ^ 1, abort, kWhereFetch)) {
            ok = false;
            break;
          }
          uint8_t* xd = smem + s * kWideStageBytes;
          mbar_arrive_expect_tx(&y.full[s], kWideStageBytes);
          tma_load_2d(xd, &p.tmX, b * kBlk, x.m0, &y.full[s]);
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            uint8_t* wd = xd + (1 + i) * kTileBytes;
            if (kT) tma_load_3d(wd, &p.tmW, x.r0 + 128 * i, b * kBlk, x.e, &y.full[s]);
            else tma_load_3d(wd, &p.tmW, b * kBlk, x.r0 + 128 * i, x.e, &y.full[s]);
          }
        }
      }
      // what is under way lands before the block may end
      for (int j = max(0, it - kWideStages); j < it; ++j)
        mbar_wait_out(&y.full[j % kWideStages], (j / kWideStages) & 1, p.st, kWhereFetch);
    }
    if ((warp == 1 || warp == 2) && lane == 0) {
      const uint32_t idesc = make_idesc_f16(kTileM, kTileR, false, kT);   // E4M3 has the format number of fp16
      const uint32_t base = smem_u32(smem);
      const int a = warp - 1;
      const uint32_t acc = tmem + a * kTileR;
      for (int it = a; it < total; it += 2) {
        const int s = it % kWideStages;
        if (!wait_for(p, &y.full[s], (it / kWideStages) & 1, abort, kWhereProduct) ||
            !wait_for(p, &y.acc_empty[a], ((it >> 1) & 1) ^ 1, abort, kWhereProduct))
          break;
        tc_fence_after();
        const uint32_t xa = base + s * kWideStageBytes, wa = xa + kTileBytes;
#pragma unroll
        for (int k = 0; k < 4; ++k)
          umma_fp8(acc, make_sdesc(xa + 32 * k, 16, 1024, kSwizzle128B),
                   kT ? make_sdesc(wa + 4096 * k, kTileBytes, 1024, kSwizzle128B)
                      : make_sdesc(wa + 32 * k, 16, 1024, kSwizzle128B),
                   idesc, k > 0 ? 1u : 0u);
        umma_commit(&y.acc_full[a]);
        umma_commit(&y.empty[s]);
      }
      umma_commit(&y.last);
      mbar_wait_out(&y.last, 0, p.st, kWhereProduct);
    }
    if (warp == 3) {
      grid_dependency_wait();
      int ft = first, fb = 0, fi = 0;   // the next block to fetch: its tile, its number there and in all
      int rows[4];
      const float* ws = p.ws;
      auto aim = [&]() {
        if (ft >= tiles) return;
        const Tile x = tile_at<kTileR>(p, groups, ft, num_m, num_r, kTileM);
#pragma unroll
        for (int i = 0; i < 4; ++i) rows[i] = min(x.m0 + i * 32 + lane, p.M - 1);
        const int rb = min(x.r0 / kBlk + (lane & 1), (p.R - 1) / kBlk);
        ws = p.ws + static_cast<int64_t>(x.e) * p.nb * p.kb + (kT ? rb : rb * p.kb);
      };
      auto fetch = [&]() {
        if (ft < tiles) {
          const int s = fi % kScaleRing;
          const float* xs = p.xs + static_cast<int64_t>(fb) * p.M;
#pragma unroll
          for (int i = 0; i < 4; ++i) cp_async4(&y.xs[s][i * 32 + lane], xs + rows[i]);
          if (lane < 2) cp_async4(&y.ws[s][lane], ws);
          ws += kT ? p.kb : 1;
          ++fi;
          if (++fb == blocks) {
            fb = 0;
            ft += step;
            aim();
          }
        }
        cp_async_commit();
      };
      aim();
      for (int i = 0; i < kScaleAhead; ++i) fetch();
      for (int it = 0; it < total; ++it) {
        // with block it - 2 the scales of block it - 1 have been read; this
        // fetch takes the place of an older one's
        static_assert(kScaleAhead + 1 <= kScaleRing - 1, "scale ring");
        if (!__all_sync(0xffffffffu, wait_for(p, &y.scale_read[it & 1], ((it >> 1) & 1) ^ 1, abort, kWhereOut))) break;
        fetch();
        cp_async_wait<kScaleAhead - 1>();   // block it + 1 is there
        __syncwarp();
        if (lane == 0) mbar_arrive(&y.acc_full[it & 1]);
      }
      cp_async_wait<0>();
    }
  } else {
    take_registers<kWideEpiRegs>();
    const int quad = warp & 3, ew = warp - 4, half = ew >> 2;   // its lanes, and half of the outputs
    const uint32_t lanes = tmem + (static_cast<uint32_t>(quad * 32) << 16) + half * kWideCols;
    uint8_t* out_s = store + ew * kWideStoreBytes;
    float* bias_s = y.bias[ew];
    grid_dependency_wait();
    if (p.offsets != nullptr && p.zero_rest)
      zero_rest(p, groups, blockIdx.x * kWideEpiWarps + ew, gridDim.x * kWideEpiWarps, lane);
    if (p.partial != nullptr)
      sum_bias(p, (static_cast<int64_t>(blockIdx.x) * kWideEpiWarps + ew) * 32 + lane, static_cast<int64_t>(gridDim.x) * kWideEpiWarps * 32);
    int it = 0, t = first;
    bool ok = true;
    float now = 0.f;   // the product of the scales of block it
    auto scale_of = [&](int i) { return y.xs[i % kScaleRing][quad * 32 + lane] * y.ws[i % kScaleRing][half]; };
    auto wait = [&]() { return __all_sync(0xffffffffu, wait_for(p, &y.acc_full[it & 1], (it >> 1) & 1, abort, kWhereOut)); };
    for (; t < tiles; t += step) {
      const Tile x = tile_at<kTileR>(p, groups, t, num_m, num_r, kTileM);
      const int row0 = x.m0 + quad * 32, r0 = x.r0 + half * kWideCols;
      float bias[4];   // used at the tile's end
#pragma unroll
      for (int i = 0; i < 4; ++i) bias[i] = bias_at(p, r0 + lane + 32 * i);
      uint64_t acc[kWideCols / 2];
#pragma unroll
      for (int i = 0; i < kWideCols / 2; ++i) acc[i] = 0;
      uint32_t d[2][32];
      if (!(ok = wait())) break;
      tc_fence_after();
      tmem_ld32_nowait(lanes + (it & 1) * kTileR, d[0]);
      if (it == 0) now = scale_of(0);
      for (int b = 0; b < blocks; ++b) {
        const int a = it & 1;
        const uint64_t scale = splat2(now);
        bool ready = true;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          tmem_ld_wait(d[c & 1]);
          if (c < 3) tmem_ld32_nowait(lanes + a * kTileR + 32 * (c + 1), d[(c + 1) & 1]);
          if (c == 1) {
            now = scale_of(it + 1);
            ready = mbar_test(&y.acc_full[a ^ 1], ((it + 1) >> 1) & 1);
          }
          if (c == 3) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
              mbar_arrive(&y.acc_empty[a]);
              mbar_arrive(&y.scale_read[a]);
            }
            ++it;
            if (b + 1 < blocks) {
              if (!__all_sync(0xffffffffu, ready)) ok = wait();
              if (!ok) break;
              tc_fence_after();
              tmem_ld32_nowait(lanes + (a ^ 1) * kTileR, d[0]);
            }
          }
#pragma unroll
          for (int i = 0; i < 16; ++i) fma2(acc[16 * c + i], d[c & 1][2 * i], d[c & 1][2 * i + 1], scale);
        }
        if (!ok) break;
      }
      if (!ok) break;
      // out through shared memory, 32 outputs of 32 rows at a time
#pragma unroll
      for (int i = 0; i < 4; ++i) bias_s[lane + 32 * i] = bias[i];
      const bool inside = p.vec && row0 + 32 <= x.end;
#pragma unroll
      for (int h = 0; h < kWideCols / 32; ++h) {
        if (lane == 0) bulk_wait_read<0>();   // the store ahead has left the buffer
        __syncwarp();
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          uint32_t q[4];
          const float4 b0 = *reinterpret_cast<const float4*>(bias_s + h * 32 + c * 8);
          const float4 b1 = *reinterpret_cast<const float4*>(bias_s + h * 32 + c * 8 + 4);
          const float bv[8] = {b0.x, b0.y, b0.z, b0.w, b1.x, b1.y, b1.z, b1.w};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float2 v = unpack2(acc[h * 16 + c * 4 + i]);
            q[i] = pack16(p.bf16, v.x + bv[2 * i], v.y + bv[2 * i + 1]);
          }
          st_shared_v4(out_s + lane * 64 + ((c ^ ((lane >> 1) & 3)) << 4), make_uint4(q[0], q[1], q[2], q[3]));
        }
        const int r = r0 + h * 32;
        if (inside) {   // outputs past the last are not written
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0 && r < p.R) {
            tma_store_2d(&p.tmOut, r, row0, out_s);
            bulk_commit();
          }
        } else {
          __syncwarp();
          write_rows(p, row0, min(32, x.end - row0), r, out_s, lane);
        }
      }
      __syncwarp();
    }
    for (; t < tiles; t += step) {   // the tiles that a wait that ran out cut off
      const Tile x = tile_at<kTileR>(p, groups, t, num_m, num_r, kTileM);
      const int row0 = x.m0 + quad * 32;
      lose_rows(p, row0, min(32, x.end - row0), x.r0 + half * kWideCols, kWideCols, lane);
    }
    if (lane == 0) bulk_wait_all();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, 512);
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------

// SMs of the current device, asked for once per device.
int sm_count() {
  static std::atomic<int> known[64];
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev < 0 || dev >= 64) return 152;
  int n = known[dev].load(std::memory_order_relaxed);
  if (n == 0) {
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n < 1) n = 152;
    known[dev].store(n, std::memory_order_relaxed);
  }
  return n;
}

// partial: NULL, or room for the sums of quantize_ranges(M, C) row ranges.
template <typename T>
cudaError_t launch_quantize_typed(const T* x, int64_t M, int64_t C, uint8_t* codes, float* scales, float* partial,
                                  DevStatus* st, cudaStream_t s) {
  const bool vec = C % (16 / static_cast<int>(sizeof(T))) == 0;
  const int c = static_cast<int>(C), ld = static_cast<int>(code_ld(C)), rows = static_cast<int>(quantize_rows(M, C));
  const dim3 grid(static_cast<unsigned>(ceil_div(C, 512)), static_cast<unsigned>(quantize_ranges(M, C)));
  ProfScope ps(K_FP8_QUANTIZE, s);
  if (partial != nullptr) fp8_quantize_kernel<T, true><<<grid, 256, 0, s>>>(x, M, c, ld, vec, rows, codes, scales, partial, st);
  else fp8_quantize_kernel<T, false><<<grid, 256, 0, s>>>(x, M, c, ld, vec, rows, codes, scales, partial, st);
  return cudaGetLastError();
}
cudaError_t launch_quantize(const void* x, int xt, int64_t M, int64_t C, uint8_t* codes, float* scales, float* partial,
                            DevStatus* st, cudaStream_t s) {
  if (xt == DT_F16) return launch_quantize_typed(static_cast<const __half*>(x), M, C, codes, scales, partial, st, s);
  if (xt == DT_BF16) return launch_quantize_typed(static_cast<const __nv_bfloat16*>(x), M, C, codes, scales, partial, st, s);
  return launch_quantize_typed(static_cast<const float*>(x), M, C, codes, scales, partial, st, s);
}

// The kernel after the quantising one: it sets itself up while that one runs.
cudaError_t launch_after(void (*kernel)(Product), int64_t grid, int threads, int smem, int cluster, const Product& p,
                         cudaStream_t s) {
  if (!ensure_smem_attr(reinterpret_cast<const void*>(kernel), smem)) return cudaGetLastError();
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(grid));
  cfg.blockDim = dim3(static_cast<unsigned>(threads));
  cfg.dynamicSmemBytes = static_cast<size_t>(smem);
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(cluster);
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  ProfScope ps(K_FP8_GEMM, s);
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

// The tensor maps of a variant whose boxes have `rows` tokens and `outputs`
// outputs (of one block of the reduction).
bool make_maps(Product& p, bool kt, const void* x, const void* w, int rows, int outputs) {
  const int64_t N = kt ? p.C : p.R, K = kt ? p.R : p.C;
  const CUtensorMapDataType u8 = CU_TENSOR_MAP_DATA_TYPE_UINT8;
  return make_tmap(&p.tmX, u8, x, code_ld(p.C), p.M, code_ld(p.C), kBlk, rows, CU_TENSOR_MAP_SWIZZLE_128B) &&
         make_tmap_3d(&p.tmW, u8, w, code_ld(K), N, p.E, 1, kt ? outputs : kBlk, kt ? kBlk : outputs,
                      kt && outputs == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B);
}

// CTAs that share a tile: enough that all of them together have HBM's latency
// covered (each has up to 90 KB under way).
int split_of(int64_t tiles, int blocks, int64_t want) {
  int split = 1;
  while (split < kMaxSplit && split * tiles < want && 4 * split <= blocks) split *= 2;
  return split;
}

template <bool kT, int kN>
int launch_few(Product& p, const void* x, const void* w, int64_t extra, cudaStream_t s) {
  const int sms = sm_count();
  const int64_t tiles = (ceil_div(p.M, kN) + extra) * ceil_div(p.R, 128);
  p.split = split_of(tiles, static_cast<int>(ceil_div(p.C, kBlk)), sms - sms / 8);
  if (!make_maps(p, kT, x, w, kN, 128)) return ST_CUDA;
  const int64_t grid = p.split > 1 ? tiles * p.split : std::min<int64_t>(tiles, 2 * sms);
  return cuda_status(launch_after(fp8_product_few_kernel<kT, kN>, grid, kFewThreads, few_smem<kN>(), p.split, p, s));
}

template <bool kT>
int launch_small(Product& p, const void* x, const void* w, int64_t tiles, cudaStream_t s) {
  constexpr int kBudget = 111000;   // two CTAs an SM
  const int sms = sm_count();
  p.stages = kMaxStages;
  while (p.stages > 2 && small_smem(p.stages) > kBudget) --p.stages;
  p.split = split_of(tiles, static_cast<int>(ceil_div(p.C, kBlk)), sms);
  if (!make_maps(p, kT, x, w, 128, kTileR)) return ST_CUDA;
  const int64_t grid = p.split > 1 ? tiles * p.split : std::min<int64_t>(tiles, 2 * sms);
  return cuda_status(launch_after(fp8_product_kernel<kT>, grid, kThreads, small_smem(p.stages), p.split, p, s));
}

template <bool kT>
int launch_wide(Product& p, const void* x, const void* w, int64_t tiles, cudaStream_t s) {
  if (!make_maps(p, kT, x, w, 128, 128)) return ST_CUDA;
  if (p.vec && !make_tmap(&p.tmOut, p.bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, p.out, p.R,
                          p.M, static_cast<uint64_t>(p.R) * 2, 32, 32, CU_TENSOR_MAP_SWIZZLE_64B))
    return ST_CUDA;
  return cuda_status(launch_after(fp8_product_wide_kernel<kT>, std::min<int64_t>(tiles, sm_count()), kWideThreads,
                                  kWideSmemBytes, 1, p, s));
}

// The kernel by sizes (times of a call, K = 4096, weights in L2):
//   up to 64 tokens a weight: the weight as first operand, the smallest tile
//     that has them.  N = 11008, 16 tokens: 15 us, tiles of 32 tokens 15, of 64
//     19, small products 33, wide 21; 64 tokens: 20, small 24, wide 21.  With
//     few tiles of 64 tokens, tiles of 32: N = 4096, 64 tokens: 18 and 13 us.
//   more: wide tiles as soon as the small ones would give every SM one.
//     128 tokens, N = 4096 (64 small tiles): small 15 us, wide 21; N = 11008
//     (172): 25 and 21; 512 tokens, N = 4096 (256): 27 and 23; 1024 tokens,
//     N = 11008: 95 and 55.  Experts of 64 tokens each, N = 2048: 44 and 35.
template <bool kT>
int launch_product(Product& p, const void* x, const void* w, cudaStream_t s) {
  const int sms = sm_count();
  const int64_t extra = p.offsets == nullptr ? 0 : p.E;   // experts' last tiles, at most
  // experts' shares differ: tiles of up to twice the mean
  const int most = p.offsets == nullptr ? p.M : 2 * (p.M / p.E);
  if (most <= 16) return launch_few<kT, 16>(p, x, w, extra, s);
  if (most <= 32 || (most <= 64 && extra == 0 && p.R < 64 * 128)) return launch_few<kT, 32>(p, x, w, extra, s);
  if (most <= 64) return launch_few<kT, 64>(p, x, w, extra, s);
  const int64_t num_m = ceil_div(p.M, 128) + extra, small = num_m * ceil_div(p.R, kTileR);
  if (small >= sms) return launch_wide<kT>(p, x, w, num_m * ceil_div(p.R, 256), s);
  return launch_small<kT>(p, x, w, small, s);
}

constexpr size_t kAlign = 256;
size_t align_up(size_t n) { return (n + kAlign - 1) / kAlign * kAlign; }
bool aligned_to(const void* p, int bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0; }
int elem_bytes(int dt) { return dt == DT_F32 ? 4 : 2; }
bool aligned256(const void* p) { return (reinterpret_cast<uintptr_t>(p) & (kAlign - 1)) == 0; }
constexpr int64_t kMaxSize = INT32_MAX / 2;

size_t codes_bytes(int64_t M, int64_t C) { return align_up(static_cast<size_t>(M) * static_cast<size_t>(code_ld(C))); }
size_t scales_bytes(int64_t M, int64_t C) { return align_up(static_cast<size_t>(M) * static_cast<size_t>(ceil_div(C, kBlk)) * 4); }

// The product of one direction.  Workspace: [status][codes of the tokens]
// [their scales][partial sums of grad_bias].
int product(bool transposed, const void* x, int xt, int64_t M, const uint8_t* codes, const float* scales, int64_t E,
            int64_t N, int64_t K, const int32_t* offsets, int zero_rest, const void* bias, int bt, void* out,
            void* grad_bias, void* ws, size_t ws_bytes, void* stream, unsigned long long limit = kWaitTimeoutNs,
            int hold = INT32_MAX) {
  const int64_t C = transposed ? N : K, R = transposed ? K : N;
  if (xt != DT_F16 && xt != DT_BF16) return ST_UNSUPPORTED_DTYPE;
  if ((bias != nullptr || grad_bias != nullptr) && !valid_dt(bt)) return ST_UNSUPPORTED_DTYPE;
  if (M < 0 || N <= 0 || K <= 0 || M > kMaxSize || N > kMaxSize || K > kMaxSize) return ST_INVALID_ARG;
  if (E < 1 || E > kMaxExperts || (E > 1 && offsets == nullptr)) return ST_INVALID_ARG;
  if (codes == nullptr || scales == nullptr) return ST_INVALID_ARG;
  if (M > 0 && (x == nullptr || (out == nullptr && grad_bias == nullptr))) return ST_INVALID_ARG;
  if (!aligned16(x) || !aligned16(codes) || !aligned16(out)) return ST_MISALIGNED;
  if (!aligned_to(scales, 4) || !aligned_to(offsets, 4) || !aligned_to(bias, elem_bytes(bt)) ||
      !aligned_to(grad_bias, elem_bytes(bt)))
    return ST_MISALIGNED;
  if (ws == nullptr) return ST_WORKSPACE;
  if (!aligned256(ws)) return ST_MISALIGNED;
  const size_t partial_bytes = grad_bias != nullptr ? i8lt_fp8_grad_bias_bytes(M, N) : 0;
  if (ws_bytes < kAlign + codes_bytes(M, C) + scales_bytes(M, C) + partial_bytes) return ST_WORKSPACE;
  if (int d = check_device()) return d;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  uint8_t* q = static_cast<uint8_t*>(ws) + kAlign;
  float* qs = reinterpret_cast<float*>(q + codes_bytes(M, C));
  DevStatus* st = static_cast<DevStatus*>(ws);
  if (M == 0) {
    if (grad_bias != nullptr && cudaMemsetAsync(grad_bias, 0, static_cast<size_t>(N) * (bt == DT_F32 ? 4 : 2), s) != cudaSuccess) return ST_CUDA;
    return cuda_status(cudaMemsetAsync(st, 0, sizeof(DevStatus), s));
  }
  float* partial = grad_bias != nullptr ? reinterpret_cast<float*>(q + codes_bytes(M, C) + scales_bytes(M, C)) : nullptr;
  Product p;
  std::memset(&p, 0, sizeof(p));
  p.partial = partial;
  p.grad_bias = grad_bias;
  p.ranges = static_cast<int>(quantize_ranges(M, C));
  p.xs = qs;
  p.ws = scales;
  p.offsets = offsets;
  p.bias = bias;
  p.bias_dt = bt;
  p.out = out;
  p.st = st;
  p.limit = limit;
  p.hold = hold;
  p.M = static_cast<int>(M);
  p.R = static_cast<int>(R);
  p.C = static_cast<int>(C);
  p.E = static_cast<int>(E);
  p.nb = static_cast<int>(ceil_div(N, kBlk));
  p.kb = static_cast<int>(ceil_div(K, kBlk));
  p.bf16 = xt == DT_BF16;
  p.vec = R % 8 == 0;
  p.zero_rest = zero_rest != 0;
  if (cudaError_t e = launch_quantize(x, xt, M, C, q, qs, partial, st, s)) return cuda_status(e);
  if (out == nullptr) {   // the bias gradient alone
    ProfScope ps(K_FP8_GEMM, s);
    fp8_sum_bias_kernel<<<static_cast<unsigned>(std::min<int64_t>(ceil_div(C, 256), 4 * sm_count())), 256, 0, s>>>(p);
    return cuda_status(cudaGetLastError());
  }
  return transposed ? launch_product<true>(p, q, codes, s) : launch_product<false>(p, q, codes, s);
}

bool sizes_ok(int64_t E, int64_t N, int64_t K) {
  return E >= 0 && N >= 0 && K >= 0 && E <= kMaxExperts && N <= kMaxSize && K <= kMaxSize;
}

}  // namespace
}  // namespace i8lt

extern "C" {

using namespace i8lt;

int64_t i8lt_fp8_ld(int64_t C) { return C < 0 ? -1 : code_ld(C); }
int64_t i8lt_fp8_blocks(int64_t C) { return C < 0 ? -1 : ceil_div(C, kBlk); }

int i8lt_fp8_quantize(const void* x, int xt, int64_t M, int64_t C, uint8_t* codes, float* scales, void* stream) {
  if (!valid_dt(xt)) return ST_UNSUPPORTED_DTYPE;
  if (M < 0 || C < 0 || M > kMaxSize || C > kMaxSize) return ST_INVALID_ARG;
  if (M == 0 || C == 0) return ST_OK;
  if (x == nullptr || codes == nullptr || scales == nullptr) return ST_INVALID_ARG;
  if (!aligned16(x) || !aligned16(codes) || !aligned_to(scales, 4)) return ST_MISALIGNED;
  if (int d = check_device()) return d;
  return cuda_status(launch_quantize(x, xt, M, C, codes, scales, nullptr, nullptr, static_cast<cudaStream_t>(stream)));
}

int i8lt_fp8_quantize_weight(const void* W, int wt, int64_t E, int64_t N, int64_t K, uint8_t* codes, float* scales,
                             void* stream) {
  if (!valid_dt(wt)) return ST_UNSUPPORTED_DTYPE;
  if (!sizes_ok(E, N, K)) return ST_INVALID_ARG;
  if (E == 0 || N == 0 || K == 0) return ST_OK;
  if (W == nullptr || codes == nullptr || scales == nullptr) return ST_INVALID_ARG;
  if (!aligned16(W) || !aligned16(codes) || !aligned_to(scales, 4)) return ST_MISALIGNED;
  if (ceil_div(N, kBlk) > 65535) return ST_INVALID_ARG;
  if (int d = check_device()) return d;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const dim3 grid(static_cast<unsigned>(ceil_div(K, kBlk)), static_cast<unsigned>(ceil_div(N, kBlk)),
                  static_cast<unsigned>(E));
  const int n = static_cast<int>(N), k = static_cast<int>(K), ld = static_cast<int>(code_ld(K));
  ProfScope ps(K_FP8_QUANTIZE, s);
  if (wt == DT_F16) fp8_quantize_weight_kernel<<<grid, 256, 0, s>>>(static_cast<const __half*>(W), n, k, ld, codes, scales);
  else if (wt == DT_BF16)
    fp8_quantize_weight_kernel<<<grid, 256, 0, s>>>(static_cast<const __nv_bfloat16*>(W), n, k, ld, codes, scales);
  else fp8_quantize_weight_kernel<<<grid, 256, 0, s>>>(static_cast<const float*>(W), n, k, ld, codes, scales);
  return cuda_status(cudaGetLastError());
}

int i8lt_fp8_dequantize_weight(const uint8_t* codes, const float* scales, int64_t E, int64_t N, int64_t K, void* out,
                               int dt, void* stream) {
  if (!valid_dt(dt)) return ST_UNSUPPORTED_DTYPE;
  if (!sizes_ok(E, N, K)) return ST_INVALID_ARG;
  if (E == 0 || N == 0 || K == 0) return ST_OK;
  if (codes == nullptr || scales == nullptr || out == nullptr) return ST_INVALID_ARG;
  if (!aligned16(codes) || !aligned16(out) || !aligned_to(scales, 4)) return ST_MISALIGNED;
  if (int d = check_device()) return d;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int64_t rows = E * N;
  const unsigned grid = static_cast<unsigned>(std::min<int64_t>(ceil_div(rows * K, 256), sm_count() * 8));
  const int n = static_cast<int>(N), k = static_cast<int>(K), ld = static_cast<int>(code_ld(K));
  ProfScope ps(K_FP8_QUANTIZE, s);
  if (dt == DT_F16) fp8_dequantize_weight_kernel<<<grid, 256, 0, s>>>(codes, scales, rows, n, k, ld, static_cast<__half*>(out));
  else if (dt == DT_BF16)
    fp8_dequantize_weight_kernel<<<grid, 256, 0, s>>>(codes, scales, rows, n, k, ld, static_cast<__nv_bfloat16*>(out));
  else fp8_dequantize_weight_kernel<<<grid, 256, 0, s>>>(codes, scales, rows, n, k, ld, static_cast<float*>(out));
  return cuda_status(cudaGetLastError());
}

size_t i8lt_fp8_workspace_size(int64_t M, int64_t C) {
  if (M < 0 || C <= 0 || M > kMaxSize || C > kMaxSize) return 0;
  return kAlign + codes_bytes(M, C) + scales_bytes(M, C);
}

size_t i8lt_fp8_grad_bias_bytes(int64_t M, int64_t N) {
  if (M < 0 || N < 0 || M > kMaxSize || N > kMaxSize) return 0;
  if (N == 0) return 0;
  return align_up(static_cast<size_t>(quantize_ranges(M, N)) * static_cast<size_t>(N) * 4);
}

int i8lt_fp8_forward(const void* x, int xt, int64_t M, const uint8_t* codes, const float* scales, int64_t N, int64_t K,
                     const void* bias, int bt, void* out, void* ws, size_t ws_bytes, void* stream) {
  if (M > 0 && out == nullptr) return ST_INVALID_ARG;
  return product(false, x, xt, M, codes, scales, 1, N, K, nullptr, 0, bias, bt, out, nullptr, ws, ws_bytes, stream);
}

int i8lt_fp8_backward_input(const void* g, int gt, int64_t M, const uint8_t* codes, const float* scales, int64_t N,
                            int64_t K, void* grad_x, void* grad_bias, int bt, void* ws, size_t ws_bytes, void* stream) {
  return product(true, g, gt, M, codes, scales, 1, N, K, nullptr, 0, nullptr, bt, grad_x, grad_bias, ws, ws_bytes,
                 stream);
}

int i8lt_fp8_experts_forward(const void* x, int xt, int64_t M, const uint8_t* codes, const float* scales, int64_t E,
                             int64_t N, int64_t K, const int32_t* offsets, int zero_rest, void* out, void* ws,
                             size_t ws_bytes, void* stream) {
  if (offsets == nullptr || (M > 0 && out == nullptr)) return ST_INVALID_ARG;
  return product(false, x, xt, M, codes, scales, E, N, K, offsets, zero_rest, nullptr, 0, out, nullptr, ws, ws_bytes,
                 stream);
}

int i8lt_debug_fp8_wait_timeout(int64_t limit_ns, int32_t fetches, int transposed, const void* x, int xt, int64_t M,
                                const uint8_t* codes, const float* scales, int64_t E, int64_t N, int64_t K,
                                const int32_t* offsets, int zero_rest, void* out, void* ws, size_t ws_bytes,
                                void* stream) {
  if (limit_ns <= 0 || limit_ns > 2000000000LL || fetches < 0 || (M > 0 && out == nullptr)) return ST_INVALID_ARG;
  return product(transposed != 0, x, xt, M, codes, scales, E, N, K, offsets, zero_rest, nullptr, 0, out, nullptr, ws,
                 ws_bytes, stream, static_cast<unsigned long long>(limit_ns), fetches);
}

int i8lt_fp8_experts_backward_input(const void* g, int gt, int64_t M, const uint8_t* codes, const float* scales,
                                    int64_t E, int64_t N, int64_t K, const int32_t* offsets, int zero_rest,
                                    void* grad_x, void* ws, size_t ws_bytes, void* stream) {
  if (offsets == nullptr || (M > 0 && grad_x == nullptr)) return ST_INVALID_ARG;
  return product(true, g, gt, M, codes, scales, E, N, K, offsets, zero_rest, nullptr, 0, grad_x, nullptr, ws, ws_bytes,
                 stream);
}

}  // extern "C"
