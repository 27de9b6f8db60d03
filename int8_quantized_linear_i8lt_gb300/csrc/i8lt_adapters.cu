// Low-rank adapters of many requests at once beside a shared projection.
// Token m uses adapter e = index[m] (none outside [0, E)):
//   t[m] = x[m] A[e]^T,            y[m]  = base[m] + scale[e] t[m] B[e]^T,
//   u[m] = scale[e] g[m] B[e],     gx[m] = addend[m] + u[m] A[e],
//   gA[e] = sum_m u[m]^T x[m],     gB[e] = scale[e] sum_m g[m]^T t[m],
// with A [E, r, K], B [E, N, r].  Every sum is fp32; y, gx, gA and gB are
// rounded once.  t and u are operands of a second 16-bit product.  They are
// kept as two 16-bit values whose sum is t (u) to twice the type's precision,
// and both take part in every output: a rounded t would be off by as much as
// the output's own rounding.  In fp16 the second is kept times 2^11, and its
// products in an accumulator of their own: as they are, the pair would be off
// by up to half of fp16's smallest number, 2^-25, 3 % of a u of 1e-6
// (gradients are that small).  Their rows are in the plan's order, so that
// the tokens of a tile are a box of consecutive rows whatever the batch's
// order: 8192 interleaved tokens of 8 adapters, 4096 -> 11008, rank 64, took
// 349 us forward and backward with t and u gathered by token, 290 us so.
#include <algorithm>

#include "i8lt.h"
#include "i8lt_internal.h"

namespace i8lt {
namespace {

constexpr int kThreads = 256;
constexpr int kTile = 128;       // tokens per tile of the plan
constexpr int kFewTile = 8;      // tokens per tile of a small batch's second list
// Batches of up to this many tokens take the kernel for few tokens.  256
// tokens of one adapter, 4096 -> 4096, rank 16: 11 us by it, 25 us by the two
// kernels of long batches; 512 tokens, 4096 -> 11008, rank 64: 49 us against
// 33 us.
constexpr int64_t kFewTokens = 256;

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
  Tile* few;      // [few_slots] up to kFewTokens tokens: tiles of kFewTile, one after another, then empty ones
  int64_t slots, few_slots;
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
  p.few_slots = M <= kFewTokens ? std::min(M, M / kFewTile + E + 1) : 0;
  p.few = reinterpret_cast<Tile*>(b + off);
  off += round_up(p.few_slots * static_cast<int64_t>(sizeof(Tile)), 256);
  p.bytes = off;
  return p;
}

// One block per group: counts the tokens of the groups before it, then places
// its own in order (a stable sort, the same on every run) and fills its slots.
// A thread takes 8 consecutive tokens per pass, so that a batch of 8192 is one
// pass of 1024 threads (8 us, against 35 us for a warp per group).
constexpr int kPlanThreads = 1024;
__global__ void __launch_bounds__(kPlanThreads) adapter_plan_kernel(const int32_t* index, int M, int E, int* offset,
                                                                    int* perm, Tile* tiles) {
  constexpr int kWarpsPlan = kPlanThreads / 32, kPer = 8;
  // the group's first tokens, so that its tiles and whole runs of perm need no
  // second trip to memory
  constexpr int kStaged = kPlanThreads * kPer;
  __shared__ int counts[2][kWarpsPlan], own[kStaged];
  grid_dependents_launch();   // a kernel that takes the plan may set itself up meanwhile
  const int e = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  auto load = [&](int m0, int(&v)[kPer]) {   // the groups of 8 tokens, -1 past the end
    if (index == nullptr) {
#pragma unroll
      for (int i = 0; i < kPer; ++i) v[i] = 0;
    } else if (m0 + kPer <= M && (reinterpret_cast<uintptr_t>(index) & 15u) == 0) {
      *reinterpret_cast<int4*>(v) = __ldg(reinterpret_cast<const int4*>(index + m0));
      *reinterpret_cast<int4*>(v + 4) = __ldg(reinterpret_cast<const int4*>(index + m0 + 4));
    } else {
#pragma unroll
      for (int i = 0; i < kPer; ++i) v[i] = m0 + i < M ? index[m0 + i] : 0;
    }
#pragma unroll
    for (int i = 0; i < kPer; ++i) v[i] = m0 + i >= M ? -1 : v[i] >= 0 && v[i] < E ? v[i] : E;
  };
  __align__(16) int v[kPer];
  // tokens of the groups before e
  int n = 0;
  for (int base = 0; base < M; base += kPlanThreads * kPer) {
    load(base + tid * kPer, v);
#pragma unroll
    for (int i = 0; i < kPer; ++i) n += v[i] >= 0 && v[i] < e;
  }
  n = __reduce_add_sync(0xffffffffu, n);
  if (lane == 0) counts[0][warp] = n;
  __syncthreads();
  int before = 0;
  for (int k = 0; k < kWarpsPlan; ++k) before += counts[0][k];
  int placed = 0;
  for (int base = 0, turn = 1; base < M; base += kPlanThreads * kPer, ++turn) {
    if (M > kPlanThreads * kPer) load(base + tid * kPer, v);   // else v still holds them
    int mine = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) mine += v[i] == e;
    int scan = mine;   // inclusive over the warp
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int up = __shfl_up_sync(0xffffffffu, scan, o);
      if (lane >= o) scan += up;
    }
    if (lane == 31) counts[turn & 1][warp] = scan;
    __syncthreads();
    int at = before + placed + scan - mine, all = 0;
    for (int k = 0; k < kWarpsPlan; ++k) {
      const int c = counts[turn & 1][k];
      if (k < warp) at += c;
      all += c;
    }
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      if (v[i] == e) {
        if (at - before < kStaged) own[at - before] = base + tid * kPer + i;
        else perm[at] = base + tid * kPer + i;
        ++at;
      }
    placed += all;
  }
  __syncthreads();   // own and perm are visible to the block
  for (int i = tid; i < min(placed, kStaged); i += kPlanThreads) perm[before + i] = own[i];
  if (tid == 0) {
    offset[e] = before;
    if (e == E) offset[E + 1] = M;
  }
  auto token = [&](int place) { return place - before < kStaged ? own[place - before] : perm[place]; };
  const int slot0 = before / kTile + e, slot1 = (before + placed) / kTile + e + 1;
  for (int s = slot0 + tid; s < slot1; s += kPlanThreads) {
    const int start = before + (s - slot0) * kTile;
    const int count = max(0, min(kTile, before + placed - start));
    int row0 = -1;
    if (count > 0 && token(start + count - 1) - token(start) == count - 1) row0 = token(start);
    tiles[s] = Tile{e, start, count, row0};
  }
}

// The plan of up to kFewTokens tokens, by one block whatever the number of
// adapters: a token's place is the number of tokens before it in (group,
// index) order.  5 us for 64 tokens of 64 adapters, all latency.
__global__ void __launch_bounds__(kFewTokens) adapter_plan_few_kernel(const int32_t* index, int M, int E, int* offset,
                                                                      int* perm, Tile* tiles, Tile* few,
                                                                      int few_slots) {
  __shared__ __align__(16) int group[kFewTokens];
  __shared__ int sorted[kFewTokens], place[kFewTokens], counts[kFewTokens / 32];
  grid_dependents_launch();   // a kernel that takes the plan may set itself up meanwhile
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int g = E + 1;   // past the end: after every token
  if (tid < M) {
    const int i = index != nullptr ? index[tid] : 0;
    g = i >= 0 && i < E ? i : E;
  }
  group[tid] = g;
  __syncthreads();
  if (tid < M) {
    int at = 0;
#pragma unroll 4
    for (int j = 0; j < M; j += 4) {
      const int4 o = *reinterpret_cast<const int4*>(group + j);
      at += (o.x < g || (o.x == g && j < tid)) + (o.y < g || (o.y == g && j + 1 < tid)) +
            (o.z < g || (o.z == g && j + 2 < tid)) + (o.w < g || (o.w == g && j + 3 < tid));
    }
    sorted[at] = g;
    place[at] = tid;
    perm[at] = tid;
  }
  __syncthreads();
  auto first_of = [&](int e) {   // the first place whose group is e or later
    int lo = 0, hi = M;
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (sorted[mid] < e) lo = mid + 1;
      else hi = mid;
    }
    return lo;
  };
  for (int e = tid; e <= E; e += kFewTokens) {
    const int before = first_of(e), end = first_of(e + 1);
    offset[e] = before;
    if (e == E) offset[E + 1] = M;
    for (int s = before / kTile + e, start = before; s <= end / kTile + e; ++s, start += kTile) {
      const int count = max(0, min(kTile, end - start));
      const bool run = count > 0 && place[start + count - 1] - place[start] == count - 1;
      tiles[s] = Tile{e, start, count, run ? place[start] : -1};
    }
  }
  bool head = false;
  int end = 0;
  if (tid < M) {
    head = (tid - first_of(sorted[tid])) % kFewTile == 0;
    end = first_of(sorted[tid] + 1);
  }
  const unsigned heads = __ballot_sync(0xffffffffu, head);
  if (lane == 0) counts[warp] = __popc(heads);
  __syncthreads();
  int at = __popc(heads & ((1u << lane) - 1)), all = 0;
  for (int k = 0; k < static_cast<int>(kFewTokens) / 32; ++k) {
    if (k < warp) at += counts[k];
    all += counts[k];
  }
  if (head) few[at] = Tile{sorted[tid], tid, min(kFewTile, end - tid), -1};
  for (int s = all + tid; s < few_slots; s += kFewTokens) few[s] = Tile{E, 0, 0, -1};
}

// ---- shared pieces of the three products ----------------------------------
//
// All three run on the tensor cores (tcgen05, 128-row tiles, fp32 accumulators
// in TMEM) on operands staged in shared memory.  Where every row starts on 16
// bytes, one warp fetches the operands by TMA, a tile of consecutive tokens
// (one request, one adapter) as a box, and one thread issues the products;
// else all threads gather them with narrower asynchronous copies that fill
// what is past an edge with zeros.  Those cost issue slots: 4096 -> 11008 at
// rank 64 on 8192 tokens took 28 + 92 us by them, 24 + 63 us by TMA.  Matrices of a width C have rows of C 16-bit
// elements; an operand tile is rows of 64 elements (128 bytes) in the
// 128-byte swizzle, either with the reduction along the row ("K-major") or
// across the rows ("MN-major").

constexpr int kRowBytes = 128;

__device__ __forceinline__ uint16_t to_16(float v, bool bf16) {
  return bf16 ? __bfloat16_as_ushort(__float2bfloat16_rn(v)) : __half_as_ushort(__float2half_rn(v));
}

__device__ __forceinline__ float from_16(uint16_t v, bool bf16) {
  return bf16 ? __uint_as_float(static_cast<uint32_t>(v) << 16) : __half2float(__ushort_as_half(v));
}
// The second part of v: what rounding it to hi left over (0 where hi
// overflowed).  fp16: times 2^11, which 2^4, half the last place of the
// largest numbers, allows; together they are off by 2^-22 of v or by 2^-36.
// bf16 has fp32's range and needs no factor.
constexpr float kRestUp = 0x1p11f, kRestDown = 0x1p-11f;
__device__ __forceinline__ uint16_t rest_16(float v, uint16_t hi, bool bf16) {
  const float rest = v - from_16(hi, bf16);
  return !isfinite(from_16(hi, bf16)) ? uint16_t(0) : to_16(bf16 ? rest : rest * kRestUp, bf16);
}

template <int kBytes>
__device__ __forceinline__ void cp_async(uint32_t dst, const void* src, bool take) {
  const int n = take ? kBytes : 0;
  if constexpr (kBytes == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(dst), "l"(src), "n"(kBytes), "r"(n) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int kPending>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(kPending) : "memory");
}

// The 16 bytes that start `shift` (0, 2 .. 14) bytes into lo, hi.
__device__ __forceinline__ uint4 realign(uint4 lo, uint4 hi, int shift) {
  uint32_t w[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
#pragma unroll
  for (int i = 0; i < 6; ++i) w[i] = shift & 8 ? w[i + 2] : w[i];
#pragma unroll
  for (int i = 0; i < 5; ++i) w[i] = shift & 4 ? w[i + 1] : w[i];
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = __funnelshift_r(w[i], w[i + 1], (shift & 2) * 8);
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// 8 elements at any address, of which the first `valid` exist: the aligned 16
// bytes that hold the first one and, where they reach into them, the next 16.
struct Unaligned {
  uint4 lo, hi;
  __device__ __forceinline__ void fetch(const uint16_t* src, int64_t valid) {
    const uintptr_t p = reinterpret_cast<uintptr_t>(src);
    const uint4* q = reinterpret_cast<const uint4*>(p & ~static_cast<uintptr_t>(15));
    lo = hi = make_uint4(0, 0, 0, 0);
    if (valid > 0) lo = q[0];
    if (static_cast<int>(p & 15) + 2 * min(valid, static_cast<int64_t>(8)) > 16) hi = q[1];
  }
  __device__ __forceinline__ void put(uint32_t dst, const uint16_t* src, int64_t valid) const {
    const uint4 v = realign(lo, hi, static_cast<int>(reinterpret_cast<uintptr_t>(src) & 15));
    uint32_t w[4] = {v.x, v.y, v.z, v.w};
    if (valid < 8)
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] &= valid > 2 * i + 1 ? 0xffffffffu : valid > 2 * i ? 0xffffu : 0u;
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(dst), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3])
                 : "memory");
  }
};

// How operands reach shared memory: tiles by TMA, or chunks of 8 elements by
// asynchronous copies of `width` bytes, which every row start and row length
// is a multiple of, or, where that is 2, as aligned 16 bytes that go through
// registers (8192 tokens, 4097 -> 5001, rank 64, take 380 us forward and
// backward so and 642 us by single elements).
enum Copy { kByTma, kByAsync, kByRegisters };

// 8 elements for the 16 bytes at `dst`, of which the first `valid` exist (the
// others are zeros; valid <= 0: none, `row` is then not read).
struct Chunk {
  uint32_t dst;
  const uint16_t* row;
  int64_t at, valid;
};
// n chunks, those that chunk(i) gives; through registers they are fetched
// together, before the first is stored.
template <Copy kCopy, int n, typename F>
__device__ __forceinline__ void load_chunks(int width, F chunk) {
  if constexpr (kCopy == kByRegisters) {
    Unaligned u[n];
#pragma unroll
    for (int i = 0; i < n; ++i) {
      const Chunk c = chunk(i);
      u[i].fetch(c.row + (c.valid > 0 ? c.at : 0), c.valid);
    }
#pragma unroll
    for (int i = 0; i < n; ++i) {
      const Chunk c = chunk(i);
      u[i].put(c.dst, c.row + (c.valid > 0 ? c.at : 0), c.valid);
    }
  } else {
#pragma unroll
    for (int i = 0; i < n; ++i) {
      const Chunk c = chunk(i);
      const uint16_t* src = c.row + (c.valid > 0 ? c.at : 0);
      if (width == 16) {
        cp_async<16>(c.dst, src, c.valid > 0);
      } else if (width == 8) {
#pragma unroll
        for (int k = 0; k < 2; ++k) cp_async<8>(c.dst + 8 * k, c.valid > 4 * k ? src + 4 * k : src, c.valid > 4 * k);
      } else {
#pragma unroll
        for (int k = 0; k < 4; ++k) cp_async<4>(c.dst + 4 * k, c.valid > 2 * k ? src + 2 * k : src, c.valid > 2 * k);
      }
    }
  }
}
// One of a second operand, whose width may be another one.
template <Copy kCopy>
__device__ __forceinline__ void load_chunk(int width, const Chunk& c) {
  if (kCopy == kByRegisters && width == 2) load_chunks<kByRegisters, 1>(width, [&](int) { return c; });
  else load_chunks<kByAsync, 1>(width, [&](int) { return c; });
}

// Byte offset of 16-byte chunk `c` (0-7) of row `i` in a swizzled tile.
__device__ __forceinline__ uint32_t swizzled(int i, int c) {
  return static_cast<uint32_t>(i * kRowBytes + ((c ^ (i & 7)) << 4));
}

__device__ __forceinline__ uint32_t align1024(uint32_t a) { return (a + 1023u) & ~1023u; }

__device__ __forceinline__ uint32_t instruction(int n, bool a_mn, bool b_mn, bool bf16) {
  return make_idesc_f16(128, n, a_mn, b_mn) | (bf16 ? (1u << 7) | (1u << 10) : 0u);
}
// K-major: 8-row atoms 1024 bytes apart, 32 bytes along the row per MMA.
__device__ __forceinline__ uint64_t desc_k(uint32_t a, int k) { return make_sdesc(a + 32 * k, 16, 1024, kSwizzle128B); }
// MN-major: blocks of 64 MN elements `block` bytes apart, 8-row atoms of the
// reduction 1024 bytes apart, 16 rows per MMA.
__device__ __forceinline__ uint64_t desc_mn(uint32_t a, int k, uint32_t block) {
  return make_sdesc(a + 2048 * k, block, 1024, kSwizzle128B);
}

__device__ __forceinline__ float4 ld_cluster4(uint32_t a) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(a)
               : "memory");
  return v;
}
__device__ __forceinline__ uint32_t map_cluster(uint32_t a, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(rank));
  return r;
}

// Barriers, the abort flag of the bounded waits and the TMEM address.
constexpr int kMaxStages = 4;
struct Sync {
  uint64_t done[kMaxStages];    // the products that read a stage have completed
  uint64_t full[kMaxStages];    // a stage's TMA copies have arrived
  uint64_t last;                // all products have completed
  uint32_t tmem;
  int abort;
};
__device__ __forceinline__ void sync_setup(Sync& y, uint32_t columns) {
  if (threadIdx.x == 0) {
    for (int i = 0; i < kMaxStages; ++i) {
      mbar_init(&y.done[i], 1);
      mbar_init(&y.full[i], 1);
    }
    mbar_init(&y.last, 1);
    y.abort = 0;
    fence_mbar_init();
  }
  if (threadIdx.x < 32) {
    tmem_alloc(&y.tmem, columns);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
}
// A wait that runs out raises `abort`: every role stops issuing, and before
// tensor memory is freed and shared memory reused, the copies and products
// under way are waited for: the last `stages` fetches of `fetched`, counted on
// full, and the last of `multiplied` products, on done.
__device__ __forceinline__ bool aborted(const int& flag) { return *static_cast<const volatile int*>(&flag) != 0; }
__device__ __forceinline__ void wind_down(uint64_t* full, int fetched, uint64_t* done, int multiplied, int stages,
                                          DevStatus* st) {
  for (int i = max(0, fetched - stages); i < fetched; ++i) mbar_wait_out(&full[i % stages], (i / stages) & 1, st, 37);
  if (multiplied > 0) mbar_wait_out(&done[(multiplied - 1) % stages], ((multiplied - 1) / stages) & 1, st, 38);
}
__device__ __forceinline__ void sync_end(const Sync& y, uint32_t columns) {
  tc_fence_before();
  __syncthreads();
  if (threadIdx.x < 32) tmem_dealloc(y.tmem, columns);
}

__host__ __device__ constexpr int rank16(int r) { return (r + 15) & ~15; }
__host__ __device__ constexpr uint32_t tmem_columns(int r16) { return r16 <= 32 ? 32u : r16 <= 64 ? 64u : 128u; }
// Row pitch (floats) of the accumulator copy that the CTAs of a cluster add
// up: 16-byte accesses of 8 rows hit 8 different bank groups.
__host__ __device__ constexpr int red_pitch(int r16) { return r16 + 4; }

// 16 columns of the second parts' products, added to those of the first ones.
__device__ __forceinline__ void add_rest(uint32_t tmem, uint32_t* v) {
  uint32_t w[16];
  tmem_ld16(tmem, w);
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = __float_as_uint(fmaf(__uint_as_float(w[i]), kRestDown, __uint_as_float(v[i])));
}

// The CTA's accumulator (128 rows x r16) into shared memory; rest > 0: with
// that of the second parts, `rest` columns on.
__device__ __forceinline__ void spill(uint32_t tmem, int r16, float* red, uint32_t rest = 0) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int row = (warp & 3) * 32 + lane;
  for (int c = (warp >> 2) * 16; c < r16; c += 32) {
    uint32_t v[16];
    tmem_ld16(tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16) + c, v);
    if (rest != 0) add_rest(tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16) + rest + c, v);
    float4* p = reinterpret_cast<float4*>(red + row * red_pitch(r16) + c);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      p[i] = make_float4(__uint_as_float(v[4 * i]), __uint_as_float(v[4 * i + 1]), __uint_as_float(v[4 * i + 2]),
                         __uint_as_float(v[4 * i + 3]));
  }
}
// The sums over the cluster of 4 elements of it, in the order of the ranks.
// The loads of all ranks are under way before the first is used: one at a
// time, they made up half of a small product's time.
__device__ __forceinline__ void cluster_sum4(uint32_t red, int at, int ranks, float (&s)[4]) {
  float4 v[8];
#pragma unroll
  for (int q = 0; q < 8; ++q)
    if (q < ranks) v[q] = ld_cluster4(map_cluster(red + 4u * at, q));
  s[0] = s[1] = s[2] = s[3] = 0.f;
#pragma unroll
  for (int q = 0; q < 8; ++q)
    if (q < ranks) {
      s[0] += v[q].x;
      s[1] += v[q].y;
      s[2] += v[q].z;
      s[3] += v[q].w;
    }
}

// ---- mid = X W^T (t and u) -------------------------------------------------

struct ShrinkArgs {
  CUtensorMap tmX, tmW;   // with kTma: X, box 64 x 128; W, box 64 x r16 (K-major) or 64 x 64
  const uint16_t* X;      // [M, C]
  const uint16_t* W;      // per group [R, C] (K-major) or [C, R] (MN-major)
  uint16_t* mid;          // [2, M, R] in the plan's order: the values rounded, and rest_16 of them
  int64_t plane;          // M R
  const float* scale;     // applied when not NULL
  const Tile* tiles;
  const int* perm;
  DevStatus* st;          // cleared by the first kernel of a call
  int64_t C;
  int R, E, cw, rw;       // cw, rw: copy widths of rows of C and of R elements
  int ranks;              // CTAs per cluster
  bool bf16;
};

__host__ __device__ constexpr int shrink_stage_bytes(int r16, bool mn) {
  return 128 * kRowBytes + (mn ? (r16 > 64 ? 2 : 1) * 64 * kRowBytes : r16 * kRowBytes);
}

// One cluster per tile of 128 tokens; its CTAs split the reduction, each
// accumulating in TMEM, and add up in the order of their ranks.  Bound by
// reading X once, and W once per tile from L2: 8192 tokens of 11008 features,
// rank 64, take 37 us, 4.9 TB/s of X.  Tiles of 256 tokens, which read W half
// as often, make no difference.  With kTma a tile of tokens here and there is
// gathered by all threads, W by TMA all the same: 4 rows per TMA request took
// 61 us for 8192 interleaved tokens of 8 adapters.
template <bool kMN, int kStages, Copy kCopy>
__global__ void __launch_bounds__(kThreads, 2) shrink_kernel(const __grid_constant__ ShrinkArgs a) {
  constexpr bool kTma = kCopy == kByTma;
  extern __shared__ uint8_t smem_raw[];
  __shared__ Sync y;
  const int ranks = a.ranks, rank = blockIdx.x % ranks;
  if (kTma && threadIdx.x == 0) {
    tma_prefetch_desc(&a.tmX);
    tma_prefetch_desc(&a.tmW);
  }
  const int tid = threadIdx.x, R = a.R, r16 = rank16(R);
  sync_setup(y, tmem_columns(r16));
  grid_dependency_wait();
  if (blockIdx.x == 0 && threadIdx.x == 0) *a.st = DevStatus{0, 0, 0, 0};
  const Tile t = a.tiles[blockIdx.x / ranks];
  if (t.count == 0 || t.group >= a.E) sync_end(y, tmem_columns(r16));
  if (t.count == 0) return;
  if (t.group >= a.E) {
    if (rank == 0)
      for (int i = tid; i < t.count * R; i += kThreads) {
        uint16_t* o = a.mid + static_cast<int64_t>(t.start) * R + i;
        o[0] = o[a.plane] = 0;
      }
    return;
  }
  const uint32_t base = align1024(smem_u32(smem_raw));
  const int stage_bytes = shrink_stage_bytes(r16, kMN);
  const int nb = static_cast<int>((a.C + 63) / 64);
  const int n = (nb - rank + ranks - 1) / ranks;   // blocks rank, rank + ranks, ...
  auto column = [&](int it) { return static_cast<int64_t>(rank + it * ranks) * 64; };
  const int64_t C = a.C;
  const uint16_t* W = a.W + static_cast<int64_t>(t.group) * R * C;

  const uint32_t idesc = instruction(r16, false, kMN, a.bf16);
  auto multiply = [&](int it) {   // one thread: the products of a stage
    const int s = it % kStages;
    const uint32_t xs = base + s * stage_bytes, ws = xs + 128 * kRowBytes;
#pragma unroll
    for (int k = 0; k < 4; ++k)
      umma_f16(y.tmem, desc_k(xs, k), kMN ? desc_mn(ws, k, 64 * kRowBytes) : desc_k(ws, k), idesc,
               it > 0 || k > 0 ? 1u : 0u);
    umma_commit(&y.done[s]);
    if (it == n - 1) umma_commit(&y.last);
  };
  const int cw = kTma ? 16 : a.cw;
  // with kTma: the tile of W of step `it`, counted on its stage's barrier
  auto load_w = [&](int it, uint8_t* ws, uint64_t* full) {
    const int c0 = static_cast<int>(column(it));
    if constexpr (kMN) {
      tma_load_3d(ws, &a.tmW, 0, c0, t.group, full);
      if (r16 > 64) tma_load_3d(ws + 64 * kRowBytes, &a.tmW, 64, c0, t.group, full);
    } else {
      tma_load_3d(ws, &a.tmW, c0, 0, t.group, full);
    }
  };
  uint8_t* stages = smem_raw + (base - smem_u32(smem_raw));
  int fetched = 0, multiplied = 0;   // steps, by the thread that issues them
  if (kTma && t.row0 >= 0) {
    if (tid == 0) {
      for (int it = 0; it < n; fetched = ++it) {
        const int s = it % kStages;
        uint8_t* xs = stages + s * stage_bytes;
        if (it >= kStages && !mbar_wait(&y.done[s], (it / kStages - 1) & 1, &y.abort, a.st, 20)) break;
        mbar_arrive_expect_tx(&y.full[s], stage_bytes);
        tma_load_2d(xs, &a.tmX, static_cast<int>(column(it)), t.row0, &y.full[s]);
        load_w(it, xs + 128 * kRowBytes, &y.full[s]);
      }
    } else if (tid == 32) {
      for (int it = 0; it < n; multiplied = ++it) {
        if (!mbar_wait(&y.full[it % kStages], (it / kStages) & 1, &y.abort, a.st, 25)) break;
        tc_fence_after();
        multiply(it);
      }
    }
    __syncwarp();
  } else {
    // this thread's rows of X: 8 threads a row
    const uint16_t* xrow[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int row = (tid >> 3) + 32 * i;
      xrow[i] = row < t.count ? a.X + static_cast<int64_t>(a.perm[t.start + row]) * C : a.X;
    }
    auto load = [&](int b, int s) {
      const int64_t c0 = column(b);
      const uint32_t xs = base + s * stage_bytes, ws = xs + 128 * kRowBytes;
      const int64_t at = c0 + (tid & 7) * 8;
      load_chunks<kCopy, 4>(cw, [&](int i) {   // of rows past the tile's tokens nothing is read
        const int row = (tid >> 3) + 32 * i;
        return Chunk{xs + swizzled(row, tid & 7), xrow[i], at, row < t.count ? C - at : 0};
      });
      if constexpr (kTma) {
        if (tid == 0 && !aborted(y.abort)) {
          mbar_arrive_expect_tx(&y.full[s], stage_bytes - 128 * kRowBytes);
          load_w(b, stages + s * stage_bytes + 128 * kRowBytes, &y.full[s]);
          fetched = b + 1;
        }
      } else if constexpr (kMN) {
        const int chunks = r16 / 8;
        for (int i = tid; i < 64 * chunks; i += kThreads) {
          const int k = i / chunks, c = i % chunks;
          load_chunk<kCopy>(a.rw, Chunk{ws + (c >> 3) * 64 * kRowBytes + swizzled(k, c & 7),
                                        W + min(c0 + k, C - 1) * R, c * 8, c0 + k < C ? R - c * 8 : 0});
        }
      } else {
        for (int j = tid >> 3; j < r16; j += kThreads / 8)
          load_chunk<kCopy>(a.cw, Chunk{ws + swizzled(j, tid & 7), W + min(j, R - 1) * C, at, j < R ? C - at : 0});
      }
    };

#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) {
      if (i < n) load(i, i);
      cp_async_commit();
    }
    for (int it = 0; it < n; ++it) {
      cp_async_wait<kStages - 2>();
      fence_proxy_async_smem();
      __syncthreads();
      if (tid == 0 && (!kTma || mbar_wait(&y.full[it % kStages], (it / kStages) & 1, &y.abort, a.st, 25)) &&
          !aborted(y.abort)) {
        multiply(it);
        multiplied = it + 1;
      }
      const int next = it + kStages - 1;
      if (next < n) {
        // the stage to refill was read by the products of step it - 1
        if (it > 0) mbar_wait(&y.done[(it - 1) % kStages], ((it - 1) / kStages) & 1, &y.abort, a.st, 20);
        load(next, next % kStages);
      }
      cp_async_commit();
    }
  }
  mbar_wait(&y.last, 0, &y.abort, a.st, 21);
  cp_async_wait<0>();
  __syncwarp();
  tc_fence_after();
  grid_dependents_launch();
  float* red = reinterpret_cast<float*>(smem_raw + (base - smem_u32(smem_raw)));
  __syncthreads();
  if (aborted(y.abort)) {
    wind_down(y.full, fetched, y.done, multiplied, kStages, a.st);
    __syncthreads();
  }
  spill(y.tmem, r16, red);
  sync_end(y, tmem_columns(r16));
  cluster_sync();
  const int rows = (128 + ranks - 1) / ranks, row0 = rank * rows;
  const float scale = a.scale != nullptr ? a.scale[t.group] : 1.f;
  const int quads = r16 / 4;
  for (int i = tid; i < rows * quads; i += kThreads) {
    const int row = row0 + i / quads, j = i % quads * 4;
    if (row >= t.count || j >= R) continue;
    float s[4];
    cluster_sum4(base, row * red_pitch(r16) + j, ranks, s);
    uint16_t* o = a.mid + static_cast<int64_t>(t.start + row) * R + j;
    uint16_t hi[4], lo[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      hi[k] = to_16(scale * s[k], a.bf16);
      lo[k] = rest_16(scale * s[k], hi[k], a.bf16);
    }
    if (R % 4 == 0) {
      *reinterpret_cast<uint2*>(o) = make_uint2(hi[0] | hi[1] << 16, hi[2] | hi[3] << 16);
      *reinterpret_cast<uint2*>(o + a.plane) = make_uint2(lo[0] | lo[1] << 16, lo[2] | lo[3] << 16);
    } else {
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (j + k < R) {
          o[k] = hi[k];
          o[a.plane + k] = lo[k];
        }
    }
  }
  cluster_sync();   // the other CTAs have read this one's sums
}

// ---- out = addend + scale mid W^T (y and gx) --------------------------------

struct ExpandArgs {
  CUtensorMap tmMid, tmW, tmAdd, tmOut;   // with kTma: mid, addend and out, box 64 x 128; W, box 64 x 64 or 64 x r16
  const uint16_t* mid;     // [2, M, R], in the plan's order
  const uint16_t* W;       // per group [C, R] (K-major) or [R, C] (MN-major)
  const uint16_t* addend;  // [M, C] or NULL; may be out
  uint16_t* out;           // [M, C]
  const float* scale;
  const Tile* tiles;
  const int* perm;
  DevStatus* st;
  int64_t C;
  int M, R, E, cw, rw, mw; // mw: the copy width of mid's second part
  int col_tiles;           // 64-column tiles per CTA
};

constexpr int kCols = 64;                                  // columns per tile
constexpr uint32_t kTileBytes = 128 * kRowBytes;           // addend / out tile: 128 tokens x 64 columns
__host__ __device__ constexpr int expand_blocks(int r16) { return r16 > 64 ? 2 : 1; }
__host__ __device__ constexpr int expand_mid_bytes(int r16) { return expand_blocks(r16) * 128 * kRowBytes; }
__host__ __device__ constexpr int expand_w_bytes(int r16) { return expand_blocks(r16) * 64 * kRowBytes; }
constexpr int kAddTiles = 4;                               // addend tiles in flight

struct ExpandSync {
  uint64_t w_full[2], w_free[2], acc_full[2], acc_free[2], add_full[4], add_free[4], mid_full;
  uint32_t tmem;
  int abort;
};
// Shared memory: mid's two parts, two tiles of W, the addend tiles and the
// barriers, with room to align the first.  Up to rank 64 two CTAs fit an SM
// exactly.
__host__ __device__ constexpr int expand_smem(int r16) {
  return 2 * expand_mid_bytes(r16) + 2 * expand_w_bytes(r16) + kAddTiles * static_cast<int>(kTileBytes) + 1024;
}
__host__ __device__ constexpr int expand_per_sm(int r16) { return r16 > 64 ? 1 : 2; }
static_assert(2 * (expand_smem(64) + 1024) <= 228 * 1024 && sizeof(ExpandSync) <= 512, "two CTAs per SM");

// One CTA per (tile of 128 tokens, run of 64-column tiles): mid stays in
// shared memory; per column tile W is read from L2, the addend tile arrives
// several tiles ahead, is updated in place and leaves as a whole.  Warps 0-7
// turn the accumulators into output, thread 256 fetches, thread 288 issues
// the products.  Bound by reading the addend and writing out: 8192 tokens of
// 11008 features, rank 64, take 63 us, 5.7 TB/s.
constexpr int kExpandThreads = 320;
template <bool kMN, Copy kCopy, bool kBf16>
__global__ void __launch_bounds__(kExpandThreads, 2) expand_kernel(const __grid_constant__ ExpandArgs a) {
  constexpr bool kTma = kCopy == kByTma;
  extern __shared__ __align__(1024) uint8_t expand_raw[];
  if (kTma && threadIdx.x == 256) {
    tma_prefetch_desc(&a.tmW);
    tma_prefetch_desc(&a.tmAdd);
    tma_prefetch_desc(&a.tmMid);
    tma_prefetch_desc(&a.tmOut);
  }
  const Tile t = a.tiles[blockIdx.x];
  if (t.count == 0) return;
  const bool adapter = t.group < a.E;
  if (!adapter && a.addend == a.out) {
    grid_dependency_wait();
    return;
  }
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, R = a.R, r16 = rank16(R);
  const int64_t C = a.C;
  const int j0 = blockIdx.y * a.col_tiles;
  const int n = min(a.col_tiles, static_cast<int>((C + kCols - 1) / kCols) - j0);
  constexpr int bufs = kAddTiles;
  uint8_t* mids = expand_raw + (align1024(smem_u32(expand_raw)) - smem_u32(expand_raw));
  uint8_t* wbuf = mids + 2 * expand_mid_bytes(r16);
  uint8_t* tiles = wbuf + 2 * expand_w_bytes(r16);
  ExpandSync& y = *reinterpret_cast<ExpandSync*>(tiles + bufs * kTileBytes);
  const float scale = a.scale != nullptr && adapter ? a.scale[t.group] : 1.f;
  // a tile that ends inside the batch or is no run of tokens is stored row by row
  const bool tma_out = kTma && t.row0 >= 0 && (t.count == 128 || t.row0 + t.count == a.M);
  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&y.w_full[i], 1);
      mbar_init(&y.w_free[i], 1);
      mbar_init(&y.acc_full[i], 1);
      mbar_init(&y.acc_free[i], 256);
    }
    for (int i = 0; i < 4; ++i) {
      mbar_init(&y.add_full[i], 1);
      mbar_init(&y.add_free[i], 1);
    }
    mbar_init(&y.mid_full, 1);
    y.abort = 0;
    fence_mbar_init();
  }
  // accumulator j & 1; in fp16 the second part's products beside it
  constexpr uint32_t rest = kBf16 ? 0 : kCols, acc = rest + kCols;
  if (warp == 0) {
    tmem_alloc(&y.tmem, 2 * acc);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();

  const uint32_t idesc = instruction(kCols, false, kMN, kBf16);
  auto multiply = [&](int j) {   // one thread: accumulator j & 1 = mid W^T
    const uint32_t d = y.tmem + (j & 1) * acc;
    const uint32_t ms = smem_u32(mids), ws = smem_u32(wbuf) + (j & 1) * expand_w_bytes(r16);
    for (int k = 0; k < r16 / 16; ++k) {
      const uint32_t m = ms + (k >> 2) * 128 * kRowBytes;
      const uint64_t w = kMN ? desc_mn(ws, k, 0) : desc_k(ws + (k >> 2) * 64 * kRowBytes, k & 3);
      umma_f16(d, desc_k(m, k & 3), w, idesc, k > 0 ? 1u : 0u);
      umma_f16(d + rest, desc_k(m + expand_mid_bytes(r16), k & 3), w, idesc, k > 0 || rest == 0 ? 1u : 0u);
    }
    umma_commit(&y.w_free[j & 1]);
    umma_commit(&y.acc_full[j & 1]);
  };
  // 8 columns of a token: addend + scale * accumulator
  auto combine = [&](uint4 w, const uint32_t* v) {
    uint32_t* e = reinterpret_cast<uint32_t*>(&w);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float lo = __uint_as_float(v[2 * i]), hi = __uint_as_float(v[2 * i + 1]);
      if constexpr (kBf16) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(fmaf(scale, lo, __uint_as_float(e[i] << 16)),
                                                       fmaf(scale, hi, __uint_as_float(e[i] & 0xffff0000u)));
        e[i] = *reinterpret_cast<const uint32_t*>(&h);
      } else {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&e[i]));
        const __half2 h = __floats2half2_rn(fmaf(scale, lo, f.x), fmaf(scale, hi, f.y));
        e[i] = *reinterpret_cast<const uint32_t*>(&h);
      }
    }
    return w;
  };
  // warps 0-7: tile j into its buffer, in place of the addend
  auto finish = [&](int j, uint8_t* buf) {
    const int row = (warp & 3) * 32 + lane, c0 = (warp >> 2) * 32;
    uint32_t v[32];
    if (adapter) {
      mbar_wait(&y.acc_full[j & 1], (j >> 1) & 1, &y.abort, a.st, 22);
      __syncwarp();
      tc_fence_after();
      const uint32_t d = y.tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16) + (j & 1) * acc + c0;
      tmem_ld32(d, v);
      if constexpr (rest != 0) {
        add_rest(d + rest, v);
        add_rest(d + rest + 16, v + 16);
      }
      tc_fence_before();
      mbar_arrive(&y.acc_free[j & 1]);
    } else {
#pragma unroll
      for (int i = 0; i < 32; ++i) v[i] = 0u;
    }
    if (tma_out && a.addend != nullptr) mbar_wait(&y.add_full[j % bufs], (j / bufs) & 1, &y.abort, a.st, 27);
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      uint8_t* p = buf + swizzled(row, c0 / 8 + q);
      st_shared_v4(p, combine(a.addend != nullptr ? ld_shared_v4(p) : make_uint4(0, 0, 0, 0), v + 8 * q));
    }
  };
  // The addend's rows of tile j, and rows of a finished tile: a thread has
  // chunk tid % 8 of rows tid / 8 + 32 i in both, so that it may fetch into
  // what it has stored.
  const int cw = kTma ? 16 : a.cw;
  int token[4] = {-1, -1, -1, -1};
  if (!tma_out && warp < 8)
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if ((tid >> 3) + 32 * i < t.count) token[i] = a.perm[t.start + (tid >> 3) + 32 * i];
  auto load_addend = [&](int j) {
    if (a.addend == nullptr || j >= n) return;
    const uint32_t buf = smem_u32(tiles) + (j % bufs) * kTileBytes;
    const int64_t at = static_cast<int64_t>(j0 + j) * kCols + (tid & 7) * 8;
    load_chunks<kCopy, 4>(cw, [&](int i) {
      return Chunk{buf + swizzled((tid >> 3) + 32 * i, tid & 7), a.addend + static_cast<int64_t>(max(token[i], 0)) * C,
                   at, token[i] >= 0 ? C - at : 0};
    });
  };
  auto store_rows = [&](int j, const uint8_t* buf) {
    const int64_t at = static_cast<int64_t>(j0 + j) * kCols + (tid & 7) * 8;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (token[i] < 0 || at >= C) continue;
      const int row = (tid >> 3) + 32 * i, q = tid & 7;
      const uint4 w = ld_shared_v4(buf + swizzled(row, q));
      uint16_t* o = a.out + static_cast<int64_t>(token[i]) * C + at;
      if (cw == 16) {
        *reinterpret_cast<uint4*>(o) = w;
        continue;
      }
      const int s = static_cast<int>(reinterpret_cast<uintptr_t>(o) & 15) / 2;
      if (s == 0 && C - at >= 8) {
        *reinterpret_cast<uint4*>(o) = w;
        continue;
      }
      // the aligned 16 bytes that hold this chunk's first element: its first
      // 8 - s elements after the last s of the chunk before
      const bool whole = q > 0 && C - at >= 8 - s;
      if (whole) {
        const uint4 before = ld_shared_v4(buf + swizzled(row, q - 1));
        *reinterpret_cast<uint4*>(o - s) = realign(before, w, 16 - 2 * s);
      }
      // what no whole 16 bytes of this tile hold
      const int from = whole ? 8 - s : 0, to = static_cast<int>(min(C - at, static_cast<int64_t>(8)));
      const bool next = q < 7 && C - at >= 16 - s;   // the next chunk's thread stores the rest
      const int end = next ? min(to, 8 - s) : to;
      const uint32_t* e = reinterpret_cast<const uint32_t*>(&w);
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (k >= from && k < end) o[k] = static_cast<uint16_t>(e[k >> 1] >> (16 * (k & 1)));
    }
  };

  int fetched = 0, added = 0, multiplied = 0;   // column tiles, by the thread that issues them
  if constexpr (kTma) {
    if (warp == 8) {
      for (int j = 0; j < n; ++j) {
        const int c0 = (j0 + j) * kCols;
        if (adapter && lane == 0 && fetched == j &&
            (j < 2 || mbar_wait(&y.w_free[j & 1], ((j >> 1) - 1) & 1, &y.abort, a.st, 28))) {
          fetched = j + 1;
          uint8_t* ws = wbuf + (j & 1) * expand_w_bytes(r16);
          if constexpr (kMN) {
            mbar_arrive_expect_tx(&y.w_full[j & 1], r16 * kRowBytes);
            tma_load_3d(ws, &a.tmW, c0, 0, t.group, &y.w_full[j & 1]);
          } else {
            mbar_arrive_expect_tx(&y.w_full[j & 1], expand_w_bytes(r16));
            for (int k = 0; k < expand_blocks(r16); ++k)
              tma_load_3d(ws + k * 64 * kRowBytes, &a.tmW, 64 * k, c0, t.group, &y.w_full[j & 1]);
          }
        }
        if (a.addend != nullptr && tma_out && lane == 0 && added == j &&
            (j < bufs || mbar_wait(&y.add_free[j % bufs], (j / bufs - 1) & 1, &y.abort, a.st, 29))) {
          added = j + 1;
          uint64_t* bar = &y.add_full[j % bufs];
          mbar_arrive_expect_tx(bar, kTileBytes);
          tma_load_2d(tiles + (j % bufs) * kTileBytes, &a.tmAdd, c0, t.row0, bar);
        }
        __syncwarp();
        // mid, the output of the kernel before this one, after the first
        // tile's W and addend are on their way
        if (j == 0 && adapter) {
          grid_dependency_wait();
          if (lane == 0) {
            mbar_arrive_expect_tx(&y.mid_full, 2 * expand_mid_bytes(r16));
            for (int p = 0; p < 2; ++p)
              for (int k = 0; k < expand_blocks(r16); ++k)
                tma_load_2d(mids + p * expand_mid_bytes(r16) + k * 128 * kRowBytes, &a.tmMid, 64 * k,
                            p * a.M + t.start, &y.mid_full);
          }
        }
      }
    } else if (tid == 288) {
      if (adapter && mbar_wait(&y.mid_full, 0, &y.abort, a.st, 30)) {
        for (int j = 0; j < n; multiplied = ++j) {
          if (!mbar_wait(&y.w_full[j & 1], (j >> 1) & 1, &y.abort, a.st, 31)) break;
          if (j >= 2 && !mbar_wait(&y.acc_free[j & 1], ((j >> 1) - 1) & 1, &y.abort, a.st, 32)) break;
          tc_fence_after();
          multiply(j);
        }
      }
    } else if (warp < 8 && tma_out) {
      for (int j = 0; j < n; ++j) {
        uint8_t* buf = tiles + (j % bufs) * kTileBytes;
        // without an addend nothing else keeps this buffer's last store ahead
        if (a.addend == nullptr && j >= bufs)
          mbar_wait(&y.add_free[j % bufs], (j / bufs - 1) & 1, &y.abort, a.st, 29);
        finish(j, buf);
        fence_proxy_async_smem();
        named_bar_sync(1, 256);
        if (tid == 0) {
          tma_store_2d(&a.tmOut, (j0 + j) * kCols, t.row0, buf);
          bulk_commit();
          bulk_wait_read<1>();   // the store of tile j - 1 has read its buffer
          if (j > 0) mbar_arrive(&y.add_free[(j - 1) % bufs]);
        }
        __syncwarp();
      }
      if (tid == 0) bulk_wait_read<0>();   // shared memory is read; the writes end with the kernel
    } else if (warp < 8) {
      // rows here and there: by the threads themselves (their 128-byte rows
      // are faster fetched and stored so than four at a time by TMA)
      for (int j = 0; j < bufs - 1; ++j) {
        load_addend(j);
        cp_async_commit();
      }
      for (int j = 0; j < n; ++j) {
        uint8_t* buf = tiles + (j % bufs) * kTileBytes;
        load_addend(j + bufs - 1);
        cp_async_commit();
        cp_async_wait<kAddTiles - 1>();
        named_bar_sync(1, 256);
        finish(j, buf);
        named_bar_sync(1, 256);
        store_rows(j, buf);
      }
      cp_async_wait<0>();
    }
    __syncwarp();
  } else if (warp < 8) {
    // the same, gathered by all of warps 0-7, one tile ahead
    grid_dependency_wait();
    const int chunks = r16 / 8;
    const uint16_t* W = a.W + static_cast<int64_t>(adapter ? t.group : 0) * R * C;
    auto load_w = [&](int j) {
      if (!adapter) return;
      const int64_t c0 = static_cast<int64_t>(j0 + j) * kCols;
      const uint32_t ws = smem_u32(wbuf) + (j & 1) * expand_w_bytes(r16);
      if constexpr (kMN) {
        for (int i = tid; i < r16 * 8; i += kThreads) {
          const int k = i >> 3, c = i & 7;
          load_chunk<kCopy>(a.cw, Chunk{ws + swizzled(k, c), W + min(k, R - 1) * C, c0 + c * 8,
                                        k < R ? C - (c0 + c * 8) : 0});
        }
      } else {
        for (int i = tid; i < 64 * chunks; i += kThreads) {
          const int row = i / chunks, c = i % chunks;
          load_chunk<kCopy>(a.rw, Chunk{ws + (c >> 3) * 64 * kRowBytes + swizzled(row, c & 7),
                                        W + min(c0 + row, C - 1) * R, c * 8, c0 + row < C ? R - c * 8 : 0});
        }
      }
    };
    if (adapter)
      for (int i = tid; i < t.count * chunks; i += kThreads) {
        const int row = i / chunks, c = i % chunks;
        const uint32_t dst = smem_u32(mids) + (c >> 3) * 128 * kRowBytes + swizzled(row, c & 7);
        const uint16_t* m = a.mid + static_cast<int64_t>(t.start + row) * R;
        load_chunk<kCopy>(a.rw, Chunk{dst, m, c * 8, R - c * 8});
        load_chunk<kCopy>(a.mw, Chunk{dst + expand_mid_bytes(r16), m + static_cast<int64_t>(a.M) * R, c * 8, R - c * 8});
      }
    // Buffers of tile j + 1: w of tile j - 1 was read by products that tile
    // j - 1's outputs waited for, its addend buffer left before the barrier
    // that ended tile j + 1 - bufs.  Copies that go through registers are
    // waited for while the tile's products run.
    constexpr bool ahead = kCopy == kByAsync;
    auto fetch = [&](int j) {
      if (j < n) {
        load_w(j);
        load_addend(j);
      }
      cp_async_commit();
    };
    fetch(0);
    for (int j = 0; j < n; ++j) {
      if (ahead) {
        fetch(j + 1);
        cp_async_wait<1>();
      } else {
        cp_async_wait<0>();
      }
      fence_proxy_async_smem();
      tc_fence_before();
      named_bar_sync(1, 256);
      if (adapter && tid == 0) {
        tc_fence_after();
        multiply(j);
        multiplied = j + 1;
      }
      __syncwarp();
      if (!ahead) fetch(j + 1);
      uint8_t* buf = tiles + (j % bufs) * kTileBytes;
      finish(j, buf);
      named_bar_sync(1, 256);
      store_rows(j, buf);
      named_bar_sync(1, 256);
    }
    cp_async_wait<0>();
  }
  grid_dependents_launch();
  grid_dependency_wait();   // what follows this kernel may rely on what came before it
  tc_fence_before();
  __syncthreads();
  if (aborted(y.abort)) {
    wind_down(y.w_full, fetched, y.acc_full, multiplied, 2, a.st);
    wind_down(y.add_full, added, nullptr, 0, bufs, a.st);
    if (fetched > 0) mbar_wait_out(&y.mid_full, 0, a.st, 37);
    __syncthreads();
  }
  if (warp == 0) tmem_dealloc(y.tmem, 2 * acc);
}

// ---- gradients of A and B ---------------------------------------------------

struct GradSide {   // gB (of g and t) or gA (of x and u)
  CUtensorMap tmX, tmX1, tmU;   // with kTma: X, box 64 x 64 and 64 x 1; mid, box 64 x 64
  const uint16_t* mid;    // [2, M, R], in the plan's order
  const uint16_t* X;      // [M, C]
  uint16_t* grad;         // per group [R, C] (rank_major) or [C, R]
  const float* scale;
  int64_t C;
  int64_t tiles;          // clusters: strips of 128 columns times groups
  int strips, cw;
  bool rank_major;
  bool wait;              // mid is the output of the kernel before this one
};
struct GradArgs {
  GradSide side[2];       // the second one's clusters follow the first one's
  const int* offset;
  const int* perm;
  DevStatus* st;
  int M, R, rw, mw;       // mw: the copy width of mid's second part
  int ranks;              // CTAs per cluster
  bool bf16;
  bool first;             // the call's first kernel: clears the status
};

__host__ __device__ constexpr int grad_mid_bytes(int r16) { return (r16 > 64 ? 2 : 1) * 64 * kRowBytes; }
__host__ __device__ constexpr int grad_stage_bytes(int r16) { return 2 * 64 * kRowBytes + 2 * grad_mid_bytes(r16); }

// grad[c, j] = scale sum_m X[m, c] mid[m, j] over a group's tokens: one
// cluster per (128 columns of X, group), its CTAs splitting the tokens.
// Bound by reading X once: both gradients of one adapter, 8192 tokens, 4096
// -> 11008, rank 64, take 51 us, 4.9 TB/s; in a launch each, 37 and 31 us.
template <int kStages, Copy kCopy>
__global__ void __launch_bounds__(kThreads, 2) grad_kernel(const __grid_constant__ GradArgs a) {
  constexpr bool kTma = kCopy == kByTma;
  extern __shared__ uint8_t smem_raw[];
  __shared__ Sync y;
  const int tid = threadIdx.x, ranks = a.ranks, rank = blockIdx.x % ranks, R = a.R, r16 = rank16(R);
  int64_t tile = blockIdx.x / ranks;
  const bool second = tile >= a.side[0].tiles;
  const GradSide& d = a.side[second ? 1 : 0];
  if (second) tile -= a.side[0].tiles;
  const int64_t C = d.C, e = tile / d.strips, c0 = tile % d.strips * 128;
  const bool rank_major = d.rank_major;
  if (kTma && tid == 0) {
    tma_prefetch_desc(&d.tmX);
    tma_prefetch_desc(&d.tmU);
  }
  if (a.first && blockIdx.x == 0 && tid == 0) *a.st = DevStatus{0, 0, 0, 0};
  const int start = a.offset[e], tokens = a.offset[e + 1] - start;
  const int cols = static_cast<int>(min(static_cast<int64_t>(128), C - c0));
  uint16_t* grad = d.grad + e * R * C;
  if (tokens == 0) {
    grid_dependency_wait();
    if (rank == 0)
      for (int i = tid; i < cols * R; i += kThreads)
        grad[rank_major ? i / cols * C + c0 + i % cols : c0 * R + i] = 0;
    return;
  }
  const uint32_t base = align1024(smem_u32(smem_raw));
  const int stage_bytes = grad_stage_bytes(r16);
  const int nb = (tokens + 63) / 64;
  const int b0 = static_cast<int>(static_cast<int64_t>(nb) * rank / ranks);
  const int n = static_cast<int>(static_cast<int64_t>(nb) * (rank + 1) / ranks) - b0;
  const int chunks = r16 / 8;
  const uint32_t rest = a.bf16 ? 0u : tmem_columns(r16), columns = tmem_columns(r16) + rest;
  sync_setup(y, columns);

  const int first = a.perm[start];
  const bool run = a.perm[start + tokens - 1] - first == tokens - 1;   // consecutive tokens
  const uint32_t idesc = instruction(r16, true, true, a.bf16);
  auto multiply = [&](int it) {   // one thread: the products of a stage
    const int s = it % kStages;
    const uint32_t xs = base + s * stage_bytes, us = xs + 2 * 64 * kRowBytes;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const uint64_t x = desc_mn(xs, k, 64 * kRowBytes);
      umma_f16(y.tmem, x, desc_mn(us, k, 64 * kRowBytes), idesc, it > 0 || k > 0 ? 1u : 0u);
      umma_f16(y.tmem + rest, x, desc_mn(us + grad_mid_bytes(r16), k, 64 * kRowBytes), idesc,
               it > 0 || k > 0 || rest == 0 ? 1u : 0u);
    }
    umma_commit(&y.done[s]);
    if (it == n - 1) umma_commit(&y.last);
  };
  // A block of consecutive tokens of X is fetched as a box, others four rows
  // at a time.  The reduction runs over tokens, so a last block of fewer than
  // 64 must not reach into other groups' rows of X (whatever they hold would
  // be multiplied by zero): its last token is repeated, and the rows of mid
  // past it are set to zero before its products.
  int fetched = 0, multiplied = 0;   // steps, by the warps that issue them
  if constexpr (kTma) {
    if (tid < 32) {
      uint8_t* stages = smem_raw + (base - smem_u32(smem_raw));
      const int half = tid >> 4, quad = tid & 15;   // lanes 0-15 fetch the first 64 columns, 16-31 the others
      auto rows_of = [&](int it, int(&rows)[4]) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int k = min((b0 + it) * 64 + 4 * quad + i, tokens - 1);
          rows[i] = run ? first + k : a.perm[start + k];
        }
      };
      int rows[4], next[4];
      rows_of(0, next);
      if (d.wait) grid_dependency_wait();
      for (int it = 0; it < n; ++it) {
        const int s = it % kStages, m0 = (b0 + it) * 64;
        uint8_t *xs = stages + s * stage_bytes, *us = xs + 2 * 64 * kRowBytes;
#pragma unroll
        for (int i = 0; i < 4; ++i) rows[i] = next[i];
        rows_of(it + 1, next);
        const int row0 = __shfl_sync(0xffffffffu, rows[0], 0);
        const bool box = __all_sync(0xffffffffu, rows[0] == row0 + 4 * quad && rows[3] == rows[0] + 3);   // ascending
        if (it >= kStages &&
            !__all_sync(0xffffffffu, mbar_wait(&y.done[s], (it / kStages - 1) & 1, &y.abort, a.st, 23)))
          break;
        fetched = it + 1;
        if (tid == 0) {
          mbar_arrive_expect_tx(&y.full[s], stage_bytes);
          for (int k = 0; k < 2; ++k) {
            uint8_t* u = us + k * grad_mid_bytes(r16);
            tma_load_2d(u, &d.tmU, 0, k * a.M + start + m0, &y.full[s]);
            if (r16 > 64) tma_load_2d(u + 64 * kRowBytes, &d.tmU, 64, k * a.M + start + m0, &y.full[s]);
          }
          if (box) {
            tma_load_2d(xs, &d.tmX, static_cast<int>(c0), row0, &y.full[s]);
            tma_load_2d(xs + 64 * kRowBytes, &d.tmX, static_cast<int>(c0) + 64, row0, &y.full[s]);
          }
        }
        __syncwarp();   // the stage is armed before its gathers arrive
        if (!box)
          tma_gather4(xs + (half * 64 + quad * 4) * kRowBytes, &d.tmX1, static_cast<int>(c0) + 64 * half, rows,
                      &y.full[s]);
      }
    } else if (tid < 64) {
      for (int it = 0; it < n; multiplied = ++it) {
        if (!__all_sync(0xffffffffu, mbar_wait(&y.full[it % kStages], (it / kStages) & 1, &y.abort, a.st, 26))) break;
        const int left = tokens - (b0 + it) * 64;
        if (left < 64) {
          uint8_t* us = smem_raw + (base - smem_u32(smem_raw)) + it % kStages * stage_bytes + 2 * 64 * kRowBytes;
          for (int i = left * 8 + (tid & 31); i < 64 * 8; i += 32)
            for (int k = 0; k < 2 * grad_mid_bytes(r16); k += 64 * kRowBytes)
              st_shared_v4(us + k + i * 16, make_uint4(0, 0, 0, 0));
          fence_proxy_async_smem();
        }
        __syncwarp();
        if (tid == 32) {
          tc_fence_after();
          multiply(it);
        }
        __syncwarp();
      }
    }
    __syncwarp();
  } else {
    if (d.wait) grid_dependency_wait();
    // the tokens of a step are read one step before their copies are issued
    constexpr int kMidPer = 4;   // up to 64 rows x 16 chunks of mid over 256 threads
    int xm[4], um[kMidPer];
    auto rows_of = [&](int b) {
      const int m0 = (b0 + b) * 64;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int k = m0 + (tid >> 4) + 16 * i;
        xm[i] = k < tokens ? (run ? first + k : a.perm[start + k]) : -1;
      }
#pragma unroll
      for (int i = 0; i < kMidPer; ++i) {
        const int k = m0 + (tid + i * kThreads) / chunks;
        um[i] = tid + i * kThreads < 64 * chunks && k < tokens ? start + k : -1;
      }
    };
    auto load = [&](int b, int s) {   // of the rows that rows_of(b) found
      const uint32_t xs = base + s * stage_bytes, us = xs + 2 * 64 * kRowBytes;
      const int c = tid & 15;
      load_chunks<kCopy, 4>(d.cw, [&](int i) {
        return Chunk{xs + (c >> 3) * 64 * kRowBytes + swizzled((tid >> 4) + 16 * i, c & 7),
                     d.X + static_cast<int64_t>(max(xm[i], 0)) * C, c0 + c * 8, xm[i] >= 0 ? C - (c0 + c * 8) : 0};
      });
#pragma unroll
      for (int i = 0; i < kMidPer; ++i) {
        const int at = tid + i * kThreads;
        if (at >= 64 * chunks) break;
        const int k = at / chunks, q = at % chunks;
        const uint32_t dst = us + (q >> 3) * 64 * kRowBytes + swizzled(k, q & 7);
        const uint16_t* row = d.mid + static_cast<int64_t>(max(um[i], 0)) * R;
        const int64_t valid = um[i] >= 0 ? R - q * 8 : 0;
        load_chunk<kCopy>(a.rw, Chunk{dst, row, q * 8, valid});
        load_chunk<kCopy>(a.mw, Chunk{dst + grad_mid_bytes(r16), row + static_cast<int64_t>(a.M) * R, q * 8, valid});
      }
      rows_of(b + 1);
    };
    rows_of(0);
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) {
      if (i < n) load(i, i);
      cp_async_commit();
    }
    for (int it = 0; it < n; ++it) {
      cp_async_wait<kStages - 2>();
      fence_proxy_async_smem();
      __syncthreads();
      if (tid == 0) multiply(it);
      multiplied = it + 1;
      const int next = it + kStages - 1;
      if (next < n) {
        if (it > 0) mbar_wait(&y.done[(it - 1) % kStages], ((it - 1) / kStages) & 1, &y.abort, a.st, 23);
        load(next, next % kStages);
      }
      cp_async_commit();
    }
  }
  float* red = reinterpret_cast<float*>(smem_raw + (base - smem_u32(smem_raw)));
  if (n > 0) {
    mbar_wait(&y.last, 0, &y.abort, a.st, 24);
    cp_async_wait<0>();
    __syncwarp();
    tc_fence_after();
    __syncthreads();
    if (aborted(y.abort)) {
      wind_down(y.full, fetched, y.done, multiplied, kStages, a.st);
      __syncthreads();
    }
    spill(y.tmem, r16, red, rest);
  } else {   // a group with fewer token blocks than CTAs
    for (int i = tid; i < 128 * red_pitch(r16); i += kThreads) red[i] = 0.f;
  }
  sync_end(y, columns);
  grid_dependents_launch();
  cluster_sync();
  const int rows = (128 + ranks - 1) / ranks, row0 = rank * rows;
  const float scale = d.scale != nullptr ? d.scale[e] : 1.f;
  const int quads = r16 / 4;
  for (int i = tid; i < rows * quads; i += kThreads) {
    // neighbouring threads on neighbouring elements of the gradient
    const int row = row0 + (rank_major ? i % rows : i / quads), j = (rank_major ? i / rows : i % quads) * 4;
    if (row >= cols || row >= 128 || j >= R) continue;
    float s[4];
    cluster_sum4(base, row * red_pitch(r16) + j, ranks, s);
    if (!rank_major && R % 4 == 0) {
      *reinterpret_cast<uint2*>(grad + (c0 + row) * R + j) =
          make_uint2(to_16(scale * s[0], a.bf16) | static_cast<uint32_t>(to_16(scale * s[1], a.bf16)) << 16,
                     to_16(scale * s[2], a.bf16) | static_cast<uint32_t>(to_16(scale * s[3], a.bf16)) << 16);
    } else {
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (j + k < R)
          grad[rank_major ? (j + k) * C + c0 + row : (c0 + row) * R + j + k] = to_16(scale * s[k], a.bf16);
    }
  }
  // what follows this kernel may rely on what came before it
  grid_dependency_wait();
  cluster_sync();
}

// The same for more strips than CTAs (many adapters, or wide layers of few):
// each CTA takes strip after strip, whole, with the fetches of the next one
// under way while the last one leaves tensor memory.  Warps 0-3 turn
// accumulators into gradients, warp 4 fetches mid and blocks of consecutive
// tokens of X by TMA, warps 6-9 gather the other blocks' rows, warp 5 issues
// the products.
// 8192 tokens of 32 adapters, 4096 -> 11008, rank 64: both gradients take 81 us
// by it and 159 us by one CTA per strip; 8 adapters, interleaved, 57 us, and
// 92 us with the rows gathered by TMA, four a request.  Bound by reading X
// where the adapters' shares of the batch are alike; 8 adapters of uneven
// shares take 71 us (a CTA's strips are dealt out without regard to them).
constexpr int kManyThreads = 320, kGatherers = 128;
struct ManySync {
  uint64_t full[kMaxStages], done[kMaxStages], acc_full[2], acc_free[2];
  uint32_t tmem;
  int abort;
};
template <int kStages>
__global__ void __launch_bounds__(kManyThreads, 2) grad_many_kernel(const __grid_constant__ GradArgs a) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ ManySync y;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, R = a.R, r16 = rank16(R);
  if (a.first && blockIdx.x == 0 && tid == 0) *a.st = DevStatus{0, 0, 0, 0};
  if (tid == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&y.full[i], 1 + kGatherers);
      mbar_init(&y.done[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&y.acc_full[i], 1);
      mbar_init(&y.acc_free[i], 128);
    }
    y.abort = 0;
    fence_mbar_init();
  }
  // of one accumulator, with that of the second parts; two of them where two
  // CTAs' fit
  const uint32_t rest = a.bf16 ? 0u : tmem_columns(r16), columns = tmem_columns(r16) + rest;
  const int more = columns <= 128 ? 1 : 0;   // accumulator acc & more, its use acc >> more
  if (warp == 0) {
    tmem_alloc(&y.tmem, columns << more);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();

  const int stage_bytes = grad_stage_bytes(r16);
  uint8_t* stages = smem_raw + (align1024(smem_u32(smem_raw)) - smem_u32(smem_raw));
  struct Strip {
    bool second;
    int e, start, tokens;
    int64_t c0;
  };
  const int64_t strips = a.side[0].tiles + a.side[1].tiles;
  auto strip_of = [&](int64_t i) {
    Strip t{i >= a.side[0].tiles, 0, 0, 0, 0};
    if (i >= strips) return t;
    const GradSide& d = a.side[t.second];
    if (t.second) i -= a.side[0].tiles;
    t.e = static_cast<int>(i / d.strips);
    t.c0 = i % d.strips * 128;
    t.start = a.offset[t.e];
    t.tokens = a.offset[t.e + 1] - t.start;
    return t;
  };
  const int64_t step = gridDim.x;
  // a block's first and last token; 64 consecutive ones are a box (they ascend)
  auto ends_of = [&](const Strip& t, int it, int(&e)[2]) {
    if (it * 64 >= t.tokens) return;
    e[0] = a.perm[t.start + it * 64];
    e[1] = a.perm[t.start + min(it * 64 + 63, t.tokens - 1)];
  };
  auto is_box = [&](const Strip& t, int it, const int(&e)[2]) {
    return it * 64 + 64 <= t.tokens && e[1] - e[0] == 63;
  };
  int fetched = 0, multiplied = 0;   // steps, by the threads that issue them
  bool going = true;                 // false once a wait of this thread ran out
  if (tid == 128) {
    int ends[2] = {0, 0};
    Strip t = strip_of(blockIdx.x);
    ends_of(t, 0, ends);
    bool waited = false;
    int& at = fetched;
    for (int64_t i = blockIdx.x; i < strips && going; i += step) {
      const Strip after = strip_of(i + step);
      const GradSide& d = a.side[t.second];
      const int n = (t.tokens + 63) / 64, c0 = static_cast<int>(t.c0);
      if (d.wait && !waited) {
        grid_dependency_wait();
        waited = true;
      }
      for (int it = 0; it < n; ++it, ++at) {
        const int s = at % kStages, row0 = ends[0];
        const bool box = is_box(t, it, ends);
        uint8_t *xs = stages + s * stage_bytes, *us = xs + 2 * 64 * kRowBytes;
        if (it + 1 < n) ends_of(t, it + 1, ends);
        else ends_of(after, 0, ends);
        if (at >= kStages && !mbar_wait(&y.done[s], (at / kStages - 1) & 1, &y.abort, a.st, 23)) {
          going = false;
          break;
        }
        mbar_arrive_expect_tx(&y.full[s], box ? stage_bytes : stage_bytes - 2 * 64 * kRowBytes);
        for (int k = 0; k < 2; ++k) {
          uint8_t* u = us + k * grad_mid_bytes(r16);
          tma_load_2d(u, &d.tmU, 0, k * a.M + t.start + it * 64, &y.full[s]);
          if (r16 > 64) tma_load_2d(u + 64 * kRowBytes, &d.tmU, 64, k * a.M + t.start + it * 64, &y.full[s]);
        }
        if (box) {
          tma_load_2d(xs, &d.tmX, c0, row0, &y.full[s]);
          tma_load_2d(xs + 64 * kRowBytes, &d.tmX, c0 + 64, row0, &y.full[s]);
        }
      }
      if (n == 0) ends_of(after, 0, ends);
      t = after;
    }
  } else if (warp >= 6) {
    // the other blocks' rows of X, 16 threads a row; a stage is passed on once
    // the next one's copies are under way
    const int g = tid - 6 * 32, q = g & 15, r0 = g >> 4;
    int ends[2] = {0, 0}, next[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) next[k] = 0;
    auto rows_of = [&](const Strip& t, int it) {
      ends_of(t, it, ends);
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (t.tokens > 0) next[k] = a.perm[t.start + min(it * 64 + r0 + 8 * k, t.tokens - 1)];
    };
    int pending = -1;   // the stage whose copies may still be under way
    auto pass_on = [&] {
      if (pending < 0) return;
      fence_proxy_async_smem();
      mbar_arrive(&y.full[pending]);
      pending = -1;
    };
    Strip t = strip_of(blockIdx.x);
    rows_of(t, 0);
    int at = 0;
    for (int64_t i = blockIdx.x; i < strips && going; i += step) {
      const Strip after = strip_of(i + step);
      const GradSide& d = a.side[t.second];
      const int n = (t.tokens + 63) / 64;
      const bool in = t.c0 + q * 8 < d.C;
      const uint16_t* X = d.X + (in ? t.c0 + q * 8 : 0);
      for (int it = 0; it < n; ++it, ++at) {
        const int s = at % kStages;
        const bool box = is_box(t, it, ends);
        int rows[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) rows[k] = next[k];
        if (it + 1 < n) rows_of(t, it + 1);
        else rows_of(after, 0);
        if (at >= kStages && !mbar_wait(&y.done[s], (at / kStages - 1) & 1, &y.abort, a.st, 34)) {
          going = false;
          break;
        }
        if (box) {
          cp_async_wait<0>();
          pass_on();
          mbar_arrive(&y.full[s]);
          continue;
        }
        const uint32_t xs = smem_u32(stages + s * stage_bytes) + (q >> 3) * 64 * kRowBytes;
#pragma unroll
        for (int k = 0; k < 8; ++k)
          cp_async<16>(xs + swizzled(r0 + 8 * k, q & 7), X + static_cast<int64_t>(rows[k]) * d.C, in);
        cp_async_commit();
        cp_async_wait<1>();
        pass_on();
        pending = s;
      }
      if (n == 0) rows_of(after, 0);
      t = after;
    }
    cp_async_wait<0>();
    pass_on();
  } else if (warp == 5) {
    const uint32_t idesc = instruction(r16, true, true, a.bf16);
    int& at = multiplied;
    int acc = 0;   // strips with tokens so far
    Strip t = strip_of(blockIdx.x);
    for (int64_t i = blockIdx.x; i < strips && going; i += step) {
      const Strip after = strip_of(i + step);
      const int n = (t.tokens + 63) / 64;
      if (n > 0 && acc > more) {
        going = __all_sync(0xffffffffu, mbar_wait(&y.acc_free[acc & more], ((acc >> more) - 1) & 1, &y.abort, a.st, 33));
        if (!going) break;
        tc_fence_after();
      }
      for (int it = 0; it < n; ++it, ++at) {
        const int s = at % kStages;
        going = __all_sync(0xffffffffu, mbar_wait(&y.full[s], (at / kStages) & 1, &y.abort, a.st, 26));
        if (!going) break;
        uint8_t* us = stages + s * stage_bytes + 2 * 64 * kRowBytes;
        const int left = t.tokens - it * 64;
        if (left < 64) {
          for (int j = left * 8 + lane; j < 64 * 8; j += 32)
            for (int k = 0; k < 2 * grad_mid_bytes(r16); k += 64 * kRowBytes)
              st_shared_v4(us + k + j * 16, make_uint4(0, 0, 0, 0));
          fence_proxy_async_smem();
        }
        __syncwarp();
        if (lane == 0) {
          tc_fence_after();
          const uint32_t x0 = smem_u32(us) - 2 * 64 * kRowBytes, u0 = smem_u32(us);
          const uint32_t out = y.tmem + (acc & more) * columns;
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const uint64_t x = desc_mn(x0, k, 64 * kRowBytes);
            umma_f16(out, x, desc_mn(u0, k, 64 * kRowBytes), idesc, it > 0 || k > 0 ? 1u : 0u);
            umma_f16(out + rest, x, desc_mn(u0 + grad_mid_bytes(r16), k, 64 * kRowBytes), idesc,
                     it > 0 || k > 0 || rest == 0 ? 1u : 0u);
          }
          umma_commit(&y.done[s]);
          if (it == n - 1) umma_commit(&y.acc_full[acc & more]);
        }
        __syncwarp();
      }
      if (n > 0) ++acc;
      t = after;
    }
  } else if (warp < 4) {
    int acc = 0;
    Strip t = strip_of(blockIdx.x);
    for (int64_t i = blockIdx.x; i < strips; i += step) {
      const Strip after = strip_of(i + step);
      const GradSide& d = a.side[t.second];
      const int64_t C = d.C, c = t.c0 + tid;
      uint16_t* grad = d.grad + t.e * R * C;
      const float scale = d.scale != nullptr ? d.scale[t.e] : 1.f;
      if (t.tokens > 0) {
        mbar_wait(&y.acc_full[acc & more], (acc >> more) & 1, &y.abort, a.st, 24);
        __syncwarp();
        tc_fence_after();
      }
      for (int j = 0; j < r16; j += 16) {
        uint32_t v[16];
        __syncwarp();
        if (t.tokens > 0) {
          const uint32_t d = y.tmem + (static_cast<uint32_t>(warp * 32) << 16) + (acc & more) * columns + j;
          tmem_ld16(d, v);
          if (rest != 0) add_rest(d + rest, v);
        } else {
#pragma unroll
          for (int k = 0; k < 16; ++k) v[k] = 0u;
        }
        if (c >= C) continue;
        if (d.rank_major) {
#pragma unroll
          for (int k = 0; k < 16; ++k)
            if (j + k < R) grad[(j + k) * C + c] = to_16(scale * __uint_as_float(v[k]), a.bf16);
        } else {
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            uint32_t w[4];
#pragma unroll
            for (int k = 0; k < 4; ++k)
              w[k] = to_16(scale * __uint_as_float(v[8 * q + 2 * k]), a.bf16) |
                     static_cast<uint32_t>(to_16(scale * __uint_as_float(v[8 * q + 2 * k + 1]), a.bf16)) << 16;
            if (j + 8 * q < R) *reinterpret_cast<uint4*>(grad + c * R + j + 8 * q) = make_uint4(w[0], w[1], w[2], w[3]);
          }
        }
      }
      if (t.tokens > 0) {
        __syncwarp();
        tc_fence_before();
        mbar_arrive(&y.acc_free[acc & more]);
        ++acc;
      }
      t = after;
    }
  }
  __syncwarp();
  grid_dependents_launch();
  tc_fence_before();
  __syncthreads();
  if (aborted(y.abort)) {
    wind_down(y.full, fetched, y.done, multiplied, kStages, a.st);
    __syncthreads();
  }
  if (warp == 0) tmem_dealloc(y.tmem, columns << more);
  // what follows this kernel may rely on what came before it
  grid_dependency_wait();
}

// ---- few tokens: t and y in one launch --------------------------------------

struct FewArgs {
  const uint16_t *x, *A, *B, *base;   // base or NULL; may be y
  uint16_t *y, *t;                    // t [2, M, R]
  int64_t plane;                      // M R
  const float* scale;
  const Tile* tiles;
  const int* perm;
  DevStatus* st;
  int64_t K, N;
  int R, E;
};

// D (16 x 8) += A (16 x 16) B (16 x 8).  A thread's 4 + 4 elements of a row of
// A and of a column of B may stand for any 4 of the 16 places of the
// reduction, as long as both take the same: it holds consecutive ones.
template <bool kBf16>
__device__ __forceinline__ void mma_16x8(float (&d)[4], uint2 a0, uint2 a1, uint2 b) {
  if constexpr (kBf16)
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a0.x), "r"(a1.x), "r"(a0.y), "r"(a1.y), "r"(b.x), "r"(b.y));
  else
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a0.x), "r"(a1.x), "r"(a0.y), "r"(a1.y), "r"(b.x), "r"(b.y));
}

// One cluster of 8 CTAs per tile of up to 8 tokens of one adapter.  Each CTA
// reads an eighth of A[e] and of the tokens' features straight into the
// operands of warp products (ranks as the rows, tokens as the columns), the
// cluster adds up t, then each CTA turns an eighth of B[e] into an eighth of
// y.  Bound by reading A[e] and B[e] once; B's part is on its way to L2 while
// t is formed.  A tensor-memory tile would be empty but for these 8 rows of
// 128, and the two kernels of long batches cost two launches: 64 tokens of 64
// adapters, 4096 -> 4096, rank 16, took 18 + 29 us by them, 10 us by this one
// (1.9 TB/s of A, B, x and y; latency).
constexpr int kFewRanks = 8;
template <bool kBf16, int kMaxRankTiles>   // tiles of 16 ranks
__global__ void __launch_bounds__(kThreads, kMaxRankTiles > 4 ? 2 : kMaxRankTiles > 1 ? 3 : 4) few_kernel(const FewArgs a) {
  __shared__ __align__(16) float part[kThreads / 32][kMaxRankTiles * 16 * kFewTile];   // per warp, then the CTA's sum
  __shared__ __align__(16) uint16_t ts[2][kFewTile][kMaxRankTiles * 16 + 8];   // t's two parts
  __shared__ __align__(16) float ys[2][kFewTile][128 + 4];
  grid_dependency_wait();
  if (blockIdx.x == 0 && threadIdx.x == 0) *a.st = DevStatus{0, 0, 0, 0};
  const Tile tile = a.tiles[blockIdx.x / kFewRanks];
  if (tile.count == 0) return;
  const int rank = blockIdx.x % kFewRanks, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = lane >> 2, q = lane & 3;
  const int R = a.R, r16 = rank16(R), tiles16 = r16 / 16;
  const bool adapter = tile.group < a.E;
  const int64_t K = a.K, N = a.N;
  // this CTA's columns of y, in steps of 128
  const int64_t steps = (N + 127) / 128;
  const int64_t s0 = steps * rank / kFewRanks, s1 = steps * (rank + 1) / kFewRanks;
  const uint16_t* B = a.B + static_cast<int64_t>(adapter ? tile.group : 0) * N * R;
  const int64_t m_of = a.perm[tile.start + min(g, tile.count - 1)];
  if (adapter) {
    if (tid == 0 && s1 > s0) {
      const int64_t bytes = (min(s1 * 128, N) - s0 * 128) * R * 2;   // rows of B are whole 16-byte units
      asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(B + s0 * 128 * R),
                   "r"(static_cast<uint32_t>(min(bytes, static_cast<int64_t>(1) << 22)))
                   : "memory");
    }
    const uint16_t* A = a.A + static_cast<int64_t>(tile.group) * R * K;
    const uint16_t* x = a.x + m_of * K;
    const int64_t blocks = (K + 31) / 32;
    const int64_t k1 = blocks * (rank + 1) / kFewRanks;
    float d[kMaxRankTiles][4];
#pragma unroll
    for (int i = 0; i < kMaxRankTiles; ++i) d[i][0] = d[i][1] = d[i][2] = d[i][3] = 0.f;
    const uint4 zero = make_uint4(0, 0, 0, 0);
#pragma unroll 2
    for (int64_t kb = blocks * rank / kFewRanks + warp; kb < k1; kb += kThreads / 32) {
      const int64_t k = kb * 32 + q * 8;
      const bool in = k < K;
      const uint4 b = in && g < tile.count ? __ldg(reinterpret_cast<const uint4*>(x + k)) : zero;
#pragma unroll
      for (int i = 0; i < kMaxRankTiles; ++i) {
        if (i >= tiles16) break;
        const int r0 = i * 16 + g, r1 = r0 + 8;
        const uint4 u = in && r0 < R ? __ldg(reinterpret_cast<const uint4*>(A + r0 * K + k)) : zero;
        const uint4 v = in && r1 < R ? __ldg(reinterpret_cast<const uint4*>(A + r1 * K + k)) : zero;
        mma_16x8<kBf16>(d[i], make_uint2(u.x, u.y), make_uint2(v.x, v.y), make_uint2(b.x, b.y));
        mma_16x8<kBf16>(d[i], make_uint2(u.z, u.w), make_uint2(v.z, v.w), make_uint2(b.z, b.w));
      }
    }
    // d: ranks g and g + 8 of each 16, tokens 2 q and 2 q + 1
#pragma unroll
    for (int i = 0; i < kMaxRankTiles; ++i) {
      if (i >= tiles16) break;
      *reinterpret_cast<float2*>(&part[warp][(i * 16 + g) * kFewTile + 2 * q]) = make_float2(d[i][0], d[i][1]);
      *reinterpret_cast<float2*>(&part[warp][(i * 16 + g + 8) * kFewTile + 2 * q]) = make_float2(d[i][2], d[i][3]);
    }
    __syncthreads();
    for (int i = tid; i < r16 * kFewTile; i += kThreads) {
      float s = 0.f;
#pragma unroll
      for (int w = 0; w < kThreads / 32; ++w) s += part[w][i];
      part[0][i] = s;   // read and written by this thread alone
    }
    cluster_sync();
    for (int i = tid * 4; i < r16 * kFewTile; i += kThreads * 4) {
      float s[4];
      cluster_sum4(smem_u32(part[0]), i, kFewRanks, s);
      const int j = i / kFewTile;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int tok = i % kFewTile + k;
        const uint16_t hi = to_16(s[k], kBf16), lo = rest_16(s[k], hi, kBf16);
        ts[0][tok][j] = hi;
        ts[1][tok][j] = lo;
        if (rank == 0 && tok < tile.count && j < R) {
          uint16_t* o = a.t + static_cast<int64_t>(tile.start + tok) * R + j;
          o[0] = hi;
          o[a.plane] = lo;
        }
      }
    }
    __syncthreads();
  } else if (rank == 0) {
    for (int i = tid; i < tile.count * R; i += kThreads) {
      uint16_t* o = a.t + static_cast<int64_t>(tile.start) * R + i;
      o[0] = o[a.plane] = 0;
    }
  }
  // y: warp w on columns 16 w .. 16 w + 15 of a step, then every warp on a token
  const float scale = adapter ? (a.scale != nullptr ? a.scale[tile.group] : 1.f) : 0.f;
  const int64_t m = a.perm[tile.start + min(warp, tile.count - 1)];
  for (int64_t s = s0; s < s1; ++s) {
    const int64_t col = s * 128 + lane * 4;
    const bool out = warp < tile.count && col < N;
    uint2 base = make_uint2(0, 0);
    if (out && a.base != nullptr) base = *reinterpret_cast<const uint2*>(a.base + m * N + col);
    if (adapter) {
      float d[4] = {0.f, 0.f, 0.f, 0.f}, r[4] = {0.f, 0.f, 0.f, 0.f};   // r: of t's second part in fp16
      const int64_t c0 = s * 128 + warp * 16 + g, c1 = c0 + 8;
      const uint2 zero = make_uint2(0, 0);
#pragma unroll 4
      for (int i = 0; i < tiles16; ++i) {
        const int k = i * 16 + q * 4;
        const bool in = k < R;
        const uint2 u = in && c0 < N ? __ldg(reinterpret_cast<const uint2*>(B + c0 * R + k)) : zero;
        const uint2 v = in && c1 < N ? __ldg(reinterpret_cast<const uint2*>(B + c1 * R + k)) : zero;
        const uint2 hi = in ? *reinterpret_cast<const uint2*>(&ts[0][g][k]) : zero;
        const uint2 lo = in ? *reinterpret_cast<const uint2*>(&ts[1][g][k]) : zero;
        if constexpr (!kBf16 && kMaxRankTiles == 1) {   // one accumulator, scaled in between, spares registers
          mma_16x8<kBf16>(d, u, v, lo);
#pragma unroll
          for (int n = 0; n < 4; ++n) d[n] *= kRestDown;
          mma_16x8<kBf16>(d, u, v, hi);
        } else {
          mma_16x8<kBf16>(d, u, v, hi);
          mma_16x8<kBf16>(kBf16 ? d : r, u, v, lo);
        }
      }
      if constexpr (!kBf16 && kMaxRankTiles > 1)
#pragma unroll
        for (int n = 0; n < 4; ++n) d[n] = fmaf(r[n], kRestDown, d[n]);
      float(*buf)[128 + 4] = ys[s & 1];
      const int c = warp * 16 + g;
      buf[2 * q][c] = d[0];
      buf[2 * q + 1][c] = d[1];
      buf[2 * q][c + 8] = d[2];
      buf[2 * q + 1][c + 8] = d[3];
      __syncthreads();
    }
    if (!out) continue;
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    if (adapter) v = *reinterpret_cast<const float4*>(&ys[s & 1][warp][lane * 4]);
    float f[4] = {v.x, v.y, v.z, v.w};
    uint32_t* w = reinterpret_cast<uint32_t*>(&base);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      float lo, hi;
      if constexpr (kBf16) {
        lo = __uint_as_float(w[i] << 16);
        hi = __uint_as_float(w[i] & 0xffff0000u);
      } else {
        const float2 h = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
        lo = h.x;
        hi = h.y;
      }
      lo = fmaf(scale, f[2 * i], lo);
      hi = fmaf(scale, f[2 * i + 1], hi);
      w[i] = to_16(lo, kBf16) | (static_cast<uint32_t>(to_16(hi, kBf16)) << 16);
    }
    *reinterpret_cast<uint2*>(a.y + m * N + col) = base;
  }
  if (adapter) cluster_sync();   // the other CTAs have read this one's sums
}

// ---- launches ---------------------------------------------------------------

struct Problem {
  int64_t M, K, N, E;
  int R;
  bool bf16;
  const float* scale;
  Plan plan;
  DevStatus* st;
  cudaStream_t s;
};

// Bytes that every row start of a matrix with rows of C 16-bit elements is a
// multiple of (the base is 16-byte aligned).
int copy_width(int64_t C) { return C % 8 == 0 ? 16 : C % 4 == 0 ? 8 : C % 2 == 0 ? 4 : 2; }

int sm_count() {
  int dev = 0, sms = 152;
  cudaGetDevice(&dev);
  cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  return sms;
}

// CTAs that share one tile: as many as keep the grid within two per SM, each
// with at least two reduction steps.
int split(int64_t tiles, int64_t steps) {
  const int64_t s = std::min<int64_t>({8, 2 * sm_count() / tiles, steps / 2});
  return static_cast<int>(std::max<int64_t>(1, s));
}

// after: it may start before the kernel ahead of it in the stream has ended
// (it waits for that where it first needs anything written before it).
template <typename Args>
cudaError_t launch(void (*kernel)(Args), const Args& a, dim3 grid, int threads, int cluster, int smem, int prof,
                   bool after, cudaStream_t s) {
  if (!ensure_smem_attr(reinterpret_cast<const void*>(kernel), smem)) return cudaGetLastError();
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(static_cast<unsigned>(threads));
  cfg.dynamicSmemBytes = static_cast<size_t>(smem);
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = static_cast<unsigned>(cluster);
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = after ? 1 : 0;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  ProfScope ps(prof, s);
  return cudaLaunchKernelEx(&cfg, kernel, a);
}

constexpr CUtensorMapSwizzle kSwz = CU_TENSOR_MAP_SWIZZLE_128B;
CUtensorMapDataType map_type(const Problem& p) {
  return p.bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
}
// Tensor maps need rows of C and of R elements that start on 16 bytes.
Copy copy_of(const Problem& p, int64_t C) {
  return C % 8 == 0 && p.R % 8 == 0 ? kByTma : C % 2 == 0 && p.R % 2 == 0 ? kByAsync : kByRegisters;
}
template <bool kMN, Copy kCopy>
auto shrink_of(int stages) {
  return stages == 4 ? shrink_kernel<kMN, 4, kCopy> : shrink_kernel<kMN, 3, kCopy>;
}
template <bool kBf16>
auto expand_of(bool mn, Copy copy) {
  return copy == kByTma     ? (mn ? expand_kernel<true, kByTma, kBf16> : expand_kernel<false, kByTma, kBf16>)
         : copy == kByAsync ? (mn ? expand_kernel<true, kByAsync, kBf16> : expand_kernel<false, kByAsync, kBf16>)
         : mn               ? expand_kernel<true, kByRegisters, kBf16>
                            : expand_kernel<false, kByRegisters, kBf16>;
}
template <Copy kCopy>
auto grad_of(int stages) {
  return stages == 3 ? grad_kernel<3, kCopy> : grad_kernel<2, kCopy>;
}

cudaError_t shrink(const Problem& p, const void* X, int64_t C, const void* W, bool mn, const float* scale,
                   void* mid) {
  ShrinkArgs a;
  a.X = static_cast<const uint16_t*>(X);
  a.W = static_cast<const uint16_t*>(W);
  a.mid = static_cast<uint16_t*>(mid);
  a.plane = p.M * p.R;
  a.scale = scale;
  a.tiles = p.plan.tiles;
  a.perm = p.plan.perm;
  a.st = p.st;
  a.C = C;
  a.R = p.R;
  a.E = static_cast<int>(p.E);
  a.cw = copy_width(C);
  a.rw = copy_width(p.R);
  a.bf16 = p.bf16;
  const int r16 = rank16(p.R), ranks = split(p.plan.slots, ceil_div(C, 64));
  a.ranks = ranks;
  const int stages = r16 > 64 ? 3 : 4;
  const int smem = 1024 + std::max(stages * shrink_stage_bytes(r16, mn), 128 * red_pitch(r16) * 4);
  const dim3 grid(static_cast<unsigned>(ranks * p.plan.slots));
  const Copy copy = copy_of(p, C);
  if (copy == kByTma && (!make_tmap(&a.tmX, map_type(p), X, C, p.M, C * 2, 64, 128, kSwz) ||
              !(mn ? make_tmap_3d(&a.tmW, map_type(p), W, p.R, C, p.E, 2, 64, 64, kSwz)
                   : make_tmap_3d(&a.tmW, map_type(p), W, C, p.R, p.E, 2, 64, r16, kSwz))))
    return cudaErrorUnknown;
  auto kernel = copy == kByTma     ? (mn ? shrink_of<true, kByTma>(stages) : shrink_of<false, kByTma>(stages))
                : copy == kByAsync ? (mn ? shrink_of<true, kByAsync>(stages) : shrink_of<false, kByAsync>(stages))
                : mn               ? shrink_of<true, kByRegisters>(stages)
                                   : shrink_of<false, kByRegisters>(stages);
  return launch(kernel, a, grid, kThreads, ranks, smem, K_ADAPTERS, true, p.s);
}

cudaError_t expand(const Problem& p, const void* mid, const void* W, int64_t C, bool mn, const float* scale,
                   const void* addend, void* out) {
  ExpandArgs a;
  a.mid = static_cast<const uint16_t*>(mid);
  a.W = static_cast<const uint16_t*>(W);
  a.addend = static_cast<const uint16_t*>(addend);
  a.out = static_cast<uint16_t*>(out);
  a.scale = scale;
  a.tiles = p.plan.tiles;
  a.perm = p.plan.perm;
  a.st = p.st;
  a.C = C;
  a.M = static_cast<int>(p.M);
  a.R = p.R;
  a.E = static_cast<int>(p.E);
  a.cw = copy_width(C);
  a.rw = copy_width(p.R);
  a.mw = std::min(a.rw, copy_width(p.M * p.R));
  const int r16 = rank16(p.R);
  const int64_t col_tiles = ceil_div(C, kCols);
  // whole waves of the CTAs that fit at once, of at most 12 tiles each; about
  // half of the groups' last slots are taken to be empty
  const int64_t work = std::min<int64_t>(p.plan.slots, ceil_div(p.M, kTile) + (p.E + 1) / 2) * col_tiles;
  const int64_t ctas = expand_per_sm(r16) * sm_count();
  const int64_t waves = ceil_div(work, ctas * 12);
  a.col_tiles = static_cast<int>(ceil_div(work, ctas * waves));
  const int smem = expand_smem(r16);
  const dim3 grid(static_cast<unsigned>(p.plan.slots), static_cast<unsigned>(ceil_div(col_tiles, a.col_tiles)));
  const Copy copy = copy_of(p, C);
  if (copy == kByTma && (!make_tmap(&a.tmMid, map_type(p), mid, p.R, 2 * p.M, p.R * 2, 64, 128, kSwz) ||
              !make_tmap(&a.tmAdd, map_type(p), addend != nullptr ? addend : out, C, p.M, C * 2, 64, 128, kSwz) ||
              !make_tmap(&a.tmOut, map_type(p), out, C, p.M, C * 2, 64, 128, kSwz) ||
              !(mn ? make_tmap_3d(&a.tmW, map_type(p), W, C, p.R, p.E, 2, 64, r16, kSwz)
                   : make_tmap_3d(&a.tmW, map_type(p), W, p.R, C, p.E, 2, 64, 64, kSwz))))
    return cudaErrorUnknown;
  auto kernel = p.bf16 ? expand_of<true>(mn, copy) : expand_of<false>(mn, copy);
  return launch(kernel, a, grid, kExpandThreads, 1, smem, K_ADAPTERS, true, p.s);
}

// One side of the gradients; count 0 when it is not wanted.
bool grad_side(const Problem& p, const void* mid, const void* X, int64_t C, bool rank_major, const float* scale,
               void* out, bool wait, bool tma, GradSide* d) {
  d->tiles = 0;
  d->strips = 1;
  if (out == nullptr) return true;
  d->mid = static_cast<const uint16_t*>(mid);
  d->X = static_cast<const uint16_t*>(X);
  d->grad = static_cast<uint16_t*>(out);
  d->scale = scale;
  d->C = C;
  d->strips = static_cast<int>(ceil_div(C, 128));
  d->tiles = p.E * d->strips;
  d->cw = copy_width(C);
  d->rank_major = rank_major;
  d->wait = wait;
  return !tma || (make_tmap(&d->tmX, map_type(p), X, C, p.M, C * 2, 64, 64, kSwz) &&
                  make_tmap(&d->tmU, map_type(p), mid, p.R, 2 * p.M, p.R * 2, 64, 64, kSwz) &&
                  make_tmap(&d->tmX1, map_type(p), X, C, p.M, C * 2, 64, 1, kSwz));
}

// Both gradients in one launch: gB needs nothing of this call, gA the u of the
// kernel before (after).
cudaError_t grads(const Problem& p, const void* g, const void* t, void* gB, const void* x, const void* u, void* gA,
                  bool after) {
  GradArgs a;
  a.rw = copy_width(p.R);
  a.mw = std::min(copy_width(p.R), copy_width(p.M * p.R));
  const Copy copy = std::max(copy_of(p, gB != nullptr ? p.N : 8), copy_of(p, gA != nullptr ? p.K : 8));
  const bool tma = copy == kByTma;
  if (!grad_side(p, t, g, p.N, false, p.scale, gB, false, tma, &a.side[0]) ||
      !grad_side(p, u, x, p.K, true, nullptr, gA, true, tma, &a.side[1]))
    return cudaErrorUnknown;
  a.offset = p.plan.offset;
  a.perm = p.plan.perm;
  a.st = p.st;
  a.M = static_cast<int>(p.M);
  a.R = p.R;
  a.bf16 = p.bf16;
  a.first = !after;
  const int r16 = rank16(p.R);
  const int64_t tiles = a.side[0].tiles + a.side[1].tiles;
  a.ranks = split(tiles, ceil_div(ceil_div(p.M, p.E), 64));
  if (tiles > INT32_MAX / a.ranks) return cudaErrorInvalidValue;
  const int stages = r16 > 64 ? 2 : 3;
  if (tma && a.ranks == 1) {
    const dim3 grid(static_cast<unsigned>(std::min<int64_t>(tiles, 2 * sm_count())));
    return launch(stages == 3 ? grad_many_kernel<3> : grad_many_kernel<2>, a, grid, kManyThreads, 1,
                  1024 + stages * grad_stage_bytes(r16), K_ADAPTERS_GRAD, after, p.s);
  }
  const int smem = 1024 + std::max(stages * grad_stage_bytes(r16), 128 * red_pitch(r16) * 4);
  const dim3 grid(static_cast<unsigned>(tiles * a.ranks));
  auto kernel = tma                ? grad_of<kByTma>(stages)
                : copy == kByAsync ? grad_of<kByAsync>(stages)
                                   : grad_of<kByRegisters>(stages);
  return launch(kernel, a, grid, kThreads, a.ranks, smem, K_ADAPTERS_GRAD, after, p.s);
}

cudaError_t forward(const Problem& p, const void* x, const void* A, const void* B, const void* base, void* y,
                    void* t) {
  if (p.plan.few_slots > 0 && p.K % 8 == 0 && p.N % 8 == 0 && p.R % 8 == 0) {
    const FewArgs a{static_cast<const uint16_t*>(x), static_cast<const uint16_t*>(A),
                    static_cast<const uint16_t*>(B), static_cast<const uint16_t*>(base),
                    static_cast<uint16_t*>(y), static_cast<uint16_t*>(t), p.M * p.R, p.scale, p.plan.few, p.plan.perm,
                    p.st, p.K, p.N, p.R, static_cast<int>(p.E)};
    const dim3 grid(static_cast<unsigned>(p.plan.few_slots * kFewRanks));
    auto kernel = p.R <= 16   ? (p.bf16 ? few_kernel<true, 1> : few_kernel<false, 1>)
                  : p.R <= 64 ? (p.bf16 ? few_kernel<true, 4> : few_kernel<false, 4>)
                              : (p.bf16 ? few_kernel<true, 8> : few_kernel<false, 8>);
    return launch(kernel, a, grid, kThreads, kFewRanks, 0, K_ADAPTERS, true, p.s);
  }
  if (cudaError_t e = shrink(p, x, p.K, A, false, nullptr, t)) return e;
  return expand(p, t, B, p.N, false, p.scale, base, y);
}

cudaError_t backward(const Problem& p, const void* g, const void* x, const void* t, const void* A, const void* B,
                     const void* addend, void* gx, void* gA, void* gB, void* u) {
  const bool need_u = gx != nullptr || gA != nullptr;
  if (need_u) {
    if (cudaError_t e = shrink(p, g, p.N, B, true, p.scale, u)) return e;
  }
  // right after the pass over g, of which a part is still in L2
  if (gA != nullptr || gB != nullptr) {
    if (cudaError_t e = grads(p, g, t, gB, x, u, gA, need_u)) return e;
  }
  return gx != nullptr ? expand(p, u, A, p.K, true, nullptr, addend, gx) : cudaSuccess;
}

constexpr int64_t kMaxRank = 128, kMaxAdapters = 65535;

bool valid_sizes(int64_t M, int64_t K, int64_t N, int64_t E, int64_t r) {
  return M >= 0 && K > 0 && N > 0 && E > 0 && r > 0 && r <= kMaxRank && E <= kMaxAdapters && M <= INT32_MAX / 2 &&
         K <= (1 << 22) && N <= (1 << 22);
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
  if (p.few_slots > 0 || M == 0)
    adapter_plan_few_kernel<<<1, kFewTokens, 0, s>>>(index, static_cast<int>(M), static_cast<int>(E), p.offset, p.perm,
                                                     p.tiles, p.few, static_cast<int>(p.few_slots));
  else
    adapter_plan_kernel<<<static_cast<unsigned>(E + 1), kPlanThreads, 0, s>>>(
        index, static_cast<int>(M), static_cast<int>(E), p.offset, p.perm, p.tiles);
  return cuda_status(cudaGetLastError());
}

size_t i8lt_adapters_workspace_size(int64_t M, int64_t K, int64_t N, int64_t E, int64_t r) {
  if (!valid_sizes(M, K, N, E, r)) return 0;
  return 256 + static_cast<size_t>(round_up(M * r * 4, 256));
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
  if (M > 0 && y == x) return I8LT_ERR_INVALID_ARG;   // a tile's y is written while others read x
  if (int d = check_device()) return d;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (M == 0) return cuda_status(cudaMemsetAsync(ws, 0, sizeof(DevStatus), s));
  const Problem p{M, K, N, E, static_cast<int>(r), dt == DT_BF16, scale, plan_layout(const_cast<void*>(plan), M, E),
                  static_cast<DevStatus*>(ws), s};
  return cuda_status(forward(p, x, A, B, base, y, t));
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
  if (M > 0 && gx != nullptr && (gx == g || gx == x)) return I8LT_ERR_INVALID_ARG;   // likewise
  if (int d = check_device()) return d;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (M == 0) {   // no tokens: the weight gradients are zeros
    if (cudaMemsetAsync(ws, 0, sizeof(DevStatus), s) != cudaSuccess) return I8LT_ERR_CUDA;
    if (gA != nullptr && cudaMemsetAsync(gA, 0, static_cast<size_t>(E * r * K) * 2, s) != cudaSuccess)
      return I8LT_ERR_CUDA;
    if (gB != nullptr && cudaMemsetAsync(gB, 0, static_cast<size_t>(E * r * N) * 2, s) != cudaSuccess)
      return I8LT_ERR_CUDA;
    return I8LT_OK;
  }
  const Problem p{M, K, N, E, static_cast<int>(r), dt == DT_BF16, scale, plan_layout(const_cast<void*>(plan), M, E),
                  static_cast<DevStatus*>(ws), s};
  void* u = static_cast<uint8_t*>(ws) + 256;
  return cuda_status(backward(p, g, x, t, A, B, addend, gx, gA, gB, u));
}

}  // extern "C"
