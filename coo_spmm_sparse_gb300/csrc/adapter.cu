// Low-rank adapters of many requests beside one projection:
//
//   H[t] = A_n X[t],  Y[t] += s_n B_n H[t]        n: the adapter of token t's request
//   dH[t] = s_n B_n^T dY[t],  dX[t] += A_n^T dH[t],
//   dA_n = sum_t dH[t] X[t]^T,  dB_n = s_n sum_t dY[t] H[t]^T
//
// Memory bound for ranks up to about 32: every element of X, Y, dY and dX
// takes 2 * rank multiply-adds.  Few tokens (decoding): a cluster of blocks
// for each token, the weights are the work.  Many tokens: they are first
// grouped by adapter (`plan`), so that requests that share one fill tiles
// together, and each product then runs over tiles of 32 tokens on the matrix
// instructions:
//
//   down   [tokens x K] x [K x rank]   K split over the block's warps, one sum through shared memory
//   up     [tokens x rank] x [rank x K], added to the rows in place
//   outer  [rank x tokens] x [tokens x K], tokens split over blocks, parts added in order
//
// The order in which the summed index is fed to a matrix instruction is free
// as long as both operands keep it, so a lane takes 16 contiguous bytes of a
// row as they lie in memory, and rows may be any tokens.  Rows come by
// asynchronous copies into a ring of shared memory that belongs to one warp:
// registers that can wait for memory, and no barrier of the block.  (Loads
// into registers left one block's 64 bytes a lane in flight: 47 us for `down`
// and 80 us for `outer` over 134 MB; now 31 and 32 us.)
//
// fp32 operands are split into two tf32 parts, x = hi + lo, and hi*hi + hi*lo
// + lo*hi is summed: what is left out is below 2^-22 of a product.  Their
// running sums leave the matrix unit's accumulator every 32 (outer) or 64
// (down; up above 64 ranks) summed elements for a 32-bit sum that rounds to
// nearest (kept in it over 300 tokens, dA was 2.4e-6 off in the 2-norm; so
// 6.6e-7).
//
// H and dH are fp32 in memory.  In 16-bit products they are two parts of the
// type, hi + lo: 16 bits of them in bf16 (off by 2^-17), 22 in fp16, beside
// the 8 and 11 bits to which the results are rounded.  Few tokens take them
// as they are.
//
// 8192 tokens, 4096 -> 4096, 4 adapters of rank 16, fp32: forward and backward
// 240 us, 160 us of which is the traffic at 6.7 TB/s.
#include <cooperative_groups.h>

#include <algorithm>
#include <type_traits>

#include "dense_ops.cuh"

namespace snack {
namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kTile = 32;            // tokens of a tile
constexpr int kPlanThreads = 1024;
constexpr int kRankPass = 64;        // ranks that one pass of `down` sums

// Ranks that one pass of `outer` sums.
__host__ __device__ constexpr int outer_ranks(int64_t rank) { return rank <= 16 ? 16 : 32; }

// Whether running sums leave the matrix unit now and then: 16-bit results
// (rounded to 2^-8 or 2^-11) do not show what its accumulator cuts off over some
// hundred steps (1e-6), and the second set of sums costs registers that the
// 32-rank products do not have.
template <typename T>
constexpr bool kFlush = sizeof(T) == 4;

// Tokens grouped by adapter.
struct Plan {
  int32_t *head;   // [0] tiles, [1] used adapters, [2] tokens with an adapter
  int32_t *perm;   // [tokens] token at each place
  int4 *tiles;     // {adapter, first place, tokens, index among the used}
  int4 *used;      // {adapter, first place, tokens, 0}
  int32_t *index;  // [adapters] index among the used, or -1
  int32_t *soff, *place, *base;  // many requests: offsets kept in order, first places, running places
  int64_t max_tiles, max_used;
};

struct AdapterArgs {
  snack_adapter_args a;
  Plan p;
  float *H;  // [tokens][rank], zeroed by the plan where a token has no adapter (or null)
};

__device__ __forceinline__ float scale_of(const snack_adapter_args &a, int n) {
  return a.scale ? a.scale[n] : a.uniform_scale;
}

// ------------------------------------------------------------------ plan

__device__ __forceinline__ int32_t clamp_offset(int32_t v, int64_t tokens) {
  return v < 0 ? 0 : (v > tokens ? (int32_t)tokens : v);
}

// Inclusive maximum over the block's values, `carry` included; `red` holds 32 ints.
__device__ __forceinline__ int32_t block_scan_max(int32_t v, int32_t carry, int32_t *red) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int32_t u = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v = max(v, u);
  }
  if (lane == 31) red[w] = v;
  __syncthreads();
  if (w == 0) {
    int32_t s = lane < (int)blockDim.x / 32 ? red[lane] : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int32_t u = __shfl_up_sync(0xffffffffu, s, o);
      if (lane >= o) s = max(s, u);
    }
    red[lane] = s;
  }
  __syncthreads();
  if (w > 0) v = max(v, red[w - 1]);
  v = max(v, carry);
  __syncthreads();
  return v;
}

// The request of token t by the ordered offsets (o[0..n]): the last that
// begins at or before t, or -1.
__device__ __forceinline__ int request_of(const int32_t *o, int n, int32_t t) {
  int lo = 0, hi = n;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (o[mid] <= t)
      lo = mid + 1;
    else
      hi = mid;
  }
  return lo == 0 || t >= o[lo] ? -1 : lo - 1;
}

__device__ __forceinline__ void zero_row(const AdapterArgs &q, int64_t t) {
  if (q.H)
    for (int64_t j = 0; j < q.a.rank; ++j) q.H[t * q.a.rank + j] = 0.f;
}

// Up to 1024 requests: every block works all of them out in shared memory
// (each request compares itself with all others) and places its own share
// of the tokens; block 0 writes the tables.
template <int TH>
__global__ void __launch_bounds__(TH) plan_small(const __grid_constant__ AdapterArgs q) {
  __shared__ int32_t off[TH + 1], place[TH], red[32];
  __shared__ int2 request[TH], leader_of[TH];  // {adapter or -1, tokens}; {adapter, tiles} of the first of each adapter
  dependency_wait();
  dependency_launch();
  const snack_adapter_args &a = q.a;
  const int R = (int)a.requests, r = threadIdx.x;
  {
    const int32_t v = r < R ? clamp_offset(a.offsets[r], a.tokens) : 0;
    const int32_t m = block_scan_max(v, 0, red);
    if (r < R) off[r] = m;
    if (r == R - 1) off[R] = max(m, clamp_offset(a.offsets[R], a.tokens));
  }
  __syncthreads();
  int n = -1;
  if (r < R) {
    const int len = off[r + 1] - off[r];
    n = a.adapter[r];
    if (n < 0 || n >= a.adapters || len == 0) n = -1;
    request[r] = make_int2(n, n < 0 ? 0 : len);
  }
  __syncthreads();
  int first = 0, total = 0, all = 0;
  bool leader = n >= 0;
  if (r < R) {
#pragma unroll 8
    for (int j = 0; j < R; ++j) {
      const int2 o = request[j];  // no tokens where it names no adapter
      all += o.y;
      first += o.x < n || (o.x == n && j < r) ? o.y : 0;
      total += o.x == n ? o.y : 0;
      leader = leader && !(o.x == n && j < r);
    }
    place[r] = first;
    leader_of[r] = make_int2(n, leader ? (total + kTile - 1) / kTile : 0);
  }
  if (blockIdx.x == 0) {
    for (int64_t i = r; i < a.adapters; i += TH) q.p.index[i] = -1;
    __syncthreads();
    int t0 = 0, u = 0, tn = 0, un = 0;
    if (r < R) {
#pragma unroll 8
      for (int j = 0; j < R; ++j) {
        const int2 o = leader_of[j];
        tn += o.y;
        un += o.y > 0;
        t0 += o.x < n ? o.y : 0;
        u += o.x < n && o.y > 0;
      }
    }
    if (r < R && leader) {
      q.p.index[n] = u;
      q.p.used[u] = make_int4(n, first, total, 0);
      for (int k = 0; k * kTile < total; ++k)
        q.p.tiles[t0 + k] = make_int4(n, first + k * kTile, min(kTile, total - k * kTile), u);
    }
    if (r == 0) {
      q.p.head[0] = tn;
      q.p.head[1] = un;
      q.p.head[2] = all;
    }
  }
  __syncthreads();
  for (int64_t t = (int64_t)blockIdx.x * TH + r; t < a.tokens; t += (int64_t)gridDim.x * TH) {
    const int i = request_of(off, R, (int32_t)t);
    if (i >= 0 && request[i].x >= 0)
      q.p.perm[place[i] + ((int32_t)t - off[i])] = (int32_t)t;
    else
      zero_row(q, t);
  }
}

// Any number of requests: one block counts the tokens of every adapter,
// places adapters and then requests, 1024 at a time.
__global__ void __launch_bounds__(kPlanThreads) plan_requests(const __grid_constant__ AdapterArgs q) {
  __shared__ int32_t key[kPlanThreads], len[kPlanThreads], red[32], carry[3];
  dependency_wait();
  dependency_launch();
  const snack_adapter_args &a = q.a;
  const Plan &p = q.p;
  const int tid = threadIdx.x;
  for (int64_t i = tid; i < a.adapters; i += kPlanThreads) p.base[i] = 0;
  int32_t top = 0;
  for (int64_t c = 0; c <= a.requests; c += kPlanThreads) {
    const int64_t i = c + tid;
    const int32_t v = i <= a.requests ? clamp_offset(a.offsets[i], a.tokens) : 0;
    const int32_t m = block_scan_max(v, top, red);
    if (i <= a.requests) p.soff[i] = m;
    if (tid == kPlanThreads - 1) carry[0] = m;
    __syncthreads();
    top = carry[0];
    __syncthreads();
  }
  for (int64_t i = tid; i < a.requests; i += kPlanThreads) {
    const int n = a.adapter[i], l = p.soff[i + 1] - p.soff[i];
    if (n >= 0 && n < a.adapters && l > 0) atomicAdd(&p.base[n], l);
  }
  if (tid < 3) carry[tid] = 0;
  __syncthreads();
  // exclusive sums over the adapters of tokens, used ones and tiles
  for (int64_t c = 0; c < a.adapters; c += kPlanThreads) {
    const int64_t n = c + tid;
    const int32_t total = n < a.adapters ? p.base[n] : 0;
    int32_t sum[3] = {total, total > 0, (total + kTile - 1) / kTile}, mine[3];
#pragma unroll
    for (int k = 0; k < 3; ++k) {
      const int lane = tid & 31, w = tid >> 5;
      int32_t v = sum[k];
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int32_t u = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += u;
      }
      if (lane == 31) red[w] = v;
      __syncthreads();
      if (w == 0) {
        int32_t s = red[lane];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int32_t u = __shfl_up_sync(0xffffffffu, s, o);
          if (lane >= o) s += u;
        }
        red[lane] = s;
      }
      __syncthreads();
      v += (w > 0 ? red[w - 1] : 0) + carry[k];
      mine[k] = v - sum[k];
      __syncthreads();
      if (tid == kPlanThreads - 1) carry[k] = v;
      __syncthreads();
    }
    if (n < a.adapters) {
      p.base[n] = mine[0];
      p.index[n] = total > 0 ? mine[1] : -1;
      if (total > 0) {
        p.used[mine[1]] = make_int4((int)n, mine[0], total, 0);
        for (int k = 0; k * kTile < total; ++k)
          p.tiles[mine[2] + k] = make_int4((int)n, mine[0] + k * kTile, min(kTile, total - k * kTile), mine[1]);
      }
    }
  }
  __syncthreads();
  if (tid == 0) {
    p.head[0] = carry[2];
    p.head[1] = carry[1];
    p.head[2] = carry[0];
  }
  for (int64_t c = 0; c < a.requests; c += kPlanThreads) {
    const int64_t i = c + tid;
    int n = -1, l = 0;
    if (i < a.requests) {
      n = a.adapter[i];
      l = p.soff[i + 1] - p.soff[i];
      if (n < 0 || n >= a.adapters || l == 0) n = -1;
    }
    key[tid] = n;
    len[tid] = l;
    __syncthreads();
    int before = 0;
    if (n >= 0)
      for (int j = 0; j < tid; ++j) before += key[j] == n ? len[j] : 0;
    if (i < a.requests) p.place[i] = n >= 0 ? p.base[n] + before : -1;
    __syncthreads();
    if (n >= 0) atomicAdd(&p.base[n], l);
    __syncthreads();
  }
}

__global__ void __launch_bounds__(kThreads) plan_tokens(const __grid_constant__ AdapterArgs q) {
  dependency_wait();
  dependency_launch();
  const snack_adapter_args &a = q.a;
  for (int64_t t = (int64_t)blockIdx.x * kThreads + threadIdx.x; t < a.tokens; t += (int64_t)gridDim.x * kThreads) {
    const int i = request_of(q.p.soff, (int)a.requests, (int32_t)t);
    if (i >= 0 && q.p.place[i] >= 0)
      q.p.perm[q.p.place[i] + ((int32_t)t - q.p.soff[i])] = (int32_t)t;
    else
      zero_row(q, t);
  }
}

// ------------------------------------------------------------------ matrix instructions

// x rounded to the 11 significant bits of tf32, halves away from zero (a
// magnitude above 2^128 - 2^116 overflows; what x - hi then is, is not a number).
__device__ __forceinline__ float tf32_of(float x) {
  return __uint_as_float((__float_as_uint(x) + 0x1000u) & 0xffffe000u);
}

__device__ __forceinline__ void mma_tf32(float (&c)[4], float a0, float a1, float a2, float a3, float b0, float b1) {
  asm("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(__float_as_uint(a0)), "r"(__float_as_uint(a1)), "r"(__float_as_uint(a2)), "r"(__float_as_uint(a3)),
        "r"(__float_as_uint(b0)), "r"(__float_as_uint(b1)));
}

template <typename T>
__device__ __forceinline__ void mma_16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                       uint32_t b0, uint32_t b1);
template <>
__device__ __forceinline__ void mma_16<__nv_bfloat16>(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                                      uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
template <>
__device__ __forceinline__ void mma_16<__half>(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                               uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The power of two that brings the largest finite magnitude of some 32-bit
// floats (its bits) to [2^14, 2^15): float16 holds neither more than 65504 nor
// the small values of a gradient to more than 2^-25, which two parts of it,
// scaled so, do to 2^-22 of any value down to 2^-16 of the largest.
__device__ __forceinline__ float half_scale(uint32_t largest) {
  const int e = (int)(largest >> 23) - 127;  // -127: zeros and subnormals
  const int up = min(max(14 - e, -126), 126);
  return __uint_as_float((uint32_t)(up + 127) << 23);
}
__device__ __forceinline__ uint32_t finite_bits(float v) {
  const uint32_t b = __float_as_uint(v) & 0x7fffffffu;
  return b < 0x7f800000u ? b : 0u;
}

// Two values as one register of T pairs, and what that rounding left out as another.
template <typename T>
__device__ __forceinline__ void split_pair(float x, float y, uint32_t &hi, uint32_t &lo) {
  alignas(4) T h[2] = {from_float<T>(x), from_float<T>(y)};
  alignas(4) T l[2] = {from_float<T>(x - to_float(h[0])), from_float<T>(y - to_float(h[1]))};
  hi = *reinterpret_cast<const uint32_t *>(h);
  lo = *reinterpret_cast<const uint32_t *>(l);
}

// 16 bytes of a row from element k on; elements from `limit` on read as 0.
template <typename T, bool ALIGNED>
__device__ __forceinline__ uint4 load16(const T *row, int64_t k, int64_t limit, bool valid) {
  constexpr int E = 16 / sizeof(T);
  uint4 v = make_uint4(0, 0, 0, 0);
  if (ALIGNED) {
    if (valid && k < limit) v = *reinterpret_cast<const uint4 *>(row + k);
  } else if (valid) {
    T *e = reinterpret_cast<T *>(&v);
#pragma unroll
    for (int i = 0; i < E; ++i)
      if (k + i < limit) e[i] = row[k + i];
  }
  return v;
}

// The same copied asynchronously into a slot of shared memory (16-byte
// aligned rows); what is not there arrives as 0.
template <typename T>
__device__ __forceinline__ void copy16(uint4 *slot, const T *row, int64_t k, int64_t limit, bool valid) {
  const bool in = valid && k < limit;
  const T *from = in ? row + k : row;
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"((uint32_t)__cvta_generic_to_shared(slot)),
               "l"(from), "r"(in ? 16 : 0)
               : "memory");
}
template <typename T>
__device__ __forceinline__ void copy8(uint2 *slot, const T *row, int64_t k, int64_t limit, bool valid) {
  const bool in = valid && k < limit;
  const T *from = in ? row + k : row;
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"((uint32_t)__cvta_generic_to_shared(slot)),
               "l"(from), "r"(in ? 8 : 0)
               : "memory");
}
// One group of the summed index (64 bytes of a row: 16 fp32 or 32 16-bit
// elements) of a 16 x 8 product: rows g and g + 8 in v0 and v1, the other
// operand's row g in w.
template <typename T>
struct Group {
  static constexpr int E = 16 / sizeof(T);
  static constexpr int K = 4 * E;
};

__device__ __forceinline__ void split4(const uint4 &v, float (&hi)[4], float (&lo)[4]) {
  const float x[4] = {__uint_as_float(v.x), __uint_as_float(v.y), __uint_as_float(v.z), __uint_as_float(v.w)};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    hi[i] = tf32_of(x[i]);
    lo[i] = x[i] - hi[i];
  }
}

// ------------------------------------------------------------------ down: H = X W^T

struct DownArgs {
  const void *X;      // rows of K elements, x_stride apart
  const void *W;      // [adapter or used index][rank][K]
  int64_t x_stride, K, rank;
  bool by_used;       // W is indexed by the tile's index among the used adapters
  bool scaled;        // times the adapter's scale
  float *H;           // [tokens][rank]
};

// A warp's step: two groups of K, 128 bytes of each row of X and W.
template <int NT>
struct DownShape {
  static constexpr int ROWS = kTile + NT * 8;
  static constexpr int STAGES = 2;  // 80 to 192 KB a block: two blocks an SM up to 16 ranks, one above
  static constexpr int LD = NT * 8 + 4;
  static constexpr size_t RING = (size_t)kWarps * STAGES * ROWS * 128;
  static constexpr size_t PART = sizeof(float) * kWarps * kTile * LD;
  static constexpr size_t SMEM = RING > PART ? RING : PART;
};

// Block, or a cluster of blocks where there are few tiles: one tile of kTile
// tokens, ranks [64 y, 64 y + 64).  The warps take steps of K in turn and
// meet in shared memory at the end, a cluster's blocks in each other's.
// (One block for each of 8 tiles of 4096 columns: 16 steps for every warp,
// each of which waits for memory.)  Eight lanes copy
// the 128 bytes of a row; chunk c of a row lies at c ^ 4 (row & 1), where the
// eight lanes that read together find two rows' halves in eight bank groups.
template <typename T, int NT, bool ALIGNED>
__global__ void __launch_bounds__(kThreads, NT <= 4 ? 2 : 1) adapter_down(const __grid_constant__ AdapterArgs q,
                                                                         const __grid_constant__ DownArgs d) {
  using S = DownShape<NT>;
  constexpr int MT = kTile / 16, E = Group<T>::E, KG = Group<T>::K;
  constexpr int kCols = NT * 8, STAGES = S::STAGES;
  extern __shared__ uint4 smem4[];
  float *part = reinterpret_cast<float *>(smem4);  // [kWarps][kTile][LD], over the ring
  dependency_wait();
  dependency_launch();
  cg::cluster_group cluster = cg::this_cluster();
  const int blocks = (int)cluster.num_blocks(), rank_of = (int)cluster.block_rank();
  const int which = (int)blockIdx.x / blocks;
  if (which >= q.p.head[0]) return;  // the whole cluster
  const int4 tile = q.p.tiles[which];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
  const int worker = rank_of * kWarps + warp, workers = blocks * kWarps;
  const int64_t j0 = (int64_t)blockIdx.y * kRankPass;
  const T *X = static_cast<const T *>(d.X);
  const T *W = static_cast<const T *>(d.W) + ((int64_t)(d.by_used ? tile.w : tile.x) * d.rank + j0) * d.K;
  const int ranks = (int)min((int64_t)kRankPass, d.rank - j0);
  // token of tile row `lane`, or -1
  const int mine = lane < tile.z ? q.p.perm[tile.y + lane] : -1;

  const int steps = ((int)((d.K + 2 * KG - 1) / (2 * KG)) - worker + workers - 1) / workers;  // of this warp
  uint4 *ring = smem4 + (int64_t)warp * STAGES * S::ROWS * 8;
  const auto fetch = [&](int i) {
    if (ALIGNED && i < steps) {
      const int64_t k = ((int64_t)i * workers + worker) * 2 * KG + (lane & 7) * E;
      uint4 *slot = ring + (i % STAGES) * S::ROWS * 8;
      const int r = lane >> 3, at = r * 8 + ((lane & 7) ^ (4 * (r & 1)));
#pragma unroll
      for (int m = 0; m < kTile / 4; ++m) {
        const int tok = __shfl_sync(0xffffffffu, mine, 4 * m + r);
        copy16(slot + m * 32 + at, X + (int64_t)max(tok, 0) * d.x_stride, k, d.K, tok >= 0);
      }
#pragma unroll
      for (int n = 0; n < NT * 2; ++n) {
        const int j = 4 * n + r;
        copy16(slot + (kTile / 4 + n) * 32 + at, W + (int64_t)(j < ranks ? j : 0) * d.K, k, d.K, j < ranks);
      }
    }
    if (ALIGNED) copies_commit();
  };
  float sum[MT][NT][4], fresh[MT][NT][4];
  auto &acc = kFlush<T> ? fresh : sum;
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) sum[m][n][i] = acc[m][n][i] = 0.f;
  const auto flush = [&] {
    if constexpr (kFlush<T>) {
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            sum[m][n][i] += acc[m][n][i];
            acc[m][n][i] = 0.f;
          }
    }
  };

#pragma unroll
  for (int i = 0; i < STAGES - 1; ++i) fetch(i);
  for (int i = 0; i < steps; ++i) {
    if (ALIGNED) {
      copies_wait<STAGES - 2>();
      __syncwarp();
      fetch(i + STAGES - 1);  // into the slots that every lane read before this barrier
    }
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      uint4 x[2 * MT], w[NT];
      if (ALIGNED) {
        const uint4 *slot = ring + (i % STAGES) * S::ROWS * 8 + g * 8 + ((4 * half + t) ^ (4 * (g & 1)));
#pragma unroll
        for (int m = 0; m < 2 * MT; ++m) x[m] = slot[m * 64];
#pragma unroll
        for (int n = 0; n < NT; ++n) w[n] = slot[(2 * MT + n) * 64];
      } else {
        const int64_t k = (((int64_t)i * workers + worker) * 2 + half) * KG + t * E;
#pragma unroll
        for (int m = 0; m < 2 * MT; ++m) {
          const int tok = __shfl_sync(0xffffffffu, mine, m * 8 + g);
          x[m] = load16<T, false>(X + (int64_t)max(tok, 0) * d.x_stride, k, d.K, tok >= 0);
        }
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          const int j = n * 8 + g;
          w[n] = load16<T, false>(W + (int64_t)(j < ranks ? j : 0) * d.K, k, d.K, j < ranks);
        }
      }
      if constexpr (sizeof(T) == 4) {
        float xh[2 * MT][4], xl[2 * MT][4];
#pragma unroll
        for (int m = 0; m < 2 * MT; ++m) split4(x[m], xh[m], xl[m]);
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          float wh[4], wl[4];
          split4(w[n], wh, wl);
#pragma unroll
          for (int s = 0; s < 4; s += 2)
#pragma unroll
            for (int m = 0; m < MT; ++m) {
              mma_tf32(acc[m][n], xl[2 * m][s], xl[2 * m + 1][s], xl[2 * m][s + 1], xl[2 * m + 1][s + 1], wh[s], wh[s + 1]);
              mma_tf32(acc[m][n], xh[2 * m][s], xh[2 * m + 1][s], xh[2 * m][s + 1], xh[2 * m + 1][s + 1], wl[s], wl[s + 1]);
              mma_tf32(acc[m][n], xh[2 * m][s], xh[2 * m + 1][s], xh[2 * m][s + 1], xh[2 * m + 1][s + 1], wh[s], wh[s + 1]);
            }
        }
      } else {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int m = 0; m < MT; ++m) {
            mma_16<T>(acc[m][n], x[2 * m].x, x[2 * m + 1].x, x[2 * m].y, x[2 * m + 1].y, w[n].x, w[n].y);
            mma_16<T>(acc[m][n], x[2 * m].z, x[2 * m + 1].z, x[2 * m].w, x[2 * m + 1].w, w[n].z, w[n].w);
          }
      }
    }
    if (i & 1) flush();
  }
  flush();
  copies_wait<0>();
  __syncthreads();
  constexpr int LD = S::LD;
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      float *at = part + ((int64_t)warp * kTile + m * 16 + g) * LD + n * 8 + 2 * t;
      at[0] = sum[m][n][0];
      at[1] = sum[m][n][1];
      at[8 * LD] = sum[m][n][2];
      at[8 * LD + 1] = sum[m][n][3];
    }
  __syncthreads();
  const float scale = d.scaled ? scale_of(q.a, tile.x) : 1.f;
  const auto block_sum_at = [&](int i, int j) {
    float s = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) s += part[((int64_t)w * kTile + i) * LD + j];
    return s;
  };
  const auto put = [&](int i, int j, float s) {
    if (i < tile.z && j < ranks) d.H[(int64_t)q.p.perm[tile.y + i] * d.rank + j0 + j] = s * scale;
  };
  if (blocks == 1) {
    for (int e = threadIdx.x; e < kTile * kCols; e += kThreads) put(e / kCols, e % kCols, block_sum_at(e / kCols, e % kCols));
    return;
  }
  // each block's sums over its warps' first part, then every block adds its share of all blocks'
  float own[kTile * kCols / kThreads];
#pragma unroll
  for (int k = 0; k < kTile * kCols / kThreads; ++k) {
    const int e = k * kThreads + threadIdx.x;
    own[k] = block_sum_at(e / kCols, e % kCols);
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < kTile * kCols / kThreads; ++k) part[k * kThreads + threadIdx.x] = own[k];
  cluster.sync();
  for (int e = rank_of * kThreads + threadIdx.x; e < kTile * kCols; e += blocks * kThreads) {
    float s = 0.f;
    for (int b = 0; b < blocks; ++b) s += cluster.map_shared_rank(part, b)[e];
    put(e / kCols, e % kCols, s);
  }
  cluster.sync();  // no block leaves while another reads its sums
}

// ------------------------------------------------------------------ up: Y += H W^T

struct UpArgs {
  const float *H;     // [tokens][rank]
  const void *W;      // [adapter or used index][K][rank]
  void *Y;            // rows of K elements, y_stride apart, added to
  int64_t y_stride, K, rank;
  bool by_used, scaled;
};

// Columns that a warp takes at once: 64 bytes of each row.
template <typename T>
struct UpShape {
  static constexpr int E = 16 / sizeof(T);
  static constexpr int NT = E / 2;                          // 8-column products side by side
  static constexpr int COLS = 4 * E;                        // 16 or 32
  static constexpr int BLOCK = kWarps * COLS;               // columns that a block takes at once
  static constexpr int PER = sizeof(T) == 4 ? 2 : 1;        // instructions for 16 ranks
  static constexpr int WBYTES = 4 * sizeof(T);              // four ranks of a weight row
  // bytes of a warp's step: its rows of Y, and the weights of RG times 16 ranks
  __host__ __device__ static constexpr int step_bytes(int rg) { return 2 * (kTile / 16) * 512 + NT * rg * 32 * WBYTES; }
  __host__ __device__ static constexpr int stages(int rg) { return rg == 2 ? 3 : 4; }
  __host__ __device__ static constexpr size_t frag_bytes(int64_t rank) { return (size_t)((rank + 15) / 16) * (kTile / 16) * 2 * PER * 512; }
  __host__ __device__ static constexpr size_t smem(int rg, int64_t rank) {
    return frag_bytes(rank) + (size_t)kWarps * stages(rg) * step_bytes(rg);
  }
};

// Four ranks of a weight row as the B operand of one or two instructions.
template <typename T>
__device__ __forceinline__ void load_ranks(const T *row, int64_t j, int64_t rank, bool vec, bool valid, T (&out)[4]) {
  if (vec) {
    if (sizeof(T) == 4) {
      uint4 v = make_uint4(0, 0, 0, 0);
      if (valid && j < rank) v = *reinterpret_cast<const uint4 *>(row + j);
      *reinterpret_cast<uint4 *>(out) = v;
    } else {
      uint2 v = make_uint2(0, 0);
      if (valid && j < rank) v = *reinterpret_cast<const uint2 *>(row + j);
      *reinterpret_cast<uint2 *>(out) = v;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) out[i] = valid && j + i < rank ? row[j + i] : from_float<T>(0.f);
  }
}

// Every block takes an equal run of the (tile, column block) pairs, tile by
// tile, so that all end together (a block for each tile and a few columns
// left a fifth of the SMs' time idle).  A tile's H is kept in shared memory,
// split in two parts, in the order in which the lanes want it.  RG: 16-rank
// groups (1 or 2, weights copied ahead with the rows; 0: any number, weights
// loaded when they are needed: ahead, 64 ranks measured the same in fp32 and
// 350 us for 330 in bf16, forward and backward; -1: fp32 above 64 ranks, summed
// 64 at a time in the matrix unit: 512 positive terms kept in it came out
// 3.8e-6 off, so 4.1e-7, at 226 us for 213 of a forward of 4096 tokens, 1024
// -> 1024; up to 64 ranks they are 4.6e-7 off as they are).
template <typename T, int RG, bool ALIGNED>
__global__ void __launch_bounds__(kThreads, 2) adapter_up(const __grid_constant__ AdapterArgs q,
                                                          const __grid_constant__ UpArgs d) {
  using S = UpShape<T>;
  constexpr int MT = kTile / 16, E = S::E, NT = S::NT, PER = S::PER, STAGES = S::stages(RG);
  constexpr int STEP = S::step_bytes(RG > 0 ? RG : 0);
  constexpr bool AHEAD = ALIGNED && RG > 0;  // rows and weights both in vectors
  extern __shared__ uint4 frag[];            // [16-rank groups][MT][2 (high and low)][PER][32 lanes], then the rings
  dependency_wait();
  dependency_launch();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
  const int rg = RG > 0 ? RG : (int)((d.rank + 15) / 16);
  // column of product n's index g: the lane that ends up with columns 2t and
  // 2t + 1 of every n holds E columns in a row
  const int gcol = (g >> 1) * E + (g & 1);
  char *ring = reinterpret_cast<char *>(frag) + S::frag_bytes(d.rank) + (size_t)warp * STAGES * STEP;
  const bool wvec = d.rank % 4 == 0 && (reinterpret_cast<uintptr_t>(d.W) & (4 * sizeof(T) - 1)) == 0;
  const int across = (int)((d.K + S::BLOCK - 1) / S::BLOCK);  // column blocks of a tile
  const int64_t all = (int64_t)q.p.head[0] * across;
  const int64_t u1 = all * (blockIdx.x + 1) / gridDim.x;
  __shared__ uint32_t largest;
  int count;  // column blocks of the tile at hand
  for (int64_t u = all * blockIdx.x / gridDim.x; u < u1; u += count) {
    const int4 tile = q.p.tiles[u / across];
    const int c0_block = (int)(u % across);
    count = (int)min((int64_t)(across - c0_block), u1 - u);
    T *rows[2 * MT];
    bool ok[2 * MT];
#pragma unroll
    for (int m = 0; m < 2 * MT; ++m) {
      const int i = m * 8 + g;
      ok[m] = i < tile.z;
      rows[m] = static_cast<T *>(d.Y) + (ok[m] ? (int64_t)q.p.perm[tile.y + i] * d.y_stride : 0);
    }
    const T *W = static_cast<const T *>(d.W) + (int64_t)(d.by_used ? tile.w : tile.x) * d.K * d.rank;
    const auto column = [&](int c) { return ((int64_t)(c0_block + c) * kWarps + warp) * S::COLS; };
    const auto fetch = [&](int c) {
      if (!ALIGNED) return;
      const int64_t c0 = column(c);
      if (c < count && c0 < d.K) {
        char *at = ring + (c % STAGES) * STEP;
#pragma unroll
        for (int m = 0; m < 2 * MT; ++m)
          copy16(reinterpret_cast<uint4 *>(at) + m * 32 + lane, rows[m], c0 + t * E, d.K, ok[m]);
        if (AHEAD) {
          at += 2 * MT * 512;
#pragma unroll
          for (int k = 0; k < RG; ++k)
#pragma unroll
            for (int n = 0; n < NT; ++n) {
              const int64_t col = c0 + gcol + 2 * n;
              const T *row = W + (col < d.K ? col * d.rank : 0);
              char *slot = at + ((k * NT + n) * 32 + lane) * S::WBYTES;
              if constexpr (sizeof(T) == 4)
                copy16(reinterpret_cast<uint4 *>(slot), row, k * 16 + 4 * t, d.rank, col < d.K);
              else
                copy8(reinterpret_cast<uint2 *>(slot), row, k * 16 + 4 * t, d.rank, col < d.K);
            }
        }
      }
      copies_commit();
    };
#pragma unroll
    for (int c = 0; c < STAGES - 1; ++c) fetch(c);

    const float scale = d.scaled ? scale_of(q.a, tile.x) : 1.f;
    const auto h_at = [&](int row, int64_t j) {
      return row < tile.z && j < d.rank ? d.H[(int64_t)q.p.perm[tile.y + row] * d.rank + j] * scale : 0.f;
    };
    float fit = 1.f;  // float16: power of two that the tile's H is scaled by
    if constexpr (std::is_same_v<T, __half>) {
      if (threadIdx.x == 0) largest = 0u;
      __syncthreads();
      uint32_t most = 0u;
      for (int i = threadIdx.x; i < kTile * d.rank; i += kThreads) most = max(most, finite_bits(h_at(i / (int)d.rank, i % d.rank)));
      atomicMax(&largest, most);
      __syncthreads();
      fit = half_scale(largest);
    }
    for (int i = warp; i < rg * MT; i += kWarps) {
      const int m = i % MT, k = i / MT;
      float h[2][4];
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const int row = m * 16 + half * 8 + g;
#pragma unroll
        for (int e = 0; e < 4; ++e) h[half][e] = h_at(row, k * 16 + 4 * t + e) * fit;
      }
      uint4 *to = frag + (int64_t)(k * MT + m) * 2 * PER * 32 + lane;
      if constexpr (sizeof(T) == 4) {
        float hi[2][4], lo[2][4];
#pragma unroll
        for (int half = 0; half < 2; ++half)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            hi[half][e] = tf32_of(h[half][e]);
            lo[half][e] = h[half][e] - hi[half][e];
          }
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          to[(0 * PER + s) * 32] = make_uint4(__float_as_uint(hi[0][2 * s]), __float_as_uint(hi[1][2 * s]),
                                              __float_as_uint(hi[0][2 * s + 1]), __float_as_uint(hi[1][2 * s + 1]));
          to[(1 * PER + s) * 32] = make_uint4(__float_as_uint(lo[0][2 * s]), __float_as_uint(lo[1][2 * s]),
                                              __float_as_uint(lo[0][2 * s + 1]), __float_as_uint(lo[1][2 * s + 1]));
        }
      } else {
        uint4 hi, lo;
        split_pair<T>(h[0][0], h[0][1], hi.x, lo.x);
        split_pair<T>(h[1][0], h[1][1], hi.y, lo.y);
        split_pair<T>(h[0][2], h[0][3], hi.z, lo.z);
        split_pair<T>(h[1][2], h[1][3], hi.w, lo.w);
        to[0] = hi;
        to[32] = lo;
      }
    }
    __syncthreads();
    for (int c = 0; c < count; ++c) {
      const int64_t c0 = column(c);
      if (c0 >= d.K) break;
      uint4 y[2 * MT];
      const char *at = ring + (c % STAGES) * STEP;
      if (ALIGNED) {
        copies_wait<STAGES - 2>();
#pragma unroll
        for (int m = 0; m < 2 * MT; ++m) y[m] = reinterpret_cast<const uint4 *>(at)[m * 32 + lane];
      } else {
#pragma unroll
        for (int m = 0; m < 2 * MT; ++m) y[m] = load16<T, false>(rows[m], c0 + t * E, d.K, ok[m]);
      }
      float acc[MT][NT][4];
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[m][n][i] = 0.f;
      const auto multiply = [&](int k) {
        const uint4 *from = frag + (int64_t)k * MT * 2 * PER * 32 + lane;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          alignas(16) T w[4];
          if (AHEAD) {
            const char *slot = at + 2 * MT * 512 + ((k * NT + n) * 32 + lane) * S::WBYTES;
            if constexpr (sizeof(T) == 4)
              *reinterpret_cast<uint4 *>(w) = *reinterpret_cast<const uint4 *>(slot);
            else
              *reinterpret_cast<uint2 *>(w) = *reinterpret_cast<const uint2 *>(slot);
          } else {
            const int64_t col = c0 + gcol + 2 * n;
            load_ranks(W + (col < d.K ? col * d.rank : 0), (int64_t)k * 16 + 4 * t, d.rank, wvec, col < d.K, w);
          }
          if constexpr (sizeof(T) == 4) {
            float wh[4], wl[4];
            split4(*reinterpret_cast<const uint4 *>(w), wh, wl);
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
              for (int s = 0; s < 2; ++s) {
                const uint4 h = from[((m * 2 + 0) * PER + s) * 32], l = from[((m * 2 + 1) * PER + s) * 32];
                const auto f = [](uint32_t v) { return __uint_as_float(v); };
                mma_tf32(acc[m][n], f(l.x), f(l.y), f(l.z), f(l.w), wh[2 * s], wh[2 * s + 1]);
                mma_tf32(acc[m][n], f(h.x), f(h.y), f(h.z), f(h.w), wl[2 * s], wl[2 * s + 1]);
                mma_tf32(acc[m][n], f(h.x), f(h.y), f(h.z), f(h.w), wh[2 * s], wh[2 * s + 1]);
              }
          } else {
            const uint2 b = *reinterpret_cast<const uint2 *>(w);
#pragma unroll
            for (int m = 0; m < MT; ++m) {
              const uint4 h = from[(m * 2 + 0) * 32], l = from[(m * 2 + 1) * 32];
              mma_16<T>(acc[m][n], l.x, l.y, l.z, l.w, b.x, b.y);
              mma_16<T>(acc[m][n], h.x, h.y, h.z, h.w, b.x, b.y);
            }
          }
        }
      };
      if constexpr (RG < 0) {
        float sum[MT][NT][4];
        for (int k0 = 0; k0 < rg; k0 += 4) {
#pragma unroll 1
          for (int k = k0; k < min(rg, k0 + 4); ++k) multiply(k);
#pragma unroll
          for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                sum[m][n][i] = k0 ? sum[m][n][i] + acc[m][n][i] : acc[m][n][i];
                acc[m][n][i] = k0 + 4 < rg ? 0.f : sum[m][n][i];
              }
        }
      } else {
#pragma unroll(RG > 0 ? RG : 1)
        for (int k = 0; k < rg; ++k) multiply(k);
      }
      fetch(c + STAGES - 1);  // into the slots that step c - 1 has read
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          if (!ok[2 * m + half]) continue;
          T *e = reinterpret_cast<T *>(&y[2 * m + half]);
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int i = 0; i < 2; ++i)
              e[2 * n + i] = from_float<T>(std::is_same_v<T, __half>
                                             ? fmaf(acc[m][n][2 * half + i], 1.f / fit, to_float(e[2 * n + i]))
                                             : to_float(e[2 * n + i]) + acc[m][n][2 * half + i]);
          T *to = rows[2 * m + half] + c0 + t * E;
          if (ALIGNED) {
            if (c0 + t * E < d.K) *reinterpret_cast<uint4 *>(to) = y[2 * m + half];
          } else {
#pragma unroll
            for (int i = 0; i < E; ++i)
              if (c0 + t * E + i < d.K) to[i] = e[i];
          }
        }
    }
    copies_wait<0>();
    __syncthreads();  // the next tile's H goes where all have read this one's
  }
}

// ------------------------------------------------------------------ outer: sum_t h[t] x[t]^T

struct OuterArgs {
  const float *H;   // [tokens][rank]
  const void *X;    // rows of K elements
  int64_t x_stride, K, rank;
  int64_t chunk;    // places of one block
  int64_t blocks;   // blocks side by side over K
  int64_t slices;   // chunks
  float *parts;     // [chunk index + used index][rank][K]
  bool vec;         // the rows of X are vectors
  void *out;        // dA or dB (null: not wanted)
  bool scaled;      // times the adapter's scale
  bool turned;      // out is [adapter][K][rank], not [adapter][rank][K]
};

// dB and dA: nothing keeps the two apart, so one launch does both.
struct OuterPair {
  OuterArgs o[2];
};

// A lane's copies: 8 KB of rows for a warp.
template <typename T>
struct OuterShape {
  static constexpr int STAGES = sizeof(T) == 4 ? 8 : 4;
  static constexpr int RING = kWarps * 512;  // 16-byte slots of all warps
};

// Block: kWarps * (128 bytes of columns), one chunk of places, 16 * RM
// ranks.  A chunk may hold the end of one adapter and the beginning of
// others: each leaves a part of its own, in the slot chunk + index among
// the used.  The chunk's H lies in shared memory, a token every LD floats:
// lane (g, t) reads rank g of token t, bank 8 t + g.
template <typename T, int RM, bool ALIGNED>
__device__ __forceinline__ void outer_block(const AdapterArgs &q, const OuterArgs &d, int64_t block) {
  constexpr int E = 16 / sizeof(T), NT = E, COLS = 8 * E, LD = 16 * RM + 8;
  constexpr int TS = sizeof(T) == 4 ? 8 : 16;  // tokens of a step
  constexpr int NR = TS / 4, STAGES = OuterShape<T>::STAGES;
  constexpr int FLUSH = 32 / TS;               // steps between two sums outside the matrix unit
  extern __shared__ uint4 smem4[];             // the warps' rings, the chunk's rows, [chunk][LD] floats of H, its tokens
  int64_t *row_of = reinterpret_cast<int64_t *>(smem4 + OuterShape<T>::RING);  // elements before the row of X
  float *hs = reinterpret_cast<float *>(row_of + d.chunk);
  int32_t *tok = reinterpret_cast<int32_t *>(hs + d.chunk * LD);
  const int64_t slice = block / d.blocks, cblock = block % d.blocks;
  const int64_t p0 = slice * d.chunk;
  const int places = (int)(min((int64_t)q.p.head[2], p0 + d.chunk) - p0);
  if (places <= 0) return;
  const int64_t j0 = (int64_t)blockIdx.y * 16 * RM;
  // the chunk's tokens, then their H: two rounds of loads, each all at once,
  // the second one over while the first rows of X are on their way
  for (int i = threadIdx.x; i < places; i += kThreads) {
    tok[i] = q.p.perm[p0 + i];
    row_of[i] = tok[i] * d.x_stride;
  }
  // the first adapter of the chunk: the last used one that begins at or before p0
  int u = 0;
  {
    int lo = 0, hi = q.p.head[1];
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (q.p.used[mid].y <= p0)
        lo = mid + 1;
      else
        hi = mid;
    }
    u = lo - 1;
  }
  __syncthreads();
  const bool hvec = d.rank % 4 == 0 && (reinterpret_cast<uintptr_t>(d.H) & 15) == 0;
  if (hvec) {
    for (int i = threadIdx.x; i < places * 4 * RM; i += kThreads) {
      const int k = i / (4 * RM), j = i % (4 * RM) * 4;
      copy16(reinterpret_cast<uint4 *>(hs + k * LD + j), d.H + tok[k] * d.rank, j0 + j, d.rank, true);
    }
  } else {
#pragma unroll 8
    for (int i = threadIdx.x; i < places * 16 * RM; i += kThreads) {
      const int k = i / (16 * RM), j = i % (16 * RM);
      hs[k * LD + j] = j0 + j < d.rank ? d.H[tok[k] * d.rank + j0 + j] : 0.f;
    }
  }
  copies_commit();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
  const int64_t c0 = (cblock * kWarps + warp) * COLS, col = c0 + g * E;
  const T *X = static_cast<const T *>(d.X);
  const bool copy_ok = c0 + (lane & 7) * E < d.K;
  const T *copy_from = X + (copy_ok ? c0 + (lane & 7) * E : 0);
  uint4 *ring = smem4 + warp * STAGES * NR * 32;
  bool first = true;
  float fit = 1.f;  // float16: power of two that an adapter's H is scaled by
  __shared__ uint32_t largest;
  for (int p = 0; p < places; ++u) {
    const int4 use = q.p.used[u];
    const int end = (int)min((int64_t)places, (int64_t)use.y + use.z - p0);
    float sum[RM][NT][4];
#pragma unroll
    for (int m = 0; m < RM; ++m)
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) sum[m][n][i] = 0.f;
    float fresh[RM][NT][4];
    auto &acc = kFlush<T> ? fresh : sum;
#pragma unroll
    for (int m = 0; m < RM; ++m)
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[m][n][i] = 0.f;
    const auto flush = [&] {
      if constexpr (kFlush<T>) {
#pragma unroll
        for (int m = 0; m < RM; ++m)
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              sum[m][n][i] += acc[m][n][i];
              acc[m][n][i] = 0.f;
            }
      }
    };
    const int steps = (end - p + TS - 1) / TS;
    // Eight lanes copy a row's 128 bytes (one line for each request: by the
    // product's own layout, a quarter of a warp would ask for four lines, 32
    // bytes of each); chunk c of a row lies at c ^ turn(row), so that the
    // eight lanes that read together find it in eight different bank groups.
    const auto turn = [](int row) { return sizeof(T) == 4 ? 2 * (row & 3) : row & 6; };
    const auto fetch = [&](int step) {
      if (!ALIGNED) return;
      if (step < steps)
#pragma unroll
        for (int i = 0; i < NR; ++i) {
          const int row = 4 * i + (lane >> 3), k = p + step * TS + row;
          const bool in = copy_ok && k < end;
          copy16(ring + (step % STAGES) * NR * 32 + row * 8 + ((lane & 7) ^ turn(row)),
                 copy_from + (in ? row_of[k] : 0), 0, 1, in);
        }
      copies_commit();
    };
#pragma unroll
    for (int i = 0; i < STAGES - 1; ++i) fetch(i);
    if (first) {  // H is there when only the rows' copies are outstanding
      if (ALIGNED)
        copies_wait<STAGES - 1>();
      else
        copies_wait<0>();
      __syncthreads();
      first = false;
    }
    if constexpr (std::is_same_v<T, __half>) {
      // of this adapter's tokens alone: its neighbours' may lie far above them
      __syncthreads();  // all have read the scale of the adapter before
      if (threadIdx.x == 0) largest = 0u;
      __syncthreads();
      uint32_t most = 0u;
      for (int i = threadIdx.x; i < (end - p) * 16 * RM; i += kThreads)
        most = max(most, finite_bits(hs[(p + i / (16 * RM)) * LD + i % (16 * RM)]));
      atomicMax(&largest, most);
      __syncthreads();
      fit = half_scale(largest);
    }
    for (int step = 0; step < steps; ++step) {
      uint4 x[NR];
      float h[NR][2 * RM];
      if (ALIGNED) {
        copies_wait<STAGES - 2>();
        __syncwarp();
      }
#pragma unroll
      for (int i = 0; i < NR; ++i) {
        // rows of a lane: fp32 t and t + 4; 16-bit 2t, 2t + 1, 2t + 8, 2t + 9
        const int row = sizeof(T) == 4 ? t + 4 * i : 2 * t + (i & 1) + 8 * (i >> 1), k = p + step * TS + row;
        if (ALIGNED)
          x[i] = ring[(step % STAGES) * NR * 32 + row * 8 + (g ^ turn(row))];
        else
          x[i] = load16<T, false>(X + (k < end ? row_of[k] : 0), col, d.K, k < end);
#pragma unroll
        for (int m = 0; m < 2 * RM; ++m) {
          h[i][m] = k < end ? hs[k * LD + m * 8 + g] : 0.f;
          if (std::is_same_v<T, __half>) h[i][m] *= fit;
        }
      }
      fetch(step + STAGES - 1);  // into the slots that every lane read before this step's barrier
      if constexpr (sizeof(T) == 4) {
        float xh[2][4], xl[2][4];
        split4(x[0], xh[0], xl[0]);
        split4(x[1], xh[1], xl[1]);
#pragma unroll
        for (int m = 0; m < RM; ++m) {
          float hh[4], hl[4];
          const float v[4] = {h[0][2 * m], h[0][2 * m + 1], h[1][2 * m], h[1][2 * m + 1]};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            hh[i] = tf32_of(v[i]);
            hl[i] = v[i] - hh[i];
          }
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            mma_tf32(acc[m][n], hl[0], hl[1], hl[2], hl[3], xh[0][n], xh[1][n]);
            mma_tf32(acc[m][n], hh[0], hh[1], hh[2], hh[3], xl[0][n], xl[1][n]);
            mma_tf32(acc[m][n], hh[0], hh[1], hh[2], hh[3], xh[0][n], xh[1][n]);
          }
        }
      } else {
        uint32_t b[2][NT];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const uint32_t lo[4] = {x[2 * e].x, x[2 * e].y, x[2 * e].z, x[2 * e].w};
          const uint32_t hi[4] = {x[2 * e + 1].x, x[2 * e + 1].y, x[2 * e + 1].z, x[2 * e + 1].w};
#pragma unroll
          for (int n = 0; n < NT; ++n) b[e][n] = __byte_perm(lo[n / 2], hi[n / 2], n % 2 ? 0x7632 : 0x5410);
        }
#pragma unroll
        for (int m = 0; m < RM; ++m) {
          uint32_t hh[4], hl[4];
          split_pair<T>(h[0][2 * m], h[1][2 * m], hh[0], hl[0]);
          split_pair<T>(h[0][2 * m + 1], h[1][2 * m + 1], hh[1], hl[1]);
          split_pair<T>(h[2][2 * m], h[3][2 * m], hh[2], hl[2]);
          split_pair<T>(h[2][2 * m + 1], h[3][2 * m + 1], hh[3], hl[3]);
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            mma_16<T>(acc[m][n], hl[0], hl[1], hl[2], hl[3], b[0][n], b[1][n]);
            mma_16<T>(acc[m][n], hh[0], hh[1], hh[2], hh[3], b[0][n], b[1][n]);
          }
        }
      }
      if (step % FLUSH == FLUSH - 1) flush();
    }
    flush();
    copies_wait<0>();
    __syncwarp();
    p = end;
    float *out = d.parts + (slice + u) * d.rank * d.K;
#pragma unroll
    for (int m = 0; m < RM; ++m)
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const int64_t j = j0 + m * 16 + half * 8 + g;
        if (j >= d.rank) continue;
        // index 2t, 2t + 1 of product n is column c0 + (2t or 2t + 1) * E + n
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            const int64_t c = c0 + (2 * t + i) * E + n;
            if (c < d.K) out[j * d.K + c] = std::is_same_v<T, __half> ? sum[m][n][2 * half + i] * (1.f / fit) : sum[m][n][2 * half + i];
          }
      }
  }
}

template <typename T, int RM>
__global__ void __launch_bounds__(kThreads, 2) adapter_outer(const __grid_constant__ AdapterArgs q,
                                                          const __grid_constant__ OuterPair pair) {
  dependency_wait();
  dependency_launch();
  const int64_t first = pair.o[0].slices * pair.o[0].blocks;
  const bool second = blockIdx.x >= first;
  const OuterArgs &d = pair.o[second];
  const int64_t block = second ? blockIdx.x - first : blockIdx.x;
  if (d.vec)
    outer_block<T, RM, true>(q, d, block);
  else
    outer_block<T, RM, false>(q, d, block);
}

// The parts of each adapter, added in order, rounded once.  Block: 32
// columns of 32 ranks of one adapter (blockIdx.y); the sums turn in shared
// memory where the output is [adapter][K][rank].
template <typename T>
__global__ void __launch_bounds__(kThreads) adapter_outer_finish(const __grid_constant__ AdapterArgs q,
                                                                 const __grid_constant__ OuterPair pair) {
  __shared__ float turn[32][33];
  dependency_wait();
  dependency_launch();
  const auto tiles = [](const OuterArgs &d) { return d.out ? (d.K + 31) / 32 * ((d.rank + 31) / 32) : 0; };
  const int64_t first = tiles(pair.o[0]);
  const bool second = blockIdx.x >= first;
  const OuterArgs &d = pair.o[second];
  const int64_t block = second ? blockIdx.x - first : blockIdx.x, across = (d.K + 31) / 32;
  const int64_t c0 = block % across * 32, j0 = block / across * 32, per = d.rank * d.K;
  const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
  T *out = static_cast<T *>(d.out);
  for (int64_t n = blockIdx.y; n < q.a.adapters; n += gridDim.y) {
    const int u = q.p.index[n];
    float s[4] = {0.f, 0.f, 0.f, 0.f};  // ranks j0 + ty + 8 i
    if (u >= 0) {
      const int4 use = q.p.used[u];
      const int chunk = (int)d.chunk, s0 = use.y / chunk + u, s1 = (use.y + use.z - 1) / chunk + u;
      const float *at = d.parts + s0 * per + (j0 + ty) * d.K + c0 + tx;
      const bool in = c0 + tx < d.K;
#pragma unroll 8
      for (int k = s0; k <= s1; ++k, at += per)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (in && j0 + ty + 8 * i < d.rank) s[i] += at[8 * i * d.K];
      if (d.scaled) {
        const float scale = scale_of(q.a, (int)n);
#pragma unroll
        for (int i = 0; i < 4; ++i) s[i] *= scale;
      }
    }
    if (d.turned) {
#pragma unroll
      for (int i = 0; i < 4; ++i) turn[ty + 8 * i][tx] = s[i];
      __syncthreads();
      // 32 columns of min(32, rank) ranks: runs of ranks, one after another where rank <= 32
      const int ranks = (int)min((int64_t)32, d.rank - j0), cols = (int)min((int64_t)32, d.K - c0);
      for (int e = threadIdx.x; e < ranks * cols; e += kThreads) {
        const int c = e / ranks, j = e % ranks;
        out[n * per + (c0 + c) * d.rank + j0 + j] = from_float<T>(turn[j][c]);
      }
      __syncthreads();
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (c0 + tx < d.K && j0 + ty + 8 * i < d.rank)
          out[n * per + (j0 + ty + 8 * i) * d.K + c0 + tx] = from_float<T>(s[i]);
    }
  }
}

// Weights of the used adapters, each [rows][cols] turned to [cols][rows];
// two arrays in one launch.
struct TurnArgs {
  const void *in[2];
  void *out[2];
  int64_t rows[2], cols[2];
};
template <typename T>
__global__ void __launch_bounds__(kThreads) adapter_turn(const __grid_constant__ AdapterArgs q,
                                                         const __grid_constant__ TurnArgs a) {
  __shared__ T tile[32][33];
  dependency_wait();
  dependency_launch();
  const int64_t first = (a.rows[0] + 31) / 32 * ((a.cols[0] + 31) / 32);
  const int which = blockIdx.x >= first;
  const int64_t block = which ? blockIdx.x - first : blockIdx.x, rows = a.rows[which], cols = a.cols[which];
  const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
  const int64_t across = (cols + 31) / 32, r0 = block / across * 32, c0 = block % across * 32;
  for (int u = blockIdx.y; u < q.p.head[1]; u += gridDim.y) {
    const T *from = static_cast<const T *>(a.in[which]) + (int64_t)q.p.used[u].x * rows * cols;
    T *to = static_cast<T *>(a.out[which]) + (int64_t)u * rows * cols;
#pragma unroll
    for (int i = ty; i < 32; i += 8)
      if (r0 + i < rows && c0 + tx < cols) tile[i][tx] = from[(r0 + i) * cols + c0 + tx];
    __syncthreads();
#pragma unroll
    for (int i = ty; i < 32; i += 8)
      if (c0 + i < cols && r0 + tx < rows) to[(c0 + i) * rows + r0 + tx] = tile[tx][i];
    __syncthreads();
  }
}

// ------------------------------------------------------------------ few tokens

// Up to this many tokens are taken one by one, forward and backward: the
// weights of each are read for it alone, and no plan is made.  4096 x 4096
// at rank 16, fp32, one by one / by tiles: forward 10 tokens 7, 64 10.3, 100
// 16.8 / 13.5 us (768 -> 2304 at rank 8: 100 tokens 9 / 12.4); forward +
// backward of 64 tokens of one adapter 50 / 46 us and of 16 adapters 35 / 74
// us, of 128 tokens 63 / 46 and 52 / 74 us.  The count alone decides, which
// at the first and the last of these four is the slower way: how many tokens
// share an adapter is not known to the host, and rank does not enter.
constexpr int kFewTokens = 96, kFewTokensBack = 64;

struct FewArgs {
  const void *dY;
  int64_t dy_stride;
  const float *H;
  void *dX;
  int64_t dx_stride;
  void *dA, *dB;
  float *dH;
};

// The adapter of token t by the caller's offsets, or -1.
__device__ __forceinline__ int adapter_of(const snack_adapter_args &a, int64_t t) {
  const int i = request_of(a.offsets, (int)a.requests, (int32_t)t);
  if (i < 0) return -1;
  const int n = a.adapter[i];
  return n >= 0 && n < a.adapters ? n : -1;
}

// The same for one token, by a whole warp: the requests that begin at or
// before it are counted 128 at a time, so that two rounds of loads do (a
// search by halves waits for memory at every step).
__device__ __forceinline__ int adapter_of_warp(const snack_adapter_args &a, int64_t t) {
  constexpr int kMost = 1024;
  if (a.requests > kMost) return adapter_of(a, t);
  const int lane = threadIdx.x & 31, R = (int)a.requests;
  int begun = 0;
  for (int b = 0; b < R; b += 128) {
    bool is[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = b + 32 * i + lane;
      is[i] = r < R && a.offsets[r] <= t;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) begun += __popc(__ballot_sync(0xffffffffu, is[i]));
  }
  if (begun == 0) return -1;
  const int end = a.offsets[begun], n = a.adapter[begun - 1];
  return t < end && n >= 0 && n < a.adapters ? n : -1;
}

// Forward of few tokens: a cluster of blocks for each token.  Every block
// takes a share of X's row and of each row of A, sends its sums to the
// others' shared memory, and then has H and a share of the columns of Y.  The
// rows of B that it will need are on their way from the start.  (Two kernels,
// one for H and one for Y, took 9.8 us for 64 tokens, 4096 -> 4096 at rank 16
// in bf16, and 5.7 us for 8 tokens, 768 -> 2304 at rank 8.)
constexpr int kFewBlocks = 8;
constexpr int kFewAhead = 32 * 1024;  // most bytes of B copied ahead by a block

template <typename T, bool ALIGNED>
__global__ void __cluster_dims__(kFewBlocks, 1, 1) __launch_bounds__(kThreads)
    adapter_few(const __grid_constant__ AdapterArgs q, T *Y, int64_t y_stride, bool ahead) {
  constexpr int E = 16 / sizeof(T), J = 4;
  extern __shared__ uint4 smem4[];  // [blocks][rank] floats: all blocks' sums; [rank]: scaled H; rows of B
  const snack_adapter_args &a = q.a;
  cg::cluster_group cluster = cg::this_cluster();
  constexpr int blocks = kFewBlocks;
  const int part = (int)cluster.block_rank(), rank = (int)a.rank;
  float *sums = reinterpret_cast<float *>(smem4), *h = sums + blocks * rank;
  T *rows = reinterpret_cast<T *>(smem4 + ((blocks + 1) * rank + 3) / 4);
  dependency_wait();
  dependency_launch();
  const int64_t tkn = blockIdx.x / blocks;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int n = adapter_of_warp(a, tkn);
  if (n < 0) {  // the whole cluster
    for (int j = part * kThreads + threadIdx.x; j < rank; j += blocks * kThreads) q.H[tkn * rank + j] = 0.f;
    return;
  }
  // this block's columns of Y, from a multiple of 8 on
  const int64_t share = ((a.out + blocks - 1) / blocks + 7) / 8 * 8;
  const int64_t o0 = min(a.out, part * share), o1 = min(a.out, o0 + share);
  const T *B = static_cast<const T *>(a.B) + ((int64_t)n * a.out + o0) * rank;
  if (ahead) {
    const int64_t bytes = (o1 - o0) * rank * (int64_t)sizeof(T);
    for (int64_t i = threadIdx.x * 16; i < bytes; i += kThreads * 16)
      copy_async16(reinterpret_cast<char *>(rows) + i, reinterpret_cast<const char *>(B) + i);
  }
  copies_commit();
  T *y = Y + tkn * y_stride + o0;
  const float y0 = threadIdx.x < o1 - o0 ? to_float(y[threadIdx.x]) : 0.f;

  const int64_t slice = ((a.in + blocks - 1) / blocks + E - 1) / E * E;
  const int64_t k0 = min(a.in, part * slice), k1 = min(a.in, k0 + slice);
  const T *x = static_cast<const T *>(a.X) + tkn * a.x_stride;
  const T *A = static_cast<const T *>(a.A) + (int64_t)n * rank * a.in;
  cluster.sync();  // all blocks are there: their shared memory may be written
  for (int j0 = warp * J; j0 < rank; j0 += kWarps * J) {
    float s[J];
#pragma unroll
    for (int i = 0; i < J; ++i) s[i] = 0.f;
#pragma unroll 2
    for (int64_t k = k0 + lane * E; k < k1; k += 32 * E) {
      const uint4 xv = load16<T, ALIGNED>(x, k, k1, true);
      uint4 w[J];
#pragma unroll
      for (int i = 0; i < J; ++i) w[i] = load16<T, ALIGNED>(A + (int64_t)min(j0 + i, rank - 1) * a.in, k, k1, j0 + i < rank);
#pragma unroll
      for (int i = 0; i < J; ++i)
#pragma unroll
        for (int e = 0; e < E; ++e)
          s[i] = fmaf(to_float(reinterpret_cast<const T *>(&xv)[e]), to_float(reinterpret_cast<const T *>(&w[i])[e]), s[i]);
    }
#pragma unroll
    for (int i = 0; i < J; ++i) s[i] = warp_sum(s[i]);
    // lane 8 i + b sends rank j0 + i to block b
    const int i = lane >> 3;
    const float v = i == 0 ? s[0] : i == 1 ? s[1] : i == 2 ? s[2] : s[3];
    if (j0 + i < rank) cluster.map_shared_rank(sums, lane & 7)[part * rank + j0 + i] = v;
  }
  cluster.sync();  // and none leaves before all have written
  const float scale = scale_of(a, n);
  for (int j = threadIdx.x; j < rank; j += kThreads) {
    float v = 0.f;
#pragma unroll
    for (int b = 0; b < blocks; ++b) v += sums[b * rank + j];
    h[j] = v * scale;
    if (part == 0) q.H[tkn * rank + j] = v;
  }
  copies_wait<0>();
  __syncthreads();
  const bool vec = rank % E == 0 && (reinterpret_cast<uintptr_t>(a.B) & 15) == 0;
  for (int64_t o = threadIdx.x; o < o1 - o0; o += kThreads) {
    const T *w = ahead ? rows + o * rank : B + o * rank;
    float s = 0.f;
    if (vec) {
#pragma unroll 4
      for (int j = 0; j < rank; j += E) {
        const uint4 v = *reinterpret_cast<const uint4 *>(w + j);
#pragma unroll
        for (int e = 0; e < E; ++e) s = fmaf(h[j + e], to_float(reinterpret_cast<const T *>(&v)[e]), s);
      }
    } else {
      for (int j = 0; j < rank; ++j) s = fmaf(h[j], to_float(w[j]), s);
    }
    y[o] = from_float<T>((o < kThreads ? y0 : to_float(y[o])) + s);
  }
}

// dH of few tokens.  Block (token, 16 ranks): a thread takes every 256th row of B.
constexpr int kFewRanks = 16;
template <typename T>
__global__ void __launch_bounds__(kThreads) adapter_few_rank(const __grid_constant__ AdapterArgs q,
                                                             const __grid_constant__ FewArgs b) {
  constexpr int E = 16 / sizeof(T);
  __shared__ float part[kWarps][kFewRanks];
  dependency_wait();
  dependency_launch();
  const snack_adapter_args &a = q.a;
  const int64_t tkn = blockIdx.x, j0 = (int64_t)blockIdx.y * kFewRanks;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int n = adapter_of_warp(a, tkn), ranks = (int)min((int64_t)kFewRanks, a.rank - j0);
  float s[kFewRanks];
#pragma unroll
  for (int j = 0; j < kFewRanks; ++j) s[j] = 0.f;
  if (n >= 0) {
    const T *dy = static_cast<const T *>(b.dY) + tkn * b.dy_stride;
    const T *w = static_cast<const T *>(a.B) + (int64_t)n * a.out * a.rank + j0;
    const bool vec = a.rank % E == 0 && (reinterpret_cast<uintptr_t>(a.B) & 15) == 0;
#pragma unroll 2
    for (int64_t o = threadIdx.x; o < a.out; o += kThreads) {
      const float d = to_float(dy[o]);
      if (vec) {
#pragma unroll
        for (int v = 0; v < kFewRanks / E; ++v) {
          const uint4 x = load16<T, true>(w + o * a.rank, v * E, ranks, true);
#pragma unroll
          for (int e = 0; e < E; ++e) s[v * E + e] = fmaf(d, to_float(reinterpret_cast<const T *>(&x)[e]), s[v * E + e]);
        }
      } else {
#pragma unroll
        for (int j = 0; j < kFewRanks; ++j)
          if (j < ranks) s[j] = fmaf(d, to_float(w[o * a.rank + j]), s[j]);
      }
    }
  }
  // sixteen sums over the warp: each step halves the ranks that a lane still holds
#pragma unroll
  for (int o = 8; o >= 1; o >>= 1)
#pragma unroll
    for (int j = 0; j < o; ++j) {
      const bool up = lane & o;
      const float send = up ? s[j] : s[j + o], keep = up ? s[j + o] : s[j];
      s[j] = keep + __shfl_xor_sync(0xffffffffu, send, o);
    }
  s[0] += __shfl_xor_sync(0xffffffffu, s[0], 16);
  if (lane < kFewRanks) part[warp][lane] = s[0];
  __syncthreads();
  if (threadIdx.x < ranks) {
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) v += part[w][threadIdx.x];
    b.dH[tkn * a.rank + j0 + threadIdx.x] = n < 0 ? 0.f : v * scale_of(a, n);
  }
}

// dX of few tokens.  Block (256 columns, token).
template <typename T>
__global__ void __launch_bounds__(kThreads) adapter_few_input(const __grid_constant__ AdapterArgs q,
                                                              const __grid_constant__ FewArgs b) {
  extern __shared__ float h[];
  dependency_wait();
  dependency_launch();
  const snack_adapter_args &a = q.a;
  const int64_t tkn = blockIdx.y, i = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  const int n = adapter_of_warp(a, tkn);
  if (n < 0) return;
  for (int64_t j = threadIdx.x; j < a.rank; j += kThreads) h[j] = b.dH[tkn * a.rank + j];
  __syncthreads();
  if (i >= a.in) return;
  const T *w = static_cast<const T *>(a.A) + (int64_t)n * a.rank * a.in + i;
  T *dx = static_cast<T *>(b.dX) + tkn * b.dx_stride + i;
  const float x0 = to_float(*dx);
  float s = 0.f;
#pragma unroll 8
  for (int64_t j = 0; j < a.rank; ++j) s = fmaf(h[j], to_float(w[j * a.in]), s);
  *dx = from_float<T>(x0 + s);
}

// dA and dB of few tokens.  Block (256 columns of in, then of out; adapter;
// 16 ranks): the adapter's tokens in their order.
template <typename T>
__global__ void __launch_bounds__(kThreads) adapter_few_weights(const __grid_constant__ AdapterArgs q,
                                                                const __grid_constant__ FewArgs b) {
  __shared__ int tok[kFewTokensBack], counts[kFewTokensBack / 32];
  __shared__ float h[kFewTokensBack][kFewRanks];
  dependency_wait();
  dependency_launch();
  const snack_adapter_args &a = q.a;
  const int64_t in_blocks = b.dA ? (a.in + kThreads - 1) / kThreads : 0;
  const bool db = blockIdx.x >= in_blocks;
  const int64_t K = db ? a.out : a.in, j0 = (int64_t)blockIdx.z * kFewRanks;
  const int64_t i = (int64_t)(blockIdx.x - (db ? in_blocks : 0)) * kThreads + threadIdx.x;
  const int ranks = (int)min((int64_t)kFewRanks, a.rank - j0);
  const int mine = threadIdx.x < a.tokens ? adapter_of(a, threadIdx.x) : -1;
  const T *X = static_cast<const T *>(db ? b.dY : a.X) + (i < K ? i : 0);
  const int64_t stride = db ? b.dy_stride : a.x_stride;
  const float *H = db ? b.H : b.dH;
  for (int64_t n = blockIdx.y; n < a.adapters; n += gridDim.y) {
    __syncthreads();  // the adapter before is done with the shared arrays
    const bool is = mine == n;
    const uint32_t vote = __ballot_sync(0xffffffffu, is);
    if (threadIdx.x < kFewTokensBack && (threadIdx.x & 31) == 0) counts[threadIdx.x / 32] = __popc(vote);
    __syncthreads();
    int before = 0, all = 0;
#pragma unroll
    for (int w = 0; w < kFewTokensBack / 32; ++w) {
      before += w < (int)threadIdx.x / 32 ? counts[w] : 0;
      all += counts[w];
    }
    if (is) tok[before + __popc(vote & ((1u << (threadIdx.x & 31)) - 1))] = threadIdx.x;
    __syncthreads();
    for (int e = threadIdx.x; e < all * kFewRanks; e += kThreads) {
      const int k = e / kFewRanks, j = e % kFewRanks;
      h[k][j] = j < ranks ? H[tok[k] * a.rank + j0 + j] : 0.f;
    }
    __syncthreads();
    if (i >= K) continue;
    float s[kFewRanks];
#pragma unroll
    for (int j = 0; j < kFewRanks; ++j) s[j] = 0.f;
#pragma unroll 4
    for (int k = 0; k < all; ++k) {
      const float x = to_float(X[tok[k] * stride]);
#pragma unroll
      for (int j = 0; j < kFewRanks; ++j) s[j] = fmaf(h[k][j], x, s[j]);
    }
    const float scale = db && all > 0 ? scale_of(a, (int)n) : 1.f;
#pragma unroll
    for (int j = 0; j < kFewRanks; ++j) {
      if (j >= ranks) continue;
      if (db)
        static_cast<T *>(b.dB)[(n * a.out + i) * a.rank + j0 + j] = from_float<T>(s[j] * scale);
      else
        static_cast<T *>(b.dA)[(n * a.rank + j0 + j) * a.in + i] = from_float<T>(s[j]);
    }
  }
}

// ------------------------------------------------------------------ host

const char *bad_args(const snack_adapter_args *a) {
  if (!a) return "args is NULL";
  if (a->tokens < 0 || a->tokens > 0x7fffffffLL || a->requests < 0 || a->requests > 0x7ffffffeLL)
    return "tokens and requests must be in [0, 2^31)";
  if (a->adapters < 0 || a->adapters > 65536) return "adapters must be in [0, 65536]";
  if (a->in < 1 || a->out < 1 || a->in > 0x7fffffffLL || a->out > 0x7fffffffLL)
    return "in and out must be in [1, 2^31)";
  if (a->rank < 1 || a->rank > 512) return "rank must be in [1, 512]";
  if (!known_type(a->type)) return "type is not one of snack_dtype";
  if (a->tokens > 0 && a->requests > 0 && (!a->offsets || !a->adapter)) return "offsets or adapter is NULL";
  if (a->tokens > 0 && a->adapters > 0 && (!a->X || !a->A || !a->B)) return "X, A or B is NULL";
  if (a->tokens > 1 && a->x_stride < a->in) return "x_stride is below in";
  const int64_t e = type_bytes(a->type);
  if (!aligned_to(a->X, e) || !aligned_to(a->A, e) || !aligned_to(a->B, e) || !aligned_to(a->offsets, 4) ||
      !aligned_to(a->adapter, 4) || !aligned_to(a->scale, 4))
    return "a pointer is not aligned to its elements";
  return nullptr;
}

// Rows of `width` elements, `stride` apart.
struct RowsAt {
  const void *p;
  int64_t stride, width;
};

// Whether two arrays of as many rows share an element.  Column ranges of one
// buffer (equal strides) do not; of other strides over one piece of memory,
// which nothing needs, it is not worked out.
bool overlap(const RowsAt &a, const RowsAt &b, int64_t rows, int type) {
  if (!a.p || !b.p || rows < 1) return false;
  const int64_t e = type_bytes(type);
  const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
  const auto bytes = [&](const RowsAt &r) { return (uintptr_t)(((rows - 1) * r.stride + r.width) * e); };
  if (x >= y + bytes(b) || y >= x + bytes(a)) return false;
  if (rows == 1 || a.stride != b.stride) return true;
  const int64_t step = a.stride * e;
  const int64_t at = x <= y ? (int64_t)((y - x) % step) : (step - (int64_t)((x - y) % step)) % step;  // b's columns from a's on
  return at < a.width * e || at + b.width * e > step;
}

int64_t align16(int64_t b) { return (b + 15) / 16 * 16; }

// Lays the plan out in `ws` (null: only its size).
int64_t lay_plan(const snack_adapter_args &a, Plan *p, char *ws) {
  p->max_used = std::min(a.adapters, std::min(a.requests, a.tokens));
  p->max_tiles = a.tokens / kTile + p->max_used;
  int64_t at = 0;
  const auto take = [&](int64_t bytes) {
    char *r = ws ? ws + at : nullptr;
    at += align16(bytes);
    return r;
  };
  p->head = reinterpret_cast<int32_t *>(take(16));
  p->tiles = reinterpret_cast<int4 *>(take(p->max_tiles * 16));
  p->used = reinterpret_cast<int4 *>(take(p->max_used * 16));
  p->perm = reinterpret_cast<int32_t *>(take(a.tokens * 4));
  p->index = reinterpret_cast<int32_t *>(take(a.adapters * 4));
  const bool many = a.requests > kPlanThreads;
  p->soff = reinterpret_cast<int32_t *>(take(many ? (a.requests + 1) * 4 : 0));
  p->place = reinterpret_cast<int32_t *>(take(many ? a.requests * 4 : 0));
  p->base = reinterpret_cast<int32_t *>(take(many ? a.adapters * 4 : 0));
  return at;
}

cudaError_t launch_plan(const AdapterArgs &q, cudaStream_t s) {
  const snack_adapter_args &a = q.a;
  if (a.requests <= kPlanThreads) {
    const int th = a.requests <= 128 ? 128 : kPlanThreads;
    const int64_t blocks = std::max<int64_t>(1, std::min<int64_t>(device_sms(), (a.tokens + th - 1) / th));
    return launch_kernel(th == 128 ? plan_small<128> : plan_small<kPlanThreads>, dim3((unsigned)blocks), th, 0, true,
                         s, q);
  }
  cudaError_t e = launch_kernel(plan_requests, dim3(1), kPlanThreads, 0, true, s, q);
  if (e != cudaSuccess) return e;
  const int64_t blocks = std::min<int64_t>((a.tokens + kThreads - 1) / kThreads, device_sms() * 8);
  return launch_kernel(plan_tokens, dim3((unsigned)blocks), kThreads, 0, true, s, q);
}

bool vector_rows(const void *p, int64_t stride, int64_t width, int type) {
  const int64_t e = 16 / type_bytes(type);
  return aligned_to(p, 16) && width % e == 0 && stride % e == 0;
}

template <typename T, int NT>
cudaError_t launch_down_nt(const AdapterArgs &q, const DownArgs &d, bool vec, cudaStream_t s) {
  const size_t smem = DownShape<NT>::SMEM;
  auto k = vec ? adapter_down<T, NT, true> : adapter_down<T, NT, false>;
  const cudaError_t e = allow_smem(k, smem);
  // blocks of a tile: while all of them fit the GPU at once and each warp keeps a step
  const int64_t room = (int64_t)device_sms() * (NT <= 2 ? 2 : 1);
  int64_t blocks = 1;
  while (blocks < 8 && 2 * q.p.max_tiles * blocks <= room && d.K > blocks * kWarps * 2 * Group<T>::K) blocks *= 2;
  if (q.p.max_tiles * blocks > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  const dim3 grid((unsigned)(q.p.max_tiles * blocks), (unsigned)((d.rank + kRankPass - 1) / kRankPass));
  return e != cudaSuccess ? e : launch_clusters(k, grid, (int)blocks, kThreads, smem, true, s, q, d);
}

template <typename T>
cudaError_t launch_down(const AdapterArgs &q, const DownArgs &d, cudaStream_t s) {
  if (q.p.max_tiles == 0) return cudaSuccess;
  const bool vec = vector_rows(d.X, d.x_stride, d.K, q.a.type) && aligned_to(d.W, 16);
  if (d.rank <= 8) return launch_down_nt<T, 1>(q, d, vec, s);
  if (d.rank <= 16) return launch_down_nt<T, 2>(q, d, vec, s);
  if (d.rank <= 32) return launch_down_nt<T, 4>(q, d, vec, s);
  return launch_down_nt<T, 8>(q, d, vec, s);
}

template <typename T>
cudaError_t launch_up(const AdapterArgs &q, const UpArgs &d, cudaStream_t s) {
  if (q.p.max_tiles == 0) return cudaSuccess;
  using S = UpShape<T>;
  const int64_t most = q.p.max_tiles * ((d.K + S::BLOCK - 1) / S::BLOCK);
  const dim3 grid((unsigned)std::min<int64_t>(most, 2 * device_sms()));
  const bool wvec = d.rank % 4 == 0 && aligned_to(d.W, 4 * sizeof(T));
  const bool vec = vector_rows(d.Y, d.y_stride, d.K, q.a.type);
  const int rg = !vec || !wvec || d.rank > 32 ? 0 : (d.rank > 16 ? 2 : 1);
  constexpr int kHigh = kFlush<T> ? -1 : 0;  // the form above 64 ranks
  auto k = rg == 2 ? adapter_up<T, 2, true> : adapter_up<T, 1, true>;
  if (rg == 0) k = vec ? adapter_up<T, 0, true> : adapter_up<T, 0, false>;
  if (d.rank > 64) k = vec ? adapter_up<T, kHigh, true> : adapter_up<T, kHigh, false>;
  const size_t smem = S::smem(rg, d.rank);
  const cudaError_t e = allow_smem(k, smem);
  return e != cudaSuccess ? e : launch_kernel(k, grid, kThreads, smem, true, s, q, d);
}

// Places of one block of `outer`: one round of blocks, two on each SM.  At
// least 64 places, below which the parts cost more than the split gains, but
// no more than an adapter has on average (a block that meets many adapters
// waits for the first rows of each): 128 tokens of 16 adapters, 4096 x 4096
// at rank 16, forward + backward 90 -> 72 us with 16 places, 256 tokens of
// one adapter 46 -> 55.  At most 448 at 16 ranks and 256 at 32 (two blocks'
// rings and H fit an SM).
int64_t outer_chunk(const snack_adapter_args &a, int64_t K) {
  const int64_t cols = kWarps * 8 * (16 / type_bytes(a.type)), ranks = outer_ranks(a.rank);
  const int64_t blocks = (K + cols - 1) / cols * ((a.rank + ranks - 1) / ranks);
  const int64_t split = std::max<int64_t>(1, (int64_t)device_sms() * 2 / blocks);
  const int64_t used = std::max<int64_t>(1, std::min(a.adapters, std::min(a.requests, a.tokens)));
  const int64_t least = std::max<int64_t>(16, std::min<int64_t>(64, a.tokens / used / 16 * 16));
  const int64_t c = (a.tokens + split - 1) / split;
  return std::max<int64_t>(least, std::min<int64_t>(ranks == 16 ? 448 : 256, (c + 15) / 16 * 16));
}

int64_t outer_bytes(const snack_adapter_args &a, int64_t K) {
  const int64_t chunk = outer_chunk(a, K), used = std::min(a.adapters, std::min(a.requests, a.tokens));
  return align16(((a.tokens + chunk - 1) / chunk + used) * a.rank * K * 4);
}

// dB and dA (those whose `out` is set), then the sums of their parts.
template <typename T>
cudaError_t launch_outer(const AdapterArgs &q, OuterPair pair, cudaStream_t s) {
  const snack_adapter_args &a = q.a;
  const int64_t cols = kWarps * 8 * (16 / (int64_t)sizeof(T)), ranks = outer_ranks(a.rank);
  int64_t blocks = 0, tiles = 0, chunk = 0;
  for (OuterArgs &d : pair.o) {
    if (!d.out) continue;
    d.chunk = outer_chunk(a, d.K);
    d.blocks = (d.K + cols - 1) / cols;
    d.slices = (a.tokens + d.chunk - 1) / d.chunk;
    d.vec = vector_rows(d.X, d.x_stride, d.K, a.type);
    blocks += d.slices * d.blocks;
    tiles += (d.K + 31) / 32 * ((d.rank + 31) / 32);
    chunk = std::max(chunk, d.chunk);
  }
  if (blocks > 0x7fffffffLL || tiles > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  cudaError_t e = cudaSuccess;
  if (q.p.max_used > 0) {
    auto k = ranks == 16 ? adapter_outer<T, 1> : adapter_outer<T, 2>;
    const size_t smem = (size_t)OuterShape<T>::RING * 16 + (size_t)chunk * ((ranks + 8 + 1) * 4 + 8);
    if ((e = allow_smem(k, smem)) != cudaSuccess) return e;
    const dim3 grid((unsigned)blocks, (unsigned)((a.rank + ranks - 1) / ranks));
    if ((e = launch_kernel(k, grid, kThreads, smem, true, s, q, pair)) != cudaSuccess) return e;
  }
  const dim3 grid((unsigned)tiles, (unsigned)std::min<int64_t>(a.adapters, 65535));
  return launch_kernel(adapter_outer_finish<T>, grid, kThreads, 0, true, s, q, pair);
}

// Turns B (and A, where dX is wanted) of the used adapters.
template <typename T>
cudaError_t launch_turn(const AdapterArgs &q, void *Bt, void *At, cudaStream_t s) {
  const snack_adapter_args &a = q.a;
  if (q.p.max_used == 0) return cudaSuccess;
  const TurnArgs t = {{a.B, a.A}, {Bt, At}, {a.out, a.rank}, {a.rank, a.in}};
  int64_t blocks = 0;
  for (int i = 0; i < (At ? 2 : 1); ++i) blocks += (t.rows[i] + 31) / 32 * ((t.cols[i] + 31) / 32);
  if (blocks > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  const dim3 grid((unsigned)blocks, (unsigned)std::min<int64_t>(q.p.max_used, 65535));
  return launch_kernel(adapter_turn<T>, grid, kThreads, 0, true, s, q, t);
}

template <typename T>
cudaError_t forward(const AdapterArgs &q, void *Y, int64_t y_stride, cudaStream_t s) {
  const snack_adapter_args &a = q.a;
  if (a.tokens <= kFewTokens) {
    constexpr int64_t blocks = kFewBlocks;
    const int64_t share = ((a.out + blocks - 1) / blocks + 7) / 8 * 8, bytes = share * a.rank * (int64_t)sizeof(T);
    const bool ahead = bytes <= kFewAhead && aligned_to(a.B, 16) && a.out * a.rank * (int64_t)sizeof(T) % 16 == 0;
    const size_t smem = (size_t)((blocks + 1) * a.rank + 3) / 4 * 16 + (ahead ? (size_t)bytes : 0);
    auto k = vector_rows(a.X, a.x_stride, a.in, a.type) && aligned_to(a.A, 16) ? adapter_few<T, true> : adapter_few<T, false>;
    const cudaError_t e = allow_smem(k, smem);
    return e != cudaSuccess ? e
                            : launch_kernel(k, dim3((unsigned)(a.tokens * blocks)), kThreads, smem, true, s, q,
                                            static_cast<T *>(Y), y_stride, ahead);
  }
  cudaError_t e = launch_plan(q, s);
  if (e != cudaSuccess) return e;
  const DownArgs d = {a.X, a.A, a.x_stride, a.in, a.rank, false, false, q.H};
  if ((e = launch_down<T>(q, d, s)) != cudaSuccess) return e;
  const UpArgs u = {q.H, a.B, Y, y_stride, a.out, a.rank, false, true};
  return launch_up<T>(q, u, s);
}

struct Back {
  const void *dY;
  int64_t dy_stride;
  const float *H;
  void *dX;
  int64_t dx_stride;
  void *dA, *dB;
  float *dH;      // [tokens][rank]
  void *At, *Bt;  // [used][in][rank], [used][rank][out]
  float *parts_a, *parts_b;
};

template <typename T>
cudaError_t few_backward(const AdapterArgs &q, const Back &b, cudaStream_t s) {
  const snack_adapter_args &a = q.a;
  const FewArgs f = {b.dY, b.dy_stride, b.H, b.dX, b.dx_stride, b.dA, b.dB, b.dH};
  const unsigned tokens = (unsigned)a.tokens, passes = (unsigned)((a.rank + kFewRanks - 1) / kFewRanks);
  const int64_t in = (a.in + kThreads - 1) / kThreads, out = (a.out + kThreads - 1) / kThreads;
  cudaError_t e = cudaSuccess;
  if (b.dX || b.dA) e = launch_kernel(adapter_few_rank<T>, dim3(tokens, passes), kThreads, 0, true, s, q, f);
  if (e == cudaSuccess && b.dX)
    e = launch_kernel(adapter_few_input<T>, dim3((unsigned)in, tokens), kThreads, (size_t)a.rank * 4, true, s, q, f);
  const int64_t blocks = (b.dA ? in : 0) + (b.dB ? out : 0);
  if (e == cudaSuccess && blocks > 0)
    e = launch_kernel(adapter_few_weights<T>,
                      dim3((unsigned)blocks, (unsigned)std::min<int64_t>(a.adapters, 65535), passes), kThreads, 0,
                      true, s, q, f);
  return e;
}

template <typename T>
cudaError_t backward(const AdapterArgs &q, const Back &b, cudaStream_t s) {
  const snack_adapter_args &a = q.a;
  if (a.tokens <= kFewTokensBack) return few_backward<T>(q, b, s);
  cudaError_t e = launch_plan(q, s);
  if (e != cudaSuccess) return e;
  if (b.dX || b.dA) {
    if ((e = launch_turn<T>(q, b.Bt, b.dX ? b.At : nullptr, s)) != cudaSuccess) return e;
    const DownArgs d = {b.dY, b.Bt, b.dy_stride, a.out, a.rank, true, true, b.dH};
    if ((e = launch_down<T>(q, d, s)) != cudaSuccess) return e;
  }
  if (b.dX) {
    const UpArgs u = {b.dH, b.At, b.dX, b.dx_stride, a.in, a.rank, true, false};
    if ((e = launch_up<T>(q, u, s)) != cudaSuccess) return e;
  }
  if (b.dA || b.dB) {
    OuterPair pair = {};
    pair.o[0] = {b.H, b.dY, b.dy_stride, a.out, a.rank, 0, 0, 0, b.parts_b, false, b.dB, true, true};
    pair.o[1] = {b.dH, a.X, a.x_stride, a.in, a.rank, 0, 0, 0, b.parts_a, false, b.dA, false, false};
    if ((e = launch_outer<T>(q, pair, s)) != cudaSuccess) return e;
  }
  return cudaSuccess;
}

#define SNACK_TYPES(type, F, ...)                                                     \
  ((type) == SNACK_F32 ? F<float>(__VA_ARGS__) : (type) == SNACK_BF16 ? F<__nv_bfloat16>(__VA_ARGS__) \
                                                                      : F<__half>(__VA_ARGS__))

}  // namespace
}  // namespace snack

extern "C" size_t snack_adapter_forward_workspace(const snack_adapter_args *args) {
  using namespace snack;
  if (bad_args(args) || args->tokens <= kFewTokens) return 0;
  Plan p;
  return (size_t)lay_plan(*args, &p, nullptr);
}

extern "C" snack_status snack_adapter_forward(const snack_adapter_args *args, void *Y, int64_t y_stride,
                                              float *H, void *workspace, void *stream) {
  using namespace snack;
  if (const char *bad = bad_args(args)) return refuse(SNACK_ERR_INVALID_ARG, bad);
  const snack_adapter_args &a = *args;
  if (a.tokens == 0) return SNACK_OK;
  if (!Y || !H) return refuse(SNACK_ERR_INVALID_ARG, "Y or H is NULL");
  if (a.tokens > kFewTokens && (!workspace || !aligned_to(workspace, 16)))
    return refuse(SNACK_ERR_INVALID_ARG, "workspace must be 16-byte aligned device memory");
  if (a.tokens > 1 && y_stride < a.out) return refuse(SNACK_ERR_INVALID_ARG, "y_stride is below out");
  if (!aligned_to(Y, type_bytes(a.type)) || !aligned_to(H, 4))
    return refuse(SNACK_ERR_INVALID_ARG, "a pointer is not aligned to its elements");
  if (overlap({a.X, a.x_stride, a.in}, {Y, y_stride, a.out}, a.tokens, a.type))
    return refuse(SNACK_ERR_INVALID_ARG, "Y overlaps X");
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  AdapterArgs q = {};
  q.a = a;
  q.H = H;
  if (a.tokens > kFewTokens) lay_plan(a, &q.p, static_cast<char *>(workspace));
  const cudaError_t e = SNACK_TYPES(a.type, forward, q, Y, y_stride, s);
  return e == cudaSuccess ? SNACK_OK : cuda_status(e, "adapter launch");
}

namespace snack {
namespace {

// The backward's scratch: the plan, dH, turned weights of the used adapters,
// parts of dA and dB.
int64_t lay_back(const snack_adapter_args &a, Plan *p, Back *b, char *ws) {
  if (a.tokens <= kFewTokensBack) {
    b->dH = reinterpret_cast<float *>(ws);
    return align16(std::max<int64_t>(4, a.tokens * a.rank * 4));
  }
  int64_t at = lay_plan(a, p, ws);
  const auto take = [&](int64_t bytes) {
    char *r = ws ? ws + at : nullptr;
    at += align16(bytes);
    return r;
  };
  const int64_t e = type_bytes(a.type);
  b->dH = reinterpret_cast<float *>(take(a.tokens * a.rank * 4));
  b->At = take(p->max_used * a.in * a.rank * e);
  b->Bt = take(p->max_used * a.out * a.rank * e);
  b->parts_a = reinterpret_cast<float *>(take(outer_bytes(a, a.in)));
  b->parts_b = reinterpret_cast<float *>(take(outer_bytes(a, a.out)));
  return at;
}

}  // namespace
}  // namespace snack

extern "C" size_t snack_adapter_backward_workspace(const snack_adapter_args *args) {
  using namespace snack;
  if (bad_args(args)) return 16;
  Plan p;
  Back b;
  return (size_t)lay_back(*args, &p, &b, nullptr);
}

extern "C" snack_status snack_adapter_backward(const snack_adapter_args *args, const void *dY,
                                               int64_t dy_stride, const float *H, void *dX, int64_t dx_stride,
                                               void *dA, void *dB, void *workspace, void *stream) {
  using namespace snack;
  if (const char *bad = bad_args(args)) return refuse(SNACK_ERR_INVALID_ARG, bad);
  const snack_adapter_args &a = *args;
  if (a.tokens > 0 && (!workspace || !aligned_to(workspace, 16)))
    return refuse(SNACK_ERR_INVALID_ARG, "workspace must be 16-byte aligned device memory");
  if (a.tokens > 0 && (!dY || !H)) return refuse(SNACK_ERR_INVALID_ARG, "dY or H is NULL");
  if (a.tokens > 1 && (dy_stride < a.out || (dX && dx_stride < a.in)))
    return refuse(SNACK_ERR_INVALID_ARG, "a row stride is below its width");
  const int64_t e0 = type_bytes(a.type);
  if (!aligned_to(dY, e0) || !aligned_to(dX, e0) || !aligned_to(dA, e0) || !aligned_to(dB, e0) || !aligned_to(H, 4))
    return refuse(SNACK_ERR_INVALID_ARG, "a pointer is not aligned to its elements");
  const RowsAt dx = {dX, dx_stride, a.in};
  if (overlap({a.X, a.x_stride, a.in}, dx, a.tokens, a.type) || overlap({dY, dy_stride, a.out}, dx, a.tokens, a.type))
    return refuse(SNACK_ERR_INVALID_ARG, "dX overlaps X or dY");
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (a.adapters == 0) return SNACK_OK;
  if (a.tokens == 0 || a.requests == 0) {
    cudaError_t e = cudaSuccess;
    if (dA) e = cudaMemsetAsync(dA, 0, (size_t)(a.adapters * a.rank * a.in * e0), s);
    if (dB && e == cudaSuccess) e = cudaMemsetAsync(dB, 0, (size_t)(a.adapters * a.rank * a.out * e0), s);
    return e == cudaSuccess ? SNACK_OK : cuda_status(e, "adapter gradients");
  }
  AdapterArgs q = {};
  Back b = {};
  q.a = a;
  lay_back(a, &q.p, &b, static_cast<char *>(workspace));
  b.dY = dY;
  b.dy_stride = dy_stride;
  b.H = H;
  b.dX = dX;
  b.dx_stride = dx_stride;
  b.dA = dA;
  b.dB = dB;
  const cudaError_t e = SNACK_TYPES(a.type, backward, q, b, s);
  return e == cudaSuccess ? SNACK_OK : cuda_status(e, "adapter backward launch");
}
