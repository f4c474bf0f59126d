// Attention on mma.sync: every type, head size, stride and length.
//
// A block holds 16 * WM rows of one side in shared memory and streams the
// other side past them in steps of WN * BN rows, copied one step ahead.  Warp
// (wm, wn) multiplies its 16 rows with the BN rows that are its share of a
// step, so that few rows still keep WN warps busy; the WN warps' results meet
// in shared memory at the end.  All products are 16 x 8 blocks of sums in
// registers: the probabilities leave the first product in the layout in which
// the second one takes them and never touch shared memory.
//
// Query rows are packed by key head: row r of a sequence is token r / group,
// query head key_head * group + r % group.  Heads that share keys share their
// copies, and a decode step of a grouped model fills its tile.
//
// 32-bit floats are split in two tf32 parts, x = hi + lo, and hi*hi + hi*lo +
// lo*hi taken (2^-22 of a product is left out); sums over many keys or queries
// are taken out of the matrix unit, which cuts them off instead of rounding,
// after every step.
#pragma once

#include <type_traits>

#include "attention.cuh"

namespace snack {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

__device__ __forceinline__ float tf32_part(float x) {
  return __uint_as_float((__float_as_uint(x) + 0x1000u) & 0xffffe000u);
}

__device__ __forceinline__ void mma_k8(float (&c)[4], const float (&a)[4], float b0, float b1) {
  asm("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(__float_as_uint(a[0])), "r"(__float_as_uint(a[1])), "r"(__float_as_uint(a[2])),
        "r"(__float_as_uint(a[3])), "r"(__float_as_uint(b0)), "r"(__float_as_uint(b1)));
}

template <typename T>
__device__ __forceinline__ void mma_k16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if constexpr (std::is_same<T, __half>::value)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], const void *p) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"((uint32_t)__cvta_generic_to_shared(p)));
}
__device__ __forceinline__ void ldmatrix4_turned(uint32_t (&r)[4], const void *p) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"((uint32_t)__cvta_generic_to_shared(p)));
}

// Products of tiles in shared memory, rows kLd elements apart (8 elements of
// padding keep every access below free of bank conflicts).
template <typename T, int DP>
struct Tile {
  static constexpr int kLd = DP + 8;

  // Which row of the streamed tile column e (0 or 1) of a lane's pair in
  // block nb of 8 belongs to.
  static __device__ __forceinline__ int column(int nb, int lane, int e) { return nb * 8 + 2 * (lane & 3) + e; }

  // acc += rows a (16) times rows b (8 * NB), over DP.
  template <int NB>
  static __device__ __forceinline__ void rows_by_rows(float (&acc)[NB][4], const T *a, const T *b, int lane) {
    const T *pa = a + (lane & 15) * kLd + (lane >> 4) * 8;
    const T *pb = b + ((lane & 7) + ((lane >> 4) & 1) * 8) * kLd + ((lane >> 3) & 1) * 8;
#pragma unroll
    for (int k = 0; k < DP; k += 16) {
      uint32_t fa[4];
      ldmatrix4(fa, pa + k);
#pragma unroll
      for (int n = 0; n < NB; n += 2) {
        uint32_t fb[4];
        ldmatrix4(fb, pb + n * 8 * kLd + k);
        mma_k16<T>(acc[n], fa, fb[0], fb[1]);
        mma_k16<T>(acc[n + 1], fa, fb[2], fb[3]);
      }
    }
  }

  // o (16 x DP) += p (16 x 8 * NB, as the first product left it) times rows b;
  // FINE: p in two parts of the type instead of rounded to it.
  template <int NB, bool FINE = false>
  static __device__ __forceinline__ void sums_by_rows(float (&o)[DP / 8][4], const float (&p)[NB][4], const T *b,
                                                      int lane) {
    uint32_t fa[NB / 2][4], low[FINE ? NB / 2 : 1][4];
#pragma unroll
    for (int k = 0; k < NB / 2; ++k)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float x = p[2 * k + (i >> 1)][(i & 1) * 2], y = p[2 * k + (i >> 1)][(i & 1) * 2 + 1];
        fa[k][i] = pack2<T>(x, y);
        if (FINE) {
          float u, v;
          unpack2<T>(fa[k][i], u, v);
          low[k][i] = pack2<T>(x - u, y - v);
        }
      }
    const T *pb = b + ((lane & 7) + ((lane >> 3) & 1) * 8) * kLd + ((lane >> 4) & 1) * 8;
#pragma unroll
    for (int n = 0; n < DP / 8; n += 2) {
#pragma unroll
      for (int k = 0; k < NB / 2; ++k) {
        uint32_t fb[4];
        ldmatrix4_turned(fb, pb + k * 16 * kLd + n * 8);
        if (FINE) {
          mma_k16<T>(o[n], low[k], fb[0], fb[1]);
          mma_k16<T>(o[n + 1], low[k], fb[2], fb[3]);
        }
        mma_k16<T>(o[n], fa[k], fb[0], fb[1]);
        mma_k16<T>(o[n + 1], fa[k], fb[2], fb[3]);
      }
    }
  }
};

// 32-bit floats.  The order of a summed index is free: a lane's two places of
// an 8-wide step are neighbours in memory.  Block column n is row n ^ (n >> 2)
// of its eight, with which both products read shared memory without conflicts.
template <int DP>
struct Tile<float, DP> {
  static constexpr int kLd = DP + 8;
  static __device__ __forceinline__ int turned(int n) { return n ^ (n >> 2 & 1); }
  static __device__ __forceinline__ int column(int nb, int lane, int e) {
    return nb * 8 + turned(2 * (lane & 3) + e);
  }

  // The small products have sums of their own: those of the large ones are cut
  // off a third as often, and where few blocks of sums would wait for one
  // another (NB <= 2) each product goes its own way.  SPLIT: rows a have their
  // high parts there and their low ones `low` elements further on.
  template <int NB, bool SPLIT = false>
  static __device__ __forceinline__ void rows_by_rows(float (&acc)[NB][4], const float *a, const float *b, int lane,
                                                      int low = 0) {
    const int g = lane >> 2, t = lane & 3;
    const float *pa = a + g * kLd + 2 * t;
    const float *pb = b + turned(g) * kLd + 2 * t;
    constexpr int kOwn = NB <= 2 ? 2 : 1;
    constexpr bool kApart = NB <= 4;
    float cross[kApart ? NB : 1][kOwn][4] = {};
#pragma unroll 4
    for (int k = 0; k < DP; k += 8) {
      float hi[4], lo[4];
      const float2 a0 = *reinterpret_cast<const float2 *>(pa + k);
      const float2 a1 = *reinterpret_cast<const float2 *>(pa + 8 * kLd + k);
      if (SPLIT) {
        const float2 l0 = *reinterpret_cast<const float2 *>(pa + low + k);
        const float2 l1 = *reinterpret_cast<const float2 *>(pa + low + 8 * kLd + k);
        hi[0] = a0.x, hi[1] = a1.x, hi[2] = a0.y, hi[3] = a1.y;
        lo[0] = l0.x, lo[1] = l1.x, lo[2] = l0.y, lo[3] = l1.y;
      } else {
        const float x[4] = {a0.x, a1.x, a0.y, a1.y};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          hi[i] = tf32_part(x[i]);
          lo[i] = tf32_part(x[i] - hi[i]);
        }
      }
#pragma unroll
      for (int n = 0; n < NB; ++n) {
        const float2 y = *reinterpret_cast<const float2 *>(pb + n * 8 * kLd + k);
        const float h0 = tf32_part(y.x), h1 = tf32_part(y.y);
        mma_k8(kApart ? cross[n][0] : acc[n], lo, h0, h1);
        mma_k8(kApart ? cross[n][kOwn - 1] : acc[n], hi, tf32_part(y.x - h0), tf32_part(y.y - h1));
        mma_k8(acc[n], hi, h0, h1);
      }
    }
    if (kApart)
#pragma unroll
      for (int n = 0; n < NB; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[n][i] += kOwn == 2 ? cross[n][0][i] + cross[n][kOwn - 1][i] : cross[n][0][i];
  }

  template <int NB, bool FINE = false>  // (always in two parts)
  static __device__ __forceinline__ void sums_by_rows(float (&o)[DP / 8][4], const float (&p)[NB][4],
                                                      const float *b, int lane) {
    const int g = lane >> 2, t = lane & 3;
    const float *p0 = b + turned(2 * t) * kLd + g;
    const float *p1 = b + turned(2 * t + 1) * kLd + g;
    float hi[NB][4], lo[NB][4];
#pragma unroll
    for (int k = 0; k < NB; ++k) {
      const float x[4] = {p[k][0], p[k][2], p[k][1], p[k][3]};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        hi[k][i] = tf32_part(x[i]);
        lo[k][i] = tf32_part(x[i] - hi[k][i]);
      }
    }
#pragma unroll
    for (int n = 0; n < DP / 8; ++n) {
      float part[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int k = 0; k < NB; ++k) {
        const float y0 = p0[k * 8 * kLd + n * 8], y1 = p1[k * 8 * kLd + n * 8];
        const float h0 = tf32_part(y0), h1 = tf32_part(y1);
        mma_k8(part, lo[k], h0, h1);
        mma_k8(part, hi[k], tf32_part(y0 - h0), tf32_part(y1 - h1));
        mma_k8(part, hi[k], h0, h1);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) o[n][i] += part[i];
    }
  }
};

// Where rows of a side lie: row r is token r / group of the span, head
// r % group further on.  group is 1 for keys and values.
template <typename T>
struct Rows {
  const T *base;
  int64_t token, head;
  int group, d;
  bool vec;  // 16-byte vectors: address and strides are multiples of 16 bytes

  __device__ __forceinline__ Rows(const Strided &s, const Span &sp, bool ragged, int head0, int group_, int d_)
      : token(s.token), head(s.head), group(group_), d(d_) {
    base = static_cast<const T *>(s.p) + (ragged ? sp.row * s.token : sp.seq * s.seq) + head0 * s.head;
    const uintptr_t all = reinterpret_cast<uintptr_t>(base) | (uintptr_t)(s.token * (int64_t)sizeof(T)) |
                          (group_ > 1 ? (uintptr_t)(s.head * (int64_t)sizeof(T)) : 0);
    vec = (all & 15) == 0;
  }
  __device__ __forceinline__ const T *row(int r) const {
    if (group == 1) return base + r * token;
    const int i = r / group;
    return base + i * token + (r - i * group) * head;
  }
};

// Four bytes; `bytes` 0: zeros.
__device__ __forceinline__ void copy_async4(void *slot, const void *from, int bytes) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"((uint32_t)__cvta_generic_to_shared(slot)),
               "l"(from), "r"(bytes)
               : "memory");
}

// Copies `count` rows from r0 on into a tile; rows at or beyond `end` and
// columns beyond the head size become zeros.  Every thread of the block takes
// part; the copies are complete after a commit, a wait and a barrier.
template <typename T, int DP>
__device__ __forceinline__ void copy_rows(T *tile, const Rows<T> &src, int r0, int count, int end) {
  constexpr int kLd = DP + 8, E = 16 / sizeof(T), C = DP / E;
  for (int i = threadIdx.x; i < count * C; i += blockDim.x) {
    const int r = i / C, col = (i - r * C) * E;
    T *to = tile + r * kLd + col;
    const int have = r0 + r < end ? min(E, src.d - col) : 0;
    if (have <= 0) {
      *reinterpret_cast<uint4 *>(to) = make_uint4(0, 0, 0, 0);
      continue;
    }
    const T *from = src.row(r0 + r) + col;
    if (src.vec) {
      copy_async16(to, from, have * (int)sizeof(T));
    } else if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int e = 0; e < E; ++e) copy_async4(to + e, e < have ? from + e : from, e < have ? 4 : 0);
    } else {
#pragma unroll
      for (int e = 0; e < E; ++e) to[e] = e < have ? from[e] : from_float<T>(0.f);
    }
  }
}

template <typename T>
__device__ __forceinline__ void store_pair(T *p, float a, float b, bool pair, bool second) {
  if (pair) {
    if constexpr (sizeof(T) == 4)
      *reinterpret_cast<float2 *>(p) = make_float2(a, b);
    else
      *reinterpret_cast<uint32_t *>(p) = pack2<T>(a, b);
  } else {
    p[0] = from_float<T>(a);
    if (second) p[1] = from_float<T>(b);
  }
}

// Stores a lane's part of a row (its pairs of columns).
template <typename T, int DP>
__device__ __forceinline__ void store_row(T *row, const float (&o)[DP / 8][4], int half, float factor, int d, int lane) {
  const bool pair = (reinterpret_cast<uintptr_t>(row) & (2 * sizeof(T) - 1)) == 0;
#pragma unroll
  for (int n = 0; n < DP / 8; ++n) {
    const int col = n * 8 + 2 * (lane & 3);
    if (col < d)
      store_pair<T>(row + col, o[n][2 * half] * factor, o[n][2 * half + 1] * factor, pair && col + 1 < d, col + 1 < d);
  }
}

// A warp's 16 x DP sums into shared memory, and the WN warps' sums together
// (in their order) back into the first one's registers.
template <int DP, int WM, int WN>
__device__ __forceinline__ void add_shares(float (&o)[DP / 8][4], float *room, int wm, int wn, int lane) {
  constexpr int kRow = DP + 8;
  const int g = lane >> 2, col = 2 * (lane & 3);
  __syncthreads();
  if (wn > 0) {
    float *p = room + ((wn - 1) * WM + wm) * 16 * kRow + g * kRow + col;
#pragma unroll
    for (int n = 0; n < DP / 8; ++n) {
      *reinterpret_cast<float2 *>(p + n * 8) = make_float2(o[n][0], o[n][1]);
      *reinterpret_cast<float2 *>(p + 8 * kRow + n * 8) = make_float2(o[n][2], o[n][3]);
    }
  }
  __syncthreads();
  if (wn == 0) {
#pragma unroll
    for (int w = 0; w < WN - 1; ++w) {
      const float *p = room + (w * WM + wm) * 16 * kRow + g * kRow + col;
#pragma unroll
      for (int n = 0; n < DP / 8; ++n) {
        const float2 a = *reinterpret_cast<const float2 *>(p + n * 8);
        const float2 b = *reinterpret_cast<const float2 *>(p + 8 * kRow + n * 8);
        o[n][0] += a.x;
        o[n][1] += a.y;
        o[n][2] += b.x;
        o[n][3] += b.y;
      }
    }
  }
}

// ------------------------------------------------------------------ forward

// The last step of 16 rows: the sums times 1 / l, and the log of the sum.  One warp.
template <typename T, int DP>
__device__ __forceinline__ void finish_rows(const AttnCall &c, const Span &qs, const float (&o)[DP / 8][4],
                                            const float (&m)[2], const float (&l)[2], const int (&token)[2],
                                            const int (&head)[2], int lane) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    if (token[h] >= qs.cover) continue;
    const float inv = l[h] == 0.f ? 0.f : c.keep_scale / l[h];
    const float lse = l[h] == 0.f ? -INFINITY : (m[h] + log2f(l[h])) * kLn2;
    const int64_t row = qs.row + token[h];
    T *out = static_cast<T *>(c.out.p) +
             (c.q_offsets ? row * c.out.token : qs.seq * c.out.seq + token[h] * c.out.token) + head[h] * c.out.head;
    store_row<T, DP>(out, o, h, inv, c.d, lane);
    if ((lane & 3) == 0) c.lse[(int64_t)head[h] * c.rows + row] = lse;
  }
}

template <typename T, int DP, int WM, int BN>
constexpr size_t rows_forward_smem() {
  return (size_t)(16 * WM + 2 * 2 * BN) * (DP + 8) * sizeof(T);
}

// Softmax with a running maximum and sum.  Grid: tile * key_heads + key head.
template <typename T, int DP, int WM, int BN>
__global__ void __launch_bounds__(32 * WM) rows_forward(const AttnCall c) {
  using Ops = Tile<T, DP>;
  constexpr int kLd = Ops::kLd, NB = BN / 8;
  extern __shared__ __align__(16) unsigned char smem[];
  T *sq = reinterpret_cast<T *>(smem);
  T *skv = sq + 16 * WM * kLd;  // [2 stages][K, V][BN]

  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int kh = blockIdx.x % c.key_heads, G = c.group;
  const Place at = find_tile(c.q_offsets, c.sequences, c.q_tokens, G, 16 * WM, blockIdx.x / c.key_heads, c.causal);
  if (at.s < 0) return;
  const Span qs = own_span(c.q_offsets, c.q_lengths, at.s, c.sequences, c.q_tokens);
  const Span ks = other_span(c.k_offsets, c.k_lengths, at.s, c.q_offsets != nullptr, c.sequences, c.k_tokens);
  const int r0 = at.tile * 16 * WM, nq = qs.valid, nk = ks.valid;
  const int last = min((r0 + 16 * WM - 1) / G, nq - 1);
  const int end = r0 / G < nq ? max(0, seen_keys(c.causal, last, nq, nk)) : 0;

  const Rows<T> qr(c.q, qs, c.q_offsets != nullptr, kh * G, G, c.d);
  const Rows<T> kr(c.k, ks, c.k_offsets != nullptr, kh, 1, c.d), vr(c.v, ks, c.k_offsets != nullptr, kh, 1, c.d);

  // the two rows of this lane
  int token[2], head[2], lim[2];
  uint64_t draw[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int r = r0 + warp * 16 + (lane >> 2) + 8 * h;
    token[h] = r / G;
    head[h] = kh * G + r % G;
    lim[h] = token[h] < nq ? min(end, seen_keys(c.causal, token[h], nq, nk)) : 0;
    if (c.drop) draw[h] = dropout_row(c.draws(), qs.row + token[h], c.heads, head[h]);
  }

  float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f}, o[DP / 8][4] = {};
  const auto copy_step = [&](int stage, int key0) {
    T *k = skv + stage * 2 * BN * kLd;
    copy_rows<T, DP>(k, kr, key0, BN, end);
    copy_rows<T, DP>(k + BN * kLd, vr, key0, BN, end);
  };
  if (end > 0) {
    copy_rows<T, DP>(sq, qr, r0, 16 * WM, nq * G);
    copy_step(0, 0);
  }
  copies_commit();
  for (int key = 0, stage = 0; key < end; key += BN, stage ^= 1) {
    if (key + BN < end) copy_step(stage ^ 1, key + BN);
    copies_commit();
    copies_wait<1>();
    __syncthreads();
    const T *k = skv + stage * 2 * BN * kLd, *v = k + BN * kLd;
    float s[NB][4] = {};
    Ops::template rows_by_rows<NB>(s, sq + warp * 16 * kLd, k, lane);
    float top[2] = {m[0], m[1]};
#pragma unroll
    for (int n = 0; n < NB; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int h = e >> 1;
        s[n][e] = key + Ops::column(n, lane, e & 1) < lim[h] ? s[n][e] * c.scale_log2 : -INFINITY;
        top[h] = fmaxf(top[h], s[n][e]);
      }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      top[h] = fmaxf(top[h], __shfl_xor_sync(0xffffffffu, top[h], 1));
      top[h] = fmaxf(top[h], __shfl_xor_sync(0xffffffffu, top[h], 2));
      const float from = top[h] == -INFINITY ? 0.f : top[h];
      const float shrink = exp2f(m[h] - from);
      m[h] = top[h];
      l[h] *= shrink;
#pragma unroll
      for (int n = 0; n < DP / 8; ++n) {
        o[n][2 * h] *= shrink;
        o[n][2 * h + 1] *= shrink;
      }
      float sum = 0.f;
#pragma unroll
      for (int n = 0; n < NB; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          s[n][2 * h + e] = exp2f(s[n][2 * h + e] - from);
          sum += s[n][2 * h + e];
        }
      l[h] += sum;
      if (c.drop) {
#pragma unroll
        for (int n = 0; n < NB; ++n) {
          const int j = key + Ops::column(n, lane, 0);
          const uint64_t z = dropout_draw(draw[h], j);
          if (draw_lane(z, j & 3) < c.drop) s[n][2 * h] = 0.f;
          if (draw_lane(z, (key + Ops::column(n, lane, 1)) & 3) < c.drop) s[n][2 * h + 1] = 0.f;
        }
      }
    }
    Ops::template sums_by_rows<NB>(o, s, v, lane);
    __syncthreads();
  }
  copies_wait<0>();
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    l[h] += __shfl_xor_sync(0xffffffffu, l[h], 1);
    l[h] += __shfl_xor_sync(0xffffffffu, l[h], 2);
  }
  finish_rows<T, DP>(c, qs, o, m, l, token, head, lane);
}

// ------------------------------------------------------------------ backward

// With P of the forward call's lse made again,
//   dP = M * (dout . v),  dS = P * (dP - delta),  dq = scale * dS k,
//   dk = scale * dS^T q,  dv = (M * P)^T dout.
// A row that sees one key has P = 1 whatever the score: dS is zero, not what two
// roundings of the same product differ by.
// dS is taken in two parts of the type: rounded to it, it made dq and dk 1.6
// times as far off as the rounding of the results alone.

// float16: brings a step's dS of a lane's two rows into range and the sums so far to
// the same power.  The four lanes of a row agree.
template <typename T, int DP, int NB>
__device__ __forceinline__ void scale_rows(float (&t)[NB][4], float (&sums)[DP / 8][4], int (&power)[2]) {
  if constexpr (std::is_same<T, __half>::value) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float top = 0.f;
#pragma unroll
      for (int n = 0; n < NB; ++n) top = fmaxf(top, fmaxf(fabsf(t[n][2 * h]), fabsf(t[n][2 * h + 1])));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
      const int now = running_power(power[h], exponent_bits(top));
      if (now != power[h]) {
        const float by = exp2f((float)(now - power[h]));
#pragma unroll
        for (int n = 0; n < DP / 8; ++n) {
          sums[n][2 * h] *= by;
          sums[n][2 * h + 1] *= by;
        }
        power[h] = now;
      }
      const float up = power_of_two(now);
#pragma unroll
      for (int n = 0; n < NB; ++n) {
        t[n][2 * h] *= up;
        t[n][2 * h + 1] *= up;
      }
    }
  }
}
// Takes those powers out again.
template <typename T, int DP>
__device__ __forceinline__ void unscale_rows(float (&sums)[DP / 8][4], const int (&power)[2]) {
  if constexpr (std::is_same<T, __half>::value) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const float by = power_of_two(-power[h]);
#pragma unroll
      for (int n = 0; n < DP / 8; ++n) {
        sums[n][2 * h] *= by;
        sums[n][2 * h + 1] *= by;
      }
    }
  }
}

template <typename T, int DP, int WM, int WN, int BQ, int ST>
constexpr size_t rows_backward_smem() {
  const size_t tiles = (size_t)(2 * 16 * WM + ST * 2 * WN * BQ) * (DP + 8) * sizeof(T);
  const size_t room = (size_t)(WN - 1) * WM * 16 * (DP + 8) * sizeof(float);
  return tiles > room ? tiles : room;
}

// Gradients of 16 * WM keys and values: the query rows that see them stream past.
template <typename T, int DP, int WM, int WN, int BQ, int ST>
__device__ __forceinline__ void keys_of_rows(const AttnCall &c, int block) {
  using Ops = Tile<T, DP>;
  constexpr int kLd = Ops::kLd, NB = BQ / 8, STEP = WN * BQ;
  extern __shared__ __align__(16) unsigned char smem[];
  T *sk = reinterpret_cast<T *>(smem), *sv = sk + 16 * WM * kLd, *sqd = sv + 16 * WM * kLd;
  __shared__ float s_lse[ST][STEP], s_delta[ST][STEP];
  __shared__ int s_lim[ST][STEP];
  __shared__ uint64_t s_draw[ST][STEP];

  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, wm = warp / WN, wn = warp % WN;
  const int kh = block % c.key_heads, G = c.group;
  const Place at = find_tile(c.k_offsets, c.sequences, c.k_tokens, 1, 16 * WM, block / c.key_heads, false);
  if (at.s < 0) return;
  const Span ks = own_span(c.k_offsets, c.k_lengths, at.s, c.sequences, c.k_tokens);
  const Span qs = other_span(c.q_offsets, c.q_lengths, at.s, c.k_offsets != nullptr, c.sequences, c.q_tokens);
  const int j0 = at.tile * 16 * WM, nq = qs.valid, nk = ks.valid;
  const int row_begin = first_query(c.causal, j0, nq, nk) * G, end = nq * G;  // rows; none see padding

  const Rows<T> kr(c.k, ks, c.k_offsets != nullptr, kh, 1, c.d), vr(c.v, ks, c.k_offsets != nullptr, kh, 1, c.d);
  const Rows<T> qr(c.q, qs, c.q_offsets != nullptr, kh * G, G, c.d);
  const Rows<T> dr(c.dout, qs, c.q_offsets != nullptr, kh * G, G, c.d);
  const uint64_t seed = c.drop ? c.draws() : 0;
  const float p_up = std::is_same<T, __half>::value ? kHalfP : 0.f, p_down = exp2f(-p_up);

  float dk[DP / 8][4] = {}, dv[DP / 8][4] = {};
  int power[2] = {kMostPower, kMostPower};
  const auto copy_step = [&](int stage, int row0) {
    T *q = sqd + stage * 2 * STEP * kLd;
    copy_rows<T, DP>(q, qr, row0, STEP, end);
    copy_rows<T, DP>(q + STEP * kLd, dr, row0, STEP, end);
  };
  // a thread's row of the next step: loaded before a step is computed, stored after it
  static_assert(STEP <= 32 * WM * WN, "a thread for each row of a step");
  float next_lse = 0.f, next_delta = 0.f;
  int next_lim = 0;
  uint64_t next_draw = 0;
  const auto load_row = [&](int row0) {
    if (threadIdx.x >= STEP) return;
    const int r = row0 + threadIdx.x, token = r / G, head = kh * G + (r - token * G);
    next_lse = INFINITY;
    next_delta = 0.f;
    next_lim = 0;
    if (r < end) {
      const int64_t place = (int64_t)head * c.rows + qs.row + token;
      next_lse = c.lse[place];
      next_delta = c.delta[place];
      next_lim = seen_keys(c.causal, token, nq, nk);
    }
    if (c.drop) next_draw = dropout_row(seed, qs.row + token, c.heads, head);
  };
  const auto store_row_stats = [&](int stage) {
    if (threadIdx.x >= STEP) return;
    s_lse[stage][threadIdx.x] = next_lse * kLog2e - p_up;
    s_delta[stage][threadIdx.x] = next_delta;
    s_lim[stage][threadIdx.x] = next_lse == -INFINITY ? 0 : next_lim;
    if (c.drop) s_draw[stage][threadIdx.x] = next_draw;
  };
  if (row_begin < end) {
    copy_rows<T, DP>(sk, kr, j0, 16 * WM, nk);
    copy_rows<T, DP>(sv, vr, j0, 16 * WM, nk);
    copy_step(0, row_begin);
    load_row(row_begin);
    store_row_stats(0);
  }
  copies_commit();
  for (int row0 = row_begin, stage = 0; row0 < end; row0 += STEP, stage ^= ST - 1) {
    const bool more = row0 + STEP < end;
    if (more) {
      if (ST == 2) copy_step(stage ^ 1, row0 + STEP);
      load_row(row0 + STEP);
    }
    if (ST == 2) copies_commit();
    copies_wait<ST - 1>();
    __syncthreads();
    const T *q = sqd + (stage * 2 * STEP + wn * BQ) * kLd, *d = q + STEP * kLd;
    if (row0 + wn * BQ < end) {
      float p[NB][4] = {}, t[NB][4] = {};
      Ops::template rows_by_rows<NB>(p, sk + wm * 16 * kLd, q, lane);
      Ops::template rows_by_rows<NB>(t, sv + wm * 16 * kLd, d, lane);
#pragma unroll
      for (int n = 0; n < NB; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int i = wn * BQ + Ops::column(n, lane, e);
          const float lse = s_lse[stage][i], delta = s_delta[stage][i];
          const int lim = s_lim[stage][i];
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int j = j0 + wm * 16 + (lane >> 2) + 8 * h, x = 2 * h + e;
            const bool seen = j < lim;
            const float prob = seen ? exp2f(p[n][x] * c.scale_log2 - lse) : 0.f;
            float mult = 1.f;
            if (c.drop)
              mult = draw_lane(dropout_draw(s_draw[stage][i], j), j & 3) >= c.drop ? c.keep_scale : 0.f;
            t[n][x] = seen && lim > 1 ? prob * ((t[n][x] * mult - delta) * p_down) : 0.f;
            p[n][x] = mult != 0.f ? prob : 0.f;
          }
        }
      scale_rows<T, DP>(t, dk, power);
      Ops::template sums_by_rows<NB>(dv, p, d, lane);
      Ops::template sums_by_rows<NB, true>(dk, t, q, lane);
    }
    if (ST == 2 && more) store_row_stats(stage ^ 1);
    __syncthreads();
    if (ST == 1 && more) {
      copy_step(0, row0 + STEP);
      store_row_stats(0);
      copies_commit();
    }
  }
  copies_wait<0>();
  unscale_rows<T, DP>(dk, power);
  if constexpr (WN > 1) {
    add_shares<DP, WM, WN>(dv, reinterpret_cast<float *>(smem), wm, wn, lane);
    add_shares<DP, WM, WN>(dk, reinterpret_cast<float *>(smem), wm, wn, lane);
    if (wn != 0) return;
  }
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int j = j0 + wm * 16 + (lane >> 2) + 8 * h;
    if (j >= ks.cover) continue;
    const auto row = [&](const Strided &s) {
      return static_cast<T *>(s.p) + (c.k_offsets ? (ks.row + j) * s.token : ks.seq * s.seq + j * s.token) + kh * s.head;
    };
    if (c.dk.p) store_row<T, DP>(row(c.dk), dk, h, c.scale, c.d, lane);
    if (c.dv.p) store_row<T, DP>(row(c.dv), dv, h, p_down * c.keep_scale, c.d, lane);
  }
}

// Gradients of 16 * WM query rows: the keys and values that they see stream past.
template <typename T, int DP, int WM, int WN, int BN, int ST>
__device__ __forceinline__ void queries_of_rows(const AttnCall &c, int block) {
  using Ops = Tile<T, DP>;
  constexpr int kLd = Ops::kLd, NB = BN / 8, STEP = WN * BN;
  extern __shared__ __align__(16) unsigned char smem[];
  T *sq = reinterpret_cast<T *>(smem), *sd = sq + 16 * WM * kLd, *skv = sd + 16 * WM * kLd;

  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, wm = warp / WN, wn = warp % WN;
  const int kh = block % c.key_heads, G = c.group;
  const Place at = find_tile(c.q_offsets, c.sequences, c.q_tokens, G, 16 * WM, block / c.key_heads, c.causal);
  if (at.s < 0) return;
  const Span qs = own_span(c.q_offsets, c.q_lengths, at.s, c.sequences, c.q_tokens);
  const Span ks = other_span(c.k_offsets, c.k_lengths, at.s, c.q_offsets != nullptr, c.sequences, c.k_tokens);
  const int r0 = at.tile * 16 * WM, nq = qs.valid, nk = ks.valid;
  const int last = min((r0 + 16 * WM - 1) / G, nq - 1);
  const int end = last >= 0 && r0 / G < nq ? max(0, seen_keys(c.causal, last, nq, nk)) : 0;

  const Rows<T> qr(c.q, qs, c.q_offsets != nullptr, kh * G, G, c.d);
  const Rows<T> dr(c.dout, qs, c.q_offsets != nullptr, kh * G, G, c.d);
  const Rows<T> kr(c.k, ks, c.k_offsets != nullptr, kh, 1, c.d), vr(c.v, ks, c.k_offsets != nullptr, kh, 1, c.d);

  int token[2], head[2], lim[2];
  float lse[2], delta[2];
  uint64_t draw[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int r = r0 + wm * 16 + (lane >> 2) + 8 * h;
    token[h] = r / G;
    head[h] = kh * G + r % G;
    lim[h] = 0;
    lse[h] = INFINITY;
    delta[h] = 0.f;
    if (token[h] < nq) {
      const int64_t place = (int64_t)head[h] * c.rows + qs.row + token[h];
      lse[h] = c.lse[place] * kLog2e;
      delta[h] = c.delta[place];
      lim[h] = lse[h] == -INFINITY ? 0 : seen_keys(c.causal, token[h], nq, nk);
    }
    if (c.drop) draw[h] = dropout_row(c.draws(), qs.row + token[h], c.heads, head[h]);
  }

  float dq[DP / 8][4] = {};
  int power[2] = {kMostPower, kMostPower};
  const auto copy_step = [&](int stage, int key0) {
    T *k = skv + stage * 2 * STEP * kLd;
    copy_rows<T, DP>(k, kr, key0, STEP, end);
    copy_rows<T, DP>(k + STEP * kLd, vr, key0, STEP, end);
  };
  if (end > 0) {
    copy_rows<T, DP>(sq, qr, r0, 16 * WM, nq * G);
    copy_rows<T, DP>(sd, dr, r0, 16 * WM, nq * G);
    copy_step(0, 0);
  }
  copies_commit();
  for (int key0 = 0, stage = 0; key0 < end; key0 += STEP, stage ^= ST - 1) {
    if (ST == 2) {
      if (key0 + STEP < end) copy_step(stage ^ 1, key0 + STEP);
      copies_commit();
    }
    copies_wait<ST - 1>();
    __syncthreads();
    const T *k = skv + (stage * 2 * STEP + wn * BN) * kLd, *v = k + STEP * kLd;
    const int key = key0 + wn * BN;
    if (key < end) {
      float p[NB][4] = {}, t[NB][4] = {};
      Ops::template rows_by_rows<NB>(p, sq + wm * 16 * kLd, k, lane);
      Ops::template rows_by_rows<NB>(t, sd + wm * 16 * kLd, v, lane);
#pragma unroll
      for (int n = 0; n < NB; ++n)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int j = key + Ops::column(n, lane, 0);
          const uint64_t z = c.drop ? dropout_draw(draw[h], j) : 0;
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int je = key + Ops::column(n, lane, e), x = 2 * h + e;
            const float mult = !c.drop ? 1.f : (draw_lane(z, je & 3) >= c.drop ? c.keep_scale : 0.f);
            t[n][x] = je < lim[h] && lim[h] > 1
                          ? exp2f(p[n][x] * c.scale_log2 - lse[h]) * (t[n][x] * mult - delta[h]) : 0.f;
          }
        }
      scale_rows<T, DP>(t, dq, power);
      Ops::template sums_by_rows<NB, true>(dq, t, k, lane);
    }
    __syncthreads();
    if (ST == 1 && key0 + STEP < end) {
      copy_step(0, key0 + STEP);
      copies_commit();
    }
  }
  copies_wait<0>();
  unscale_rows<T, DP>(dq, power);
  if constexpr (WN > 1) {
    add_shares<DP, WM, WN>(dq, reinterpret_cast<float *>(smem), wm, wn, lane);
    if (wn != 0) return;
  }
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    if (token[h] >= qs.cover) continue;
    T *row = static_cast<T *>(c.dq.p) +
             (c.q_offsets ? (qs.row + token[h]) * c.dq.token : qs.seq * c.dq.seq + token[h] * c.dq.token) +
             head[h] * c.dq.head;
    store_row<T, DP>(row, dq, h, c.scale, c.d, lane);
  }
}

// The first `key_blocks` blocks take keys, the others queries.  ONLY: the
// kernel has code for one of them (1: keys, 2: queries) and that one's registers.
template <typename T, int DP, int WM, int WN, int BN, int ST, int ONLY>
__global__ void __launch_bounds__(32 * WM * WN, DP == 64 && ONLY == 2 ? 2 : 1) rows_backward(const AttnCall c, int key_blocks) {
  if (ONLY == 1 || (ONLY == 0 && (int)blockIdx.x < key_blocks))
    keys_of_rows<T, DP, WM, WN, BN, ST>(c, blockIdx.x);
  else
    queries_of_rows<T, DP, WM, WN, BN, ST>(c, blockIdx.x - key_blocks);
}

}  // namespace snack
