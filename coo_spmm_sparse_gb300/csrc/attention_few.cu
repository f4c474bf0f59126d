// The forward call of few query rows (decode steps, short prompts): 16 rows to
// a block, whose warps take the keys in turn, each on its own.
//
// The caches' bytes are the work.  A warp copies its next tiles (16 keys and
// their values; 8 in 32 bits at head sizes above 64) with 16-byte asynchronous
// copies whose addresses advance by constants, and waits for its own copies
// only: no barrier of the block until the end.  (Copies whose rows and columns
// were computed for each vector took most of the instructions and held the
// kernel at 2.4 TB/s; one bulk copy a row reached 4.3.)  Long caches are cut
// into chunks for more blocks, joined by join_splits.
#include "attention_rows.cuh"

namespace snack {
namespace {

// Four warps, three tiles each (two in 32 bits: two blocks to an SM); sixteen warps with one tile each where there are
// few blocks, so that short caches take one step.
template <typename T, int DP, int W>
struct Few {
  static constexpr int kKeys = sizeof(T) == 4 && DP > 64 ? 8 : 16;  // of a warp's tile
  static constexpr int kStages = W != 4 ? 1 : sizeof(T) == 4 ? 2 : 3, kStep = W * kKeys, kLd = DP + 8;
  static constexpr int kTileElems = 2 * kKeys * kLd;
  static constexpr size_t ring = (size_t)W * kStages * kTileElems * sizeof(T);
  static constexpr size_t room = (size_t)W * 16 * kLd * sizeof(float);
  static constexpr int kQueries = (sizeof(T) == 4 ? 2 : 1) * 16 * kLd;  // 32 bits: high and low parts
  static constexpr size_t smem = kQueries * sizeof(T) + (ring > room ? ring : room);
};

template <typename T, int DP, int W>
__global__ void __launch_bounds__(32 * W) few_forward(const AttnCall c) {
  using Ops = Tile<T, DP>;
  using F = Few<T, DP, W>;
  constexpr int kLd = F::kLd, kKeys = F::kKeys, NB = kKeys / 8, kStages = F::kStages;
  constexpr int E = 16 / sizeof(T), kChunks = DP / E, kRows = 32 / kChunks;  // rows that a warp copies at once
  extern __shared__ __align__(16) unsigned char smem[];
  __shared__ float stat[2][W][16];
  T *const sq = reinterpret_cast<T *>(smem);

  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int kh = blockIdx.x % c.key_heads, G = c.group;
  const Place at = find_tile(c.q_offsets, c.sequences, c.q_tokens, G, 16, blockIdx.x / c.key_heads, c.causal);
  if (at.s < 0) return;
  const Span qs = own_span(c.q_offsets, c.q_lengths, at.s, c.sequences, c.q_tokens);
  const Span ks = other_span(c.k_offsets, c.k_lengths, at.s, c.q_offsets != nullptr, c.sequences, c.k_tokens);
  const int r0 = at.tile * 16, nq = qs.valid, nk = ks.valid;
  const int last = min((r0 + 15) / G, nq - 1);
  const int begin = blockIdx.y * c.chunk;
  int end = r0 / G < nq ? max(0, seen_keys(c.causal, last, nq, nk)) : 0;
  if (c.splits > 1) end = begin + min(end - begin, c.chunk);  // (begin + chunk may pass 31 bits)

  T *const ring = sq + F::kQueries + warp * kStages * F::kTileElems;
  const Rows<T> kr(c.k, ks, c.k_offsets != nullptr, kh, 1, c.d), vr(c.v, ks, c.k_offsets != nullptr, kh, 1, c.d);
  const bool vec = kr.vec && vr.vec;
  const int first = begin + warp * kKeys;
  const int steps = first < end ? (end - first + F::kStep - 1) / F::kStep : 0;
  const int my_row = lane / kChunks, my_col = lane % kChunks * E;
  const int bytes = max(0, min(E, c.d - my_col)) * (int)sizeof(T);  // what lies behind the head size becomes zero
  // Rows behind the last key become zeros too: values that meet zero probabilities have to be numbers.
  const auto copy_tile = [&](int step) {
    const int key0 = first + step * F::kStep;
    T *const k = ring + step % kStages * F::kTileElems;
    if (vec) {
      T *const to = k + my_row * kLd + my_col;
      const T *const pk = kr.base + (int64_t)(key0 + my_row) * kr.token + my_col;
      const T *const pv = vr.base + (int64_t)(key0 + my_row) * vr.token + my_col;
#pragma unroll
      for (int i = 0; i < kKeys; i += kRows) {
        const int n = key0 + my_row + i < end ? bytes : 0;
        copy_async16(to + i * kLd, n ? pk + i * kr.token : kr.base, n);
        copy_async16(to + (kKeys + i) * kLd, n ? pv + i * vr.token : vr.base, n);
      }
    } else {
      for (int r = 0; r < kKeys; ++r)
#pragma unroll
        for (int col = lane; col < DP; col += 32) {
          const bool have = key0 + r < end && col < c.d;
          const int64_t row = have ? key0 + r : 0;
          const T *const fk = have ? kr.base + row * kr.token + col : kr.base;
          const T *const fv = have ? vr.base + row * vr.token + col : vr.base;
          if constexpr (sizeof(T) == 4) {
            copy_async4(k + r * kLd + col, fk, have ? 4 : 0);
            copy_async4(k + (kKeys + r) * kLd + col, fv, have ? 4 : 0);
          } else {
            k[r * kLd + col] = have ? *fk : from_float<T>(0.f);
            k[(kKeys + r) * kLd + col] = have ? *fv : from_float<T>(0.f);
          }
        }
    }
  };
  // the keys are on their way before the queries are waited for
  constexpr int kAhead = kStages > 1 ? kStages - 1 : 1;
  if (begin < end) {
    const Rows<T> qr(c.q, qs, c.q_offsets != nullptr, kh * G, G, c.d);
    copy_rows<T, DP>(sq, qr, r0, 16, nq * G);
  }
  copies_commit();
#pragma unroll
  for (int i = 0; i < kAhead; ++i) {
    if (i < steps) copy_tile(i);
    copies_commit();
  }

  // the two rows of this lane; the second eight hold nothing where there are no more rows
  const int rows = min(16, nq * G - r0);
  int token[2], head[2], lim[2];
  uint64_t draw[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int r = r0 + (lane >> 2) + 8 * h;
    token[h] = r / G;
    head[h] = kh * G + r % G;
    lim[h] = token[h] < nq ? min(end, seen_keys(c.causal, token[h], nq, nk)) : 0;
    if (c.drop) draw[h] = dropout_row(c.draws(), qs.row + token[h], c.heads, head[h]);
  }

  float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f}, o[DP / 8][4] = {};
  copies_wait<kAhead>();
  __syncthreads();
  constexpr bool kParts = sizeof(T) == 4;
  if constexpr (kParts) {  // the queries' parts are made once, not for every tile of keys
    for (int i = threadIdx.x; i < 16 * kLd; i += 32 * W) {
      const float x = sq[i], hi = tf32_part(x);
      sq[i] = hi;
      sq[16 * kLd + i] = tf32_part(x - hi);
    }
    __syncthreads();
  }
  for (int step = 0; step < steps; ++step) {
    const int key = first + step * F::kStep;
    if (kStages > 1) {
      if (step + kAhead < steps) copy_tile(step + kAhead);
      copies_commit();
    }
    copies_wait<kStages - 1>();
    __syncwarp();
    const T *const k = ring + step % kStages * F::kTileElems, *const v = k + kKeys * kLd;
    float s[NB][4] = {};
    if constexpr (kParts)
      Ops::template rows_by_rows<NB, true>(s, sq, k, lane, 16 * kLd);
    else
      Ops::template rows_by_rows<NB>(s, sq, k, lane);
    float shrink[2] = {1.f, 1.f};
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      if (h == 1 && rows <= 8) {
#pragma unroll
        for (int n = 0; n < NB; ++n) s[n][2] = s[n][3] = 0.f;
        continue;
      }
      float top = m[h];
#pragma unroll
      for (int n = 0; n < NB; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float &x = s[n][2 * h + e];
          x = key + Ops::column(n, lane, e) < lim[h] ? x * c.scale_log2 : -INFINITY;
          top = fmaxf(top, x);
        }
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
      const float from = top == -INFINITY ? 0.f : top;
      shrink[h] = exp2f(m[h] - from);
      m[h] = top;
      float sum = 0.f;
#pragma unroll
      for (int n = 0; n < NB; ++n) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          s[n][2 * h + e] = exp2f(s[n][2 * h + e] - from);
          sum += s[n][2 * h + e];
        }
        if (c.drop) {
          const int j = key + Ops::column(n, lane, 0);
          const uint64_t z = dropout_draw(draw[h], j);
          if (draw_lane(z, j & 3) < c.drop) s[n][2 * h] = 0.f;
          if (draw_lane(z, (key + Ops::column(n, lane, 1)) & 3) < c.drop) s[n][2 * h + 1] = 0.f;
        }
      }
      l[h] = l[h] * shrink[h] + sum;
    }
    if (__any_sync(0xffffffffu, shrink[0] != 1.f || shrink[1] != 1.f)) {
#pragma unroll
      for (int n = 0; n < DP / 8; ++n) {
        o[n][0] *= shrink[0];
        o[n][1] *= shrink[0];
        o[n][2] *= shrink[1];
        o[n][3] *= shrink[1];
      }
    }
    Ops::template sums_by_rows<NB>(o, s, v, lane);
    __syncwarp();
    if (kStages == 1 && step + 1 < steps) {
      copy_tile(step + 1);
      copies_commit();
    }
  }
  copies_wait<0>();
  dependency_launch();
  const int row = lane >> 2;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    l[h] += __shfl_xor_sync(0xffffffffu, l[h], 1);
    l[h] += __shfl_xor_sync(0xffffffffu, l[h], 2);
    if ((lane & 3) == 0) {
      stat[0][warp][row + 8 * h] = m[h];
      stat[1][warp][row + 8 * h] = l[h];
    }
  }
  __syncthreads();  // (and the tiles are read: their memory takes the warps' sums)
  float *const room = reinterpret_cast<float *>(sq + F::kQueries);
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    if (row + 8 * h >= rows) continue;
    float top = -INFINITY;
#pragma unroll
    for (int w = 0; w < W; ++w) top = fmaxf(top, stat[0][w][row + 8 * h]);
    const float shrink = exp2f(m[h] - (top == -INFINITY ? 0.f : top));
    float *const to = room + (warp * 16 + row + 8 * h) * kLd + 2 * (lane & 3);
#pragma unroll
    for (int n = 0; n < DP / 8; ++n)
      *reinterpret_cast<float2 *>(to + n * 8) = make_float2(o[n][2 * h] * shrink, o[n][2 * h + 1] * shrink);
  }
  __syncthreads();
  // a warp takes a row, a lane its columns: the warps' sums in their order
  for (int r = warp; r < 16; r += W) {
    const int i = (r0 + r) / G, hd = kh * G + (r0 + r) % G;
    if (i >= qs.cover) break;
    float top = -INFINITY, sum = 0.f, sums[DP / 32] = {};
    if (r < rows) {
#pragma unroll
      for (int w = 0; w < W; ++w) top = fmaxf(top, stat[0][w][r]);
      const float from = top == -INFINITY ? 0.f : top;
#pragma unroll
      for (int w = 0; w < W; ++w) {
        sum += stat[1][w][r] * exp2f(stat[0][w][r] - from);
#pragma unroll
        for (int x = 0; x < DP / 32; ++x) sums[x] += room[(w * 16 + r) * kLd + lane + 32 * x];
      }
    }
    const float by = sum == 0.f ? 0.f : c.keep_scale / sum;
    const float lse = sum == 0.f ? -INFINITY : (top + log2f(sum)) * kLn2;
    const int64_t token_row = qs.row + i, slot = (blockIdx.y * c.rows + token_row) * c.heads + hd;
    T *const out = static_cast<T *>(c.out.p) +
                   (c.q_offsets ? token_row * c.out.token : qs.seq * c.out.seq + i * c.out.token) + hd * c.out.head;
#pragma unroll
    for (int x = 0; x < DP / 32; ++x) {
      const int col = lane + 32 * x;
      if (col >= c.d) break;
      if (c.splits > 1)
        c.part[slot * c.d + col] = sum == 0.f ? 0.f : sums[x] * by;
      else
        out[col] = from_float<T>(sum == 0.f ? 0.f : sums[x] * by);
    }
    if (lane == 0) {
      if (c.splits > 1)
        c.part[(int64_t)c.splits * c.rows * c.heads * c.d + slot] = lse;
      else
        c.lse[(int64_t)hd * c.rows + token_row] = lse;
    }
  }
}

template <typename T, int DP, int W>
cudaError_t few_sized(const AttnCall &c, int64_t blocks, cudaStream_t s) {
  const auto kern = few_forward<T, DP, W>;
  const cudaError_t e = allow_smem(kern, Few<T, DP, W>::smem);
  if (e != cudaSuccess) return e;
  return launch_kernel(kern, dim3((unsigned)blocks, (unsigned)c.splits), 32 * W, Few<T, DP, W>::smem, false, s, c);
}

template <typename T, int DP>
cudaError_t few_warps(const AttnCall &c, cudaStream_t s) {
  const int64_t blocks = tiles_of(c.q_offsets != nullptr, c.sequences, c.q_tokens, c.group, 16) * c.key_heads;
  if (blocks * c.splits <= device_sms()) return few_sized<T, DP, 16>(c, blocks, s);
  return few_sized<T, DP, 4>(c, blocks, s);
}

template <typename T>
cudaError_t few_typed(const AttnCall &c, cudaStream_t s) {
  return c.d <= 64 ? few_warps<T, 64>(c, s) : few_warps<T, 128>(c, s);
}

}  // namespace

cudaError_t few_forward_launch(const AttnCall &c, int type, cudaStream_t s) {
  return type == SNACK_F32    ? few_typed<float>(c, s)
         : type == SNACK_BF16 ? few_typed<__nv_bfloat16>(c, s)
                              : few_typed<__half>(c, s);
}

}  // namespace snack
