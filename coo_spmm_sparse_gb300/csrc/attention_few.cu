// The forward call of few query rows (decode steps, short prompts): 16 rows to
// a block, whose four warps take the keys in turn, each on its own.
//
// The caches' bytes are the work.  A lane copies a row of a warp's next tile
// (16 keys and their values; 8 in 32 bits at head sizes above 64) with one bulk
// copy, three tiles deep, complete on the warp's own barrier: no barrier of the
// block and hardly an instruction is spent on a copy, where 16-byte copies by
// every thread took most of the instructions and held the kernel at 2.4 TB/s.
// Rows that are not whole aligned vectors are copied element by element.
// Long caches are cut into chunks for more blocks, joined by join_splits.
#include "attention_rows.cuh"
#include "tcgen05.cuh"

namespace snack {
namespace {

__device__ int g_few_failed = 0;

constexpr int kWarps = 4, kStages = 3;

template <typename T, int DP>
struct Few {
  static constexpr int kKeys = sizeof(T) == 4 && DP > 64 ? 8 : 16;  // of a warp's tile
  static constexpr int kStep = kWarps * kKeys, kLd = DP + 8;
  static constexpr int kTileElems = 2 * kKeys * kLd;
  static constexpr size_t ring = (size_t)kWarps * kStages * kTileElems * sizeof(T);
  static constexpr size_t room = (size_t)(kWarps - 1) * 16 * kLd * sizeof(float);
  static constexpr size_t smem = 16 * kLd * sizeof(T) + (ring > room ? ring : room);
};

__device__ __forceinline__ void copy_row(void *to, const void *from, uint32_t bytes, uint64_t *bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                   tc::smem_addr(to)),
               "l"(from), "r"(bytes), "r"(tc::smem_addr(bar))
               : "memory");
}

template <typename T, int DP>
__global__ void __launch_bounds__(32 * kWarps) few_forward(const AttnCall c) {
  using Ops = Tile<T, DP>;
  using F = Few<T, DP>;
  constexpr int kLd = F::kLd, NB = F::kKeys / 8, KEYS = F::kKeys;
  extern __shared__ __align__(16) unsigned char smem[];
  __shared__ uint64_t bars[kWarps][kStages];
  __shared__ float stat[2][kWarps][16];
  __shared__ int failed_flag;
  T *const sq = reinterpret_cast<T *>(smem);
  volatile int *const failed = &failed_flag;

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
  if (c.splits > 1) end = min(end, begin + c.chunk);

  T *const ring = sq + 16 * kLd + warp * kStages * F::kTileElems;
  const Rows<T> kr(c.k, ks, c.k_offsets != nullptr, kh, 1, c.d), vr(c.v, ks, c.k_offsets != nullptr, kh, 1, c.d);
  const uint32_t row_bytes = (uint32_t)(c.d * sizeof(T));
  const bool bulk = kr.vec && vr.vec && row_bytes % 16 == 0;
  if (begin < end) {
    const Rows<T> qr(c.q, qs, c.q_offsets != nullptr, kh * G, G, c.d);
    copy_rows<T, DP>(sq, qr, r0, 16, nq * G);
    // columns behind the head size stay zero; what is copied never reaches them
    if (c.d < DP)
      for (int r = lane; r < kStages * 2 * KEYS; r += 32)
        for (int col = c.d; col < DP; ++col) ring[r * kLd + col] = from_float<T>(0.f);
  }
  copies_commit();
  if (threadIdx.x == 0) failed_flag = 0;
  if (lane == 0) {
    for (int s = 0; s < kStages; ++s) tc::bar_init(&bars[warp][s], 1);
    tc::fence_bar_init();
  }
  tc::fence_async_proxy();
  copies_wait<0>();
  __syncthreads();

  const int first = begin + warp * KEYS;
  const int steps = first < end ? (end - first + F::kStep - 1) / F::kStep : 0;
  const auto copy_tile = [&](int step) {
    const int key0 = first + step * F::kStep, rows = min(KEYS, end - key0), stage = step % kStages;
    T *const k = ring + stage * F::kTileElems, *const v = k + KEYS * kLd;
    uint64_t *const bar = &bars[warp][stage];
    if (bulk) {
      if (lane == 0) tc::bar_expect(bar, 2 * rows * row_bytes);
      __syncwarp();
    }
    for (int r = lane; r < 2 * KEYS; r += 32) {
      const bool is_v = r >= KEYS;
      const int i = is_v ? r - KEYS : r;
      T *const to = (is_v ? v : k) + i * kLd;
      const T *const from = (is_v ? vr : kr).row(key0 + min(i, rows - 1));
      if (i >= rows) {  // values that meet zero probabilities have to be numbers
        for (int col = 0; col < DP; ++col) to[col] = from_float<T>(0.f);
      } else if (bulk) {
        copy_row(to, from, row_bytes, bar);
      }
    }
    if (!bulk) {
      for (int r = 0; r < 2 * rows; ++r) {
        const bool is_v = r >= rows;
        const int i = is_v ? r - rows : r;
        const T *const from = (is_v ? vr : kr).row(key0 + i);
        T *const to = (is_v ? v : k) + i * kLd;
        for (int col = lane; col < c.d; col += 32) to[col] = from[col];
      }
      __syncwarp();
    }
  };

  // the two rows of this lane; the second eight hold nothing where there are no more rows
  const bool both = r0 + 8 < min(qs.cover * G, nq * G);
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
  for (int i = 0; i < min(steps, kStages - 1); ++i) copy_tile(i);
  bool ok = true;
  for (int step = 0; step < steps; ++step) {
    const int stage = step % kStages, key = first + step * F::kStep;
    if (step + kStages - 1 < steps) copy_tile(step + kStages - 1);
    if (bulk) ok = __all_sync(0xffffffffu, tc::bar_wait(&bars[warp][stage], (step / kStages) & 1, failed));
    if (!ok) break;
    __syncwarp();
    const T *const k = ring + stage * F::kTileElems, *const v = k + KEYS * kLd;
    float s[NB][4] = {};
    Ops::template rows_by_rows<NB>(s, sq, k, lane);
    float shrink[2] = {1.f, 1.f};
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      if (h == 1 && !both) {
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
  }
  if (!ok) {  // the copies of this warp end before the block does
    int unseen = 0;
    for (int s = 0; s < kStages; ++s)
      for (int phase = 0; phase < 2; ++phase) tc::bar_wait(&bars[warp][s], phase, &unseen);
  }
  dependency_launch();
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    l[h] += __shfl_xor_sync(0xffffffffu, l[h], 1);
    l[h] += __shfl_xor_sync(0xffffffffu, l[h], 2);
  }
  const int row = lane >> 2;
  if ((lane & 3) == 0)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      stat[0][warp][row + 8 * h] = m[h];
      stat[1][warp][row + 8 * h] = l[h];
    }
  __syncthreads();
  if (threadIdx.x == 0 && failed_flag) g_few_failed = 1;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    float top = -INFINITY, sum = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) top = fmaxf(top, stat[0][w][row + 8 * h]);
    const float from = top == -INFINITY ? 0.f : top;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) sum += stat[1][w][row + 8 * h] * exp2f(stat[0][w][row + 8 * h] - from);
    const float shrink = exp2f(m[h] - from);
#pragma unroll
    for (int n = 0; n < DP / 8; ++n) {
      o[n][2 * h] *= shrink;
      o[n][2 * h + 1] *= shrink;
    }
    m[h] = top;
    l[h] = sum;
  }
  add_shares<DP, 1, kWarps>(o, reinterpret_cast<float *>(sq + 16 * kLd), 0, warp, lane);
  if (warp == 0) finish_rows<T, DP>(c, qs, o, m, l, token, head, lane);
}

template <typename T, int DP>
cudaError_t few_sized(const AttnCall &c, cudaStream_t s) {
  const int64_t blocks = tiles_of(c.q_offsets != nullptr, c.sequences, c.q_tokens, c.group, 16) * c.key_heads;
  const auto kern = few_forward<T, DP>;
  const cudaError_t e = allow_smem(kern, Few<T, DP>::smem);
  if (e != cudaSuccess) return e;
  return launch_kernel(kern, dim3((unsigned)blocks, (unsigned)c.splits), 32 * kWarps, Few<T, DP>::smem, false, s, c);
}

template <typename T>
cudaError_t few_typed(const AttnCall &c, cudaStream_t s) {
  return c.d <= 64 ? few_sized<T, 64>(c, s) : few_sized<T, 128>(c, s);
}

}  // namespace

cudaError_t few_forward_launch(const AttnCall &c, int type, cudaStream_t s) {
  return type == SNACK_F32    ? few_typed<float>(c, s)
         : type == SNACK_BF16 ? few_typed<__nv_bfloat16>(c, s)
                              : few_typed<__half>(c, s);
}

cudaError_t few_forward_failed(int *flag, cudaStream_t s) { return read_flag(g_few_failed, flag, s); }

}  // namespace snack
