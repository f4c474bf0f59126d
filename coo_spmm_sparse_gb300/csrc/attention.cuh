// What the attention kernels share: the call as the device sees it, its
// sequences and tiles, the mask that dropout makes of a probability's place.
#pragma once

#include "counter_random.cuh"
#include "dense_ops.cuh"

namespace snack {

struct Strided {
  void *p;
  int64_t seq, token, head;  // elements
};

struct AttnCall {
  Strided q, k, v, out, dout, dq, dk, dv;
  float *lse;    // [heads][rows]: log of the sum of exp(scale * q . k), -inf where no key is seen
  float *delta;  // [heads][rows]: dout . out
  float *part;   // partial results of a split call
  // Operands made in float16.  32-bit calls: the power of two that the parts of each
  // tile of 128 tokens of a head are scaled by, [tile][head] (tiles numbered as Span
  // says).  bfloat16 calls: bits of the largest magnitude of each sequence and key head,
  // [sequence][key head], from which the power follows
  const int32_t *q_power, *k_power, *v_power, *dout_power;
  int64_t rows;  // rows of lse for a head: all tokens of q
  int sequences, q_tokens, k_tokens;
  int heads, key_heads, group, d;
  int causal, splits, chunk;
  float scale, scale_log2;  // scale * log2(e)
  const int32_t *q_offsets, *k_offsets, *q_lengths, *k_lengths;
  uint32_t drop;  // 0: no dropout; else a probability is kept where its 16 bits are at least this
  float keep_scale;  // 1 without dropout
  uint64_t seed;
  const uint64_t *seed_at;
  int polls;  // of a wait on tcgen05, before it gives up

  __device__ __forceinline__ uint64_t draws() const { return seed_at ? *seed_at : seed; }
};

constexpr int kTile = 128;  // tokens of a tile on tcgen05

// The tokens of one sequence on one side.  Rows `valid` .. cover-1 belong to the
// tensor but not to the sequence (padding): their results are zero.
struct Span {
  int64_t row;   // number of the first token among all
  int64_t tile;  // number of the first tile of kTile tokens among all (a ragged side leaves numbers out)
  int valid, cover;
  int seq;  // of a dense side; 0 in a ragged one, whose tokens are numbered through
};

// Numbers of tiles that a side can have: the tiles of ragged sequence s begin at
// offset / kTile + s, which is at least where those of sequence s - 1 end.
inline int64_t tile_numbers(bool ragged, int64_t n, int64_t tokens) {
  return ragged ? tokens / kTile + n + 3 : n * ((tokens + kTile - 1) / kTile);
}

// Sequences are numbered 0 .. sequences-1 in a dense side.  A ragged side has
// two more, without partners on the other side: the tokens before the first
// offset (number 0) and behind the last (sequences + 1), whose results are
// zero.  Broken offsets are cut to the tensor: nothing outside is touched.
__device__ __forceinline__ int clamped(const int32_t *offsets, int i, int tokens) {
  const int v = offsets[i];
  return v < 0 ? 0 : (v > tokens ? tokens : v);
}

__device__ __forceinline__ int ragged_begin(const int32_t *offsets, int s, int tokens) {
  return s == 0 ? 0 : clamped(offsets, s - 1, tokens);
}
__device__ __forceinline__ int ragged_end(const int32_t *offsets, int s, int n, int tokens) {
  return s == n + 1 ? tokens : clamped(offsets, s, tokens);
}

// The span of sequence `s` of the side that is cut into tiles.
__device__ __forceinline__ Span own_span(const int32_t *offsets, const int32_t *lengths, int s, int n, int tokens) {
  Span sp;
  if (offsets) {
    const int a = ragged_begin(offsets, s, tokens), b = ragged_end(offsets, s, n, tokens);
    sp.row = a;
    sp.tile = a / kTile + s;
    sp.cover = b > a ? b - a : 0;
    sp.valid = s == 0 || s == n + 1 ? 0 : sp.cover;
    sp.seq = 0;
    return sp;
  }
  sp.row = (int64_t)s * tokens;
  sp.tile = (int64_t)s * ((tokens + kTile - 1) / kTile);
  sp.cover = tokens;
  sp.valid = lengths ? min(max(lengths[s], 0), tokens) : tokens;
  sp.seq = s;
  return sp;
}

// The span of the same sequence on the other side; `ragged` says how s is
// numbered.
__device__ __forceinline__ Span other_span(const int32_t *offsets, const int32_t *lengths, int s, bool ragged, int n,
                                           int tokens) {
  const int i = ragged ? s - 1 : s;
  if (i < 0 || i >= n) return Span{0, 0, 0, 0, 0};
  if (offsets) return own_span(offsets, nullptr, i + 1, n, tokens);
  return own_span(nullptr, lengths, i, n, tokens);
}

// Sequence and tile of tile number t, where each sequence has ceil(cover *
// per_token / tile_rows) tiles.  Called by whole warps.  s < 0: no such tile.
// Tiles of a sequence are numbered from its end where `back`: under a causal
// mask the later rows have the most to do and start first.
struct Place {
  int s, tile;
};
__device__ __forceinline__ Place find_tile(const int32_t *offsets, int n, int tokens, int per_token, int tile_rows,
                                           int t, bool back) {
  if (!offsets) {
    const int per = (int)(((int64_t)tokens * per_token + tile_rows - 1) / tile_rows);
    const int s = t / per, i = t - s * per;
    if (s >= n) return Place{-1, 0};
    return Place{s, back ? per - 1 - i : i};
  }
  const int lane = threadIdx.x & 31;
  for (int s0 = 0; s0 < n + 2; s0 += 32) {
    const int s = s0 + lane;
    int own = 0;
    if (s < n + 2) {
      const int a = ragged_begin(offsets, s, tokens), b = ragged_end(offsets, s, n, tokens);
      if (b > a) own = (int)(((int64_t)(b - a) * per_token + tile_rows - 1) / tile_rows);
    }
    int upto = own;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += v;
    }
    const unsigned hit = __ballot_sync(0xffffffffu, t < upto);
    if (hit) {
      const int l = __ffs(hit) - 1;
      const int cnt = __shfl_sync(0xffffffffu, own, l), end = __shfl_sync(0xffffffffu, upto, l);
      const int i = t - (end - cnt);
      return Place{s0 + l, back ? cnt - 1 - i : i};
    }
    t -= __shfl_sync(0xffffffffu, upto, 31);
  }
  return Place{-1, 0};
}

// The launches of attention on mma.sync, by type (attention_rows_*.cu).
template <typename T>
cudaError_t rows_forward_launch(const AttnCall &c, cudaStream_t s);
template <typename T>
cudaError_t rows_backward_launch(const AttnCall &c, cudaStream_t s);

// The forward call of few rows (attention_few.cu).
cudaError_t few_forward_launch(const AttnCall &c, int type, cudaStream_t s);

// Where operands that were made are: [tokens][heads][width]; width 0: none are.
struct SplitParts {
  int width;
  bool halves;  // bfloat16's made in float16
  void *q, *k, *v, *dout;
};

// Those of attention on tcgen05 (attention_tiles*.cu): which calls they take,
// whether TMA can bring a 16-bit call's tensors as they lie (else they are copied
// first), and whether one of their bounded waits has run out since the last question.
bool tiles_take(const AttnCall &c, int type);
bool tiles_read(const AttnCall &c);  // as the tensors lie
int64_t tile_forward_blocks(const AttnCall &c);
cudaError_t tile_forward_launch(const AttnCall &c, int type, const SplitParts &parts, cudaStream_t s);
cudaError_t tile_forward_failed(int *flag, cudaStream_t s);
cudaError_t tile_backward_launch(const AttnCall &c, int type, const SplitParts &parts, cudaStream_t s);
cudaError_t tile_backward_failed(int *flag, cudaStream_t s);

// Reads a sticky flag of the current device and clears it.
template <typename S>
inline cudaError_t read_flag(S &symbol, int *flag, cudaStream_t s) {
  int v = 0;
  const int zero = 0;
  cudaError_t e = cudaMemcpyFromSymbolAsync(&v, symbol, sizeof(int), 0, cudaMemcpyDeviceToHost, s);
  if (e == cudaSuccess) e = cudaStreamSynchronize(s);
  if (e == cudaSuccess && v) {
    e = cudaMemcpyToSymbolAsync(symbol, &zero, sizeof(int), 0, cudaMemcpyHostToDevice, s);
    if (e == cudaSuccess) e = cudaStreamSynchronize(s);
    *flag = 1;
  }
  return e;
}

// Tiles that a grid needs so that every sequence finds all of its own.
inline int64_t tiles_of(bool ragged, int64_t n, int64_t tokens, int64_t per_token, int64_t tile_rows) {
  const int64_t per = (tokens * per_token + tile_rows - 1) / tile_rows;
  return ragged ? per + n + 2 : n * per;
}

// float16 holds neither a small gradient's dS nor small probabilities well: the
// backward kernels take P 2^14 fold there, and a row's dS (a query's where dq is
// summed, a key's where dk is) times a power of two of its own, which the row's sums
// are divided by again.  Nothing of it comes from other rows: with one power for a
// call, tokens whose dout was 1e-4 of the largest had dq off by 7e-3 in 32 bits.
//
// 2^power brings a magnitude with these exponent bits (of a 32-bit float) to
// [2^top, 2^(top + 1)); a row without one, or one that is not finite, takes `other`.
constexpr float kHalfP = 14.f;
constexpr int kMostPower = 100;
__device__ __forceinline__ uint32_t exponent_bits(float magnitude) { return __float_as_uint(magnitude) >> 23; }
__device__ __forceinline__ int row_power(uint32_t exponent, int top, int other) {
  return exponent == 0 || exponent == 255 ? other : min(max(top + 127 - (int)exponent, -kMostPower), kMostPower);
}
__device__ __forceinline__ float power_of_two(int n) { return __uint_as_float((uint32_t)(n + 127) << 23); }  // |n| <= 126

// The power of a row whose sums stay where they are from step to step: they are
// multiplied down when a step's largest would pass 2^15.  Sixteen fold room is left,
// so that this is rare; two float16 parts still reach down to 2^-36 of the largest.
__device__ __forceinline__ int running_power(int power, uint32_t exponent) {
  const int need = row_power(exponent, 11, power);
  return power > need + 3 ? need : power;
}

// The power of two that brings the largest magnitude to [2^14, 2^15).
__device__ __forceinline__ int power_to_half(uint32_t peak) {
  const float v = __uint_as_float(peak);
  if (!(v > 0.f) || !(v < INFINITY)) return 0;
  return min(max(14 - ilogbf(v), -113), 120);
}

// Keys that query i of a sequence sees: j < seen_keys(...).
__device__ __forceinline__ int seen_keys(int causal, int i, int nq, int nk) {
  return causal ? min(nk, i + nk - nq + 1) : nk;
}

// The first query that sees one of the keys from j0 on; nq where there is none: a
// tile that lies wholly in padding has no queries (j0 - nk + nq would be up to
// j0 then, and that times the group passes 31 bits).
__host__ __device__ inline int first_query(int causal, int j0, int nq, int nk) {
  if (j0 >= nk) return nq;
  const int first = causal ? j0 - nk + nq : 0;
  return first > 0 ? first : 0;
}

// The number of the draw that decides about keys 4c .. 4c+3 of a query row is
// row * 2^30 + c, with row = token * heads + head.
__device__ __forceinline__ uint64_t dropout_row(uint64_t seed, int64_t token, int heads, int head) {
  return seed + ((((uint64_t)token * heads + head) << 30) + 1ull) * kSplitMixStep;
}
__device__ __forceinline__ uint64_t dropout_draw(uint64_t row, int key) {
  return splitmix_finish(row + (uint64_t)(uint32_t)(key >> 2) * kSplitMixStep);
}

}  // namespace snack
