// Attention: argument checks, the choice of kernels, and what runs around
// them (delta, the joining of split calls).
#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstring>

#include "attention_rows.cuh"
#include "tcgen05.cuh"

namespace snack {
namespace {

std::atomic<int> g_polls{tc::kPolls};

template <typename T>
__device__ __forceinline__ void unpack16(const uint4 &u, float (&v)[16 / sizeof(T)]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (sizeof(T) == 4)
      v[i] = __uint_as_float(w[i]);
    else
      unpack2<T>(w[i], v[2 * i], v[2 * i + 1]);
  }
}

// The tokens of a side that belong to a sequence.
__device__ __forceinline__ bool in_sequence(const int32_t *offsets, const int32_t *lengths, int n, int tokens,
                                            int64_t row, int *seq, int *token) {
  if (offsets) {
    *seq = 0;
    *token = (int)row;
    return row >= clamped(offsets, 0, tokens) && row < clamped(offsets, n, tokens);
  }
  *seq = row >> 31 ? (int)(row / tokens) : (int)((uint32_t)row / (uint32_t)tokens);
  *token = (int)(row - (int64_t)*seq * tokens);
  return !lengths || *token < lengths[*seq];
}

__device__ __forceinline__ float larger(float a, float b) {
  return __uint_as_float(max(__float_as_uint(a), __float_as_uint(fabsf(b))));
}

// 16 bytes of elements from v on, of which `left` are there.
template <typename T>
__device__ __forceinline__ uint4 load_vector(const T *v, int left) {
  constexpr int E = 16 / sizeof(T);
  if (left >= E && (reinterpret_cast<uintptr_t>(v) & 15) == 0) return *reinterpret_cast<const uint4 *>(v);
  uint4 u = make_uint4(0, 0, 0, 0);
  T x[E];
#pragma unroll
  for (int e = 0; e < E; ++e) x[e] = e < left ? v[e] : from_float<T>(0.f);
  memcpy(&u, x, 16);
  return u;
}

// 16-bit types: delta of a row that sees 2 to kFewKeys keys is sum_j M P (dout . v_j),
// from the tensors themselves.  out is rounded, and with delta from it causal calls'
// dq and dk were off by this many times what rounding the results alone costs (worst
// of 5 draws, three shapes): 7.3 at 2 keys, 2.1 at 8, 1.6 at 32 and 1.3 at 64; from
// here 1.0.  Which rows do depends on the keys that they see and on nothing else of
// the call.
constexpr int kFewKeys = 32;
__device__ __forceinline__ bool few_keys(int seen) { return seen >= 2 && seen <= kFewKeys; }

// The keys that a row of all sequences sees.
__device__ __forceinline__ int seen_by_row(const AttnCall &c, int64_t row, int seq, int token) {
  int s = seq;
  if (c.q_offsets) {  // the last sequence that begins at or before the row
    int lo = 0, hi = c.sequences;
    while (hi - lo > 1) {
      const int mid = (lo + hi) / 2;
      if (clamped(c.q_offsets, mid, c.q_tokens) <= row) lo = mid; else hi = mid;
    }
    s = lo;
  }
  const Span qs = own_span(c.q_offsets, c.q_lengths, c.q_offsets ? s + 1 : s, c.sequences, c.q_tokens);
  const Span ks = own_span(c.k_offsets, c.k_lengths, c.k_offsets ? s + 1 : s, c.sequences, c.k_tokens);
  return seen_keys(c.causal, c.q_offsets ? (int)(row - qs.row) : token, qs.valid, ks.valid);
}

// Those rows of a sequence are neighbours (the first ones of a causal call).  A block
// takes 32 of them and one head at a time, every `parts`-th of its sequence and head;
// both products on mma.sync, a warp 16 rows and 16 keys of them.  (A warp a row, its lanes
// side by side along keys, took 170 us of a call of 500 x 40 tokens.)
template <int DP>
constexpr size_t few_keys_smem() { return 4 * kFewKeys * (DP + 8) * 2; }
template <typename T, int DP>
__device__ __forceinline__ void delta_of_few_keys(const AttnCall &c, int64_t block, int parts) {
  using Ops = Tile<T, DP>;
  constexpr int kLd = Ops::kLd, kRows = 32;
  extern __shared__ __align__(16) unsigned char smem[];
  __shared__ float sums[2][kRows];
  T *const sq = reinterpret_cast<T *>(smem), *const sd = sq + kRows * kLd, *const sk = sd + kRows * kLd,
           *const sv = sk + kFewKeys * kLd;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, part = (int)(block % parts);
  const int head = (int)(block / parts % c.heads), s = (int)(block / parts / c.heads), kh = head / c.group;
  const Span qs = own_span(c.q_offsets, c.q_lengths, c.q_offsets ? s + 1 : s, c.sequences, c.q_tokens);
  const Span ks = own_span(c.k_offsets, c.k_lengths, c.k_offsets ? s + 1 : s, c.sequences, c.k_tokens);
  const int nq = qs.valid, nk = ks.valid;
  const int lo = c.causal ? max(0, nq - nk + 1) : 0;
  const int hi = c.causal ? min((int64_t)nq, (int64_t)nq - nk + kFewKeys) : few_keys(nk) ? nq : 0;
  int64_t i0 = lo + (int64_t)part * kRows;
  if (i0 >= hi) return;
  const Rows<T> kr(c.k, ks, c.k_offsets != nullptr, kh, 1, c.d), vr(c.v, ks, c.k_offsets != nullptr, kh, 1, c.d);
  const Rows<T> qr(c.q, qs, c.q_offsets != nullptr, head, 1, c.d), dr(c.dout, qs, c.q_offsets != nullptr, head, 1, c.d);
  copy_rows<T, DP>(sk, kr, 0, kFewKeys, min(nk, kFewKeys));
  copy_rows<T, DP>(sv, vr, 0, kFewKeys, min(nk, kFewKeys));
  const int row0 = (warp & 1) * 16, key0 = (warp >> 1) * 16;
  for (; i0 < hi; i0 += (int64_t)parts * kRows) {
    copy_rows<T, DP>(sq, qr, (int)i0, kRows, hi);
    copy_rows<T, DP>(sd, dr, (int)i0, kRows, hi);
    copies_commit();
    copies_wait<0>();
    __syncthreads();
    if (warp < 4) {
      float score[2][4] = {}, dprob[2][4] = {};
      Ops::template rows_by_rows<2>(score, sq + row0 * kLd, sk + key0 * kLd, lane);
      Ops::template rows_by_rows<2>(dprob, sd + row0 * kLd, sv + key0 * kLd, lane);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int r = row0 + (lane >> 2) + 8 * h, i = (int)i0 + r;
        const int seen = i < hi ? seen_keys(c.causal, i, nq, nk) : 0;
        const int64_t row = qs.row + i;
        const float lse = seen > 0 ? c.lse[(int64_t)head * c.rows + row] : 0.f;
        const uint64_t draws = c.drop ? dropout_row(c.draws(), row, c.heads, head) : 0;
        float sum = 0.f;
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int j = key0 + Ops::column(n, lane, e), x = 2 * h + e;
            float p = j < seen ? expf(score[n][x] * c.scale - lse) * dprob[n][x] : 0.f;
            if (c.drop) p = draw_lane(dropout_draw(draws, j), j & 3) >= c.drop ? p * c.keep_scale : 0.f;
            sum += p;
          }
        sum += __shfl_xor_sync(0xffffffffu, sum, 1);
        sum += __shfl_xor_sync(0xffffffffu, sum, 2);
        if ((lane & 3) == 0) sums[warp >> 1][r] = lse == -INFINITY ? 0.f : sum;
      }
    }
    __syncthreads();
    if (threadIdx.x < kRows && i0 + threadIdx.x < hi)
      c.delta[(int64_t)head * c.rows + qs.row + i0 + threadIdx.x] = sums[0][threadIdx.x] + sums[1][threadIdx.x];
  }
}

// delta of the other rows, dout . out.  A team of lanes takes a row with one 16-byte
// load of each tensor a lane, and kItems rows at a time, whose loads are in flight
// together.  The first `few` blocks take the rows of few keys: bf16 backward calls, us,
// with delta of out alone / with them (the rest of the call as it was): 8 x 24 tokens, 24
// heads over 12 of 128, 27 / 31; 64 x 33, 12 over 4, 70 / 79; 300 x 2, 24 over 12, 303 / 357 (two
// rows to a block); 500 x 40 at 128 columns 698 / 736.
constexpr int kItems = 4;
template <typename T, int TEAM, bool VEC>
__global__ void __launch_bounds__(256, 3) attention_delta(const AttnCall c, int few, int parts) {
  if constexpr (sizeof(T) == 2)
    if ((int)blockIdx.x < few) {
      for (int64_t b = blockIdx.x; b < (int64_t)c.sequences * c.heads * parts; b += few) {
        delta_of_few_keys<T, TEAM == 8 ? 64 : 128>(c, b, parts);
        __syncthreads();
      }
      return;
    }
  constexpr int E = 16 / sizeof(T), kTeams = 256 / TEAM;
  const int lane = threadIdx.x % TEAM;
  const int64_t first = (int64_t)(blockIdx.x - few) * (kTeams * kItems) + threadIdx.x / TEAM;
  float sum[kItems] = {};
  int64_t place[kItems];
  uint4 x[kItems], y[kItems];
#pragma unroll
  for (int i = 0; i < kItems; ++i) {
    const int64_t item = first + i * kTeams;
    const int64_t row = item >> 31 ? item / c.heads : (int64_t)((uint32_t)item / (uint32_t)c.heads);
    const int head = (int)(item - row * c.heads);
    int seq = 0, token = 0;
    const bool have = row < c.rows && in_sequence(c.q_offsets, c.q_lengths, c.sequences, c.q_tokens, row, &seq, &token);
    place[i] = have ? (int64_t)head * c.rows + row : -1;
    x[i] = y[i] = make_uint4(0, 0, 0, 0);
    if (!have) continue;
    const T *d = static_cast<const T *>(c.dout.p) + seq * c.dout.seq + token * c.dout.token + head * c.dout.head;
    const T *o = static_cast<const T *>(c.out.p) + seq * c.out.seq + token * c.out.token + head * c.out.head;
    if (VEC) {
      if (lane * E < c.d) {
        x[i] = *reinterpret_cast<const uint4 *>(d + lane * E);
        y[i] = *reinterpret_cast<const uint4 *>(o + lane * E);
      }
    } else {
      for (int col = lane; col < c.d; col += TEAM) sum[i] += to_float(d[col]) * to_float(o[col]);
    }
    if (sizeof(T) == 2 && few && few_keys(seen_by_row(c, row, seq, token))) place[i] = -1;
  }
#pragma unroll
  for (int i = 0; i < kItems; ++i) {
    if (VEC) {
      float a[E], b[E];
      unpack16<T>(x[i], a);
      unpack16<T>(y[i], b);
#pragma unroll
      for (int e = 0; e < E; ++e) sum[i] += a[e] * b[e];
    }
#pragma unroll
    for (int o = TEAM / 2; o > 0; o >>= 1) sum[i] += __shfl_xor_sync(0xffffffffu, sum[i], o);
    if (place[i] >= 0 && lane == 0) c.delta[place[i]] = sum[i];
  }
}

template <typename T>
cudaError_t delta_launch(const AttnCall &c, cudaStream_t s) {
  constexpr int E = 16 / sizeof(T);
  const auto even = [](const Strided &t) {
    return aligned_to(t.p, 16) && t.seq % E == 0 && t.token % E == 0 && t.head % E == 0;
  };
  const bool vec = c.d % E == 0 && even(c.dout) && even(c.out);
  const int lanes = vec ? (c.d * (int)sizeof(T) + 15) / 16 : 32;
  const int team = lanes <= 8 ? 8 : lanes <= 16 ? 16 : 32;
  const int64_t each = 256 / team * kItems;
  // blocks for rows of few keys: one for 32 of a sequence and head, or as many as keep the SMs busy
  int64_t few = 0, parts = 0;
  const bool all_long = !c.causal && !c.k_offsets && !c.k_lengths && c.k_tokens > kFewKeys;
  if (sizeof(T) == 2 && c.sequences && !all_long) {
    const int64_t rows = c.causal ? std::min(c.q_tokens, kFewKeys - 1) : c.q_tokens;
    const int64_t units = (int64_t)c.sequences * c.heads;
    parts = std::max<int64_t>(1, std::min<int64_t>((rows + 31) / 32, 16 * device_sms() / units));
    few = std::min<int64_t>(units * parts, 1 << 24);
  }
  const dim3 grid((unsigned)((c.rows * c.heads + each - 1) / each + few));
  const auto launch = [&](auto kern) {
    return launch_kernel(kern, grid, 256, !few ? 0 : team == 8 ? few_keys_smem<64>() : few_keys_smem<128>(), false, s, c,
                         (int)few, (int)parts);
  };
  if (!vec) return launch(attention_delta<T, 32, false>);
  return team == 8    ? launch(attention_delta<T, 8, true>)
         : team == 16 ? launch(attention_delta<T, 16, true>)
                      : launch(attention_delta<T, 32, true>);
}

// One tensor of a call and what is made of it.
struct Source {
  Strided from;
  const int32_t *offsets, *lengths;
  int tokens, heads;
  int64_t rows;    // tokens of all sequences
  void *made;      // receives what the tiles read
  int32_t *power;  // made in float16: and the powers of two of its tiles, or peaks of its sequences
};
struct Sources {
  Source t[4];
};

// A warp takes a token, a lane 16 bytes of one of its heads at a time: one
// division a token, where one for every row of a head took longer than the
// memory does.
__device__ __forceinline__ bool token_of(const Source &t, int sequences, int64_t row, int64_t *at) {
  int seq, token;
  const bool have = in_sequence(t.offsets, t.lengths, sequences, t.tokens, row, &seq, &token);
  *at = seq * t.from.seq + token * t.from.token;
  return have;
}

// 16-bit tensors as TMA can bring them: rows of W columns of each head, zeros behind
// the head size and for tokens outside every sequence.  Grid: y = tensor.
template <typename T, int W>
__global__ void __launch_bounds__(256) copy_operands(const Sources all, int sequences, int d) {
  constexpr int E = 16 / sizeof(T), kPlaces = W / E, kAhead = 4;
  const Source &t = all.t[blockIdx.y];
  const int lane = threadIdx.x & 31, work = t.heads * kPlaces;
  for (int64_t row = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5); row < t.rows; row += (int64_t)gridDim.x * 8) {
    int64_t at;
    const bool have = token_of(t, sequences, row, &at);
    const T *const v = static_cast<const T *>(t.from.p) + at;
    uint4 *const made = static_cast<uint4 *>(t.made) + row * work;
    for (int i0 = lane; i0 < work; i0 += 32 * kAhead) {
      uint4 u[kAhead];
#pragma unroll
      for (int n = 0; n < kAhead; ++n) {
        const int i = i0 + n * 32, head = i / kPlaces, col = i % kPlaces * E;
        u[n] = have && i < work && col < d ? load_vector(v + head * t.from.head + col, d - col) : make_uint4(0, 0, 0, 0);
      }
#pragma unroll
      for (int n = 0; n < kAhead; ++n)
        if (i0 + n * 32 < work) made[i0 + n * 32] = u[n];
    }
  }
}

// Sequence and tile of a tile's number (as Span counts them): by bisection, where
// find_tile, whose order is the products', goes through the sequences.  s < 0: the
// number is left out.
__device__ __forceinline__ Place numbered_tile(const Source &t, int n, int64_t number) {
  if (!t.offsets) {
    const int per = (t.tokens + kTile - 1) / kTile;
    const int s = (int)(number / per);
    return s < n ? Place{s, (int)(number - (int64_t)s * per)} : Place{-1, 0};
  }
  int lo = 0, hi = n + 2;  // the last sequence whose tiles begin at or before the number
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (ragged_begin(t.offsets, mid, t.tokens) / kTile + mid <= number) lo = mid; else hi = mid;
  }
  const int a = ragged_begin(t.offsets, lo, t.tokens), b = ragged_end(t.offsets, lo, n, t.tokens);
  const int64_t tile = number - (a / kTile + lo);
  return tile >= 0 && tile * kTile < b - a ? Place{lo, (int)tile} : Place{-1, 0};
}

// 32-bit tensors as two float16 parts, rows of 64 high and 64 low halves (zeros as
// above), of the elements times the power of two that brings the largest of their
// tile to [2^14, 2^15).  A block takes a tile of a head, which stays in registers
// from the search for its largest on: the memory is read once.  Grid: x = the tile's
// number * heads + head, y = tensor.
__global__ void __launch_bounds__(256) split_operands(const Sources all, int sequences, int d) {
  __shared__ uint32_t tops[8];
  const Source &t = all.t[blockIdx.y];
  const int head = blockIdx.x % t.heads;
  const Place at = numbered_tile(t, sequences, blockIdx.x / t.heads);
  if (at.s < 0) return;
  const Span sp = own_span(t.offsets, t.lengths, at.s, sequences, t.tokens);
  constexpr int kRows = kTile / 16;  // of a thread; 16 threads take a row
  const int col = threadIdx.x % 16 * 4, first = at.tile * kTile + threadIdx.x / 16;
  const float *const from = static_cast<const float *>(t.from.p) +
                            (t.offsets ? sp.row * t.from.token : sp.seq * t.from.seq) + head * t.from.head + col;
  float x[kRows][4], top = 0.f;
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    const int row = first + 16 * i;
    const uint4 u = row < sp.valid && col < d ? load_vector(from + row * t.from.token, d - col) : make_uint4(0, 0, 0, 0);
    unpack16<float>(u, x[i]);
  }
#pragma unroll
  for (int i = 0; i < kRows; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) top = larger(top, x[i][e]);
  uint32_t most = __reduce_max_sync(0xffffffffu, __float_as_uint(top));  // magnitudes: their bits order as they do
  if ((threadIdx.x & 31) == 0) tops[threadIdx.x >> 5] = most;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < 8; ++w) most = max(most, tops[w]);
  const int power = power_to_half(most);
  if (threadIdx.x == 0) t.power[blockIdx.x] = power;
  const float by = power_of_two(power);
  uint16_t *const made = static_cast<uint16_t *>(t.made) + head * 128 + col;
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    const int row = first + 16 * i;
    if (row >= sp.cover) break;
    uint32_t hi[2], lo[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      float a, b;
      const float l = x[i][2 * e] * by, r = x[i][2 * e + 1] * by;
      hi[e] = pack2<__half>(l, r);
      unpack2<__half>(hi[e], a, b);
      lo[e] = pack2<__half>(l - a, r - b);
    }
    uint16_t *const to = made + (sp.row + row) * t.heads * 128;
    *reinterpret_cast<uint2 *>(to) = make_uint2(hi[0], hi[1]);
    *reinterpret_cast<uint2 *>(to + 64) = make_uint2(lo[0], lo[1]);
  }
}

// bfloat16 tensors in float16, rows of 128 columns: of the elements times the power of
// two that brings the largest of their sequence and key head to [2^14, 2^15), so that
// nothing depends on other sequences and key heads; the eight bits lose nothing down
// to 2^-28 of it.  Two launches of the same blocks, each a tile of a head: the first finds
// the largest, the second writes.  Grid as above.
template <bool WRITE>
__global__ void __launch_bounds__(256) half_operands(const Sources all, int sequences, int key_heads, int d) {
  using T = __nv_bfloat16;
  __shared__ uint32_t tops[8];
  const Source &t = all.t[blockIdx.y];
  const int head = blockIdx.x % t.heads, kh = head / (t.heads / key_heads);
  const Place at = numbered_tile(t, sequences, blockIdx.x / t.heads);
  if (at.s < 0) return;
  const Span sp = own_span(t.offsets, t.lengths, at.s, sequences, t.tokens);
  constexpr int kRows = kTile / 16;  // of a thread; 16 threads take a row
  const int col = threadIdx.x % 16 * 8, first = at.tile * kTile + threadIdx.x / 16;
  const T *const from = static_cast<const T *>(t.from.p) +
                        (t.offsets ? sp.row * t.from.token : sp.seq * t.from.seq) + head * t.from.head + col;
  uint32_t *const peak = reinterpret_cast<uint32_t *>(t.power) + (int64_t)at.s * key_heads + kh;
  uint4 u[kRows];
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    const int row = first + 16 * i;
    u[i] = row < sp.valid && col < d ? load_vector(from + row * t.from.token, d - col) : make_uint4(0, 0, 0, 0);
  }
  if constexpr (!WRITE) {
    float top = 0.f;
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      float x[8];
      unpack16<T>(u[i], x);
#pragma unroll
      for (int e = 0; e < 8; ++e) top = larger(top, x[e]);
    }
    uint32_t most = __reduce_max_sync(0xffffffffu, __float_as_uint(top));
    if ((threadIdx.x & 31) == 0) tops[threadIdx.x >> 5] = most;
    __syncthreads();
    if (threadIdx.x == 0) {
#pragma unroll
      for (int w = 0; w < 8; ++w) most = max(most, tops[w]);
      atomicMax(peak, most);  // (a maximum does not depend on the order)
    }
  } else {
    const float by = power_of_two(power_to_half(*peak));
    uint16_t *const made = static_cast<uint16_t *>(t.made) + head * 128 + col;
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      const int row = first + 16 * i;
      if (row >= sp.cover) break;
      float x[8];
      unpack16<T>(u[i], x);
      *reinterpret_cast<uint4 *>(made + (sp.row + row) * t.heads * 128) =
          make_uint4(pack2<__half>(x[0] * by, x[1] * by), pack2<__half>(x[2] * by, x[3] * by),
                     pack2<__half>(x[4] * by, x[5] * by), pack2<__half>(x[6] * by, x[7] * by));
    }
  }
}

// Joins the parts of a split forward call: a block for each row and head, a
// thread for each column.  Launched early; waits for the parts' kernel here.
constexpr int kMostSplits = 128;
template <typename T>
__global__ void __launch_bounds__(128) join_splits(const AttnCall c) {
  __shared__ float weight[kMostSplits], top_of[4], sum_of[4];
  dependency_wait();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t items = c.rows * c.heads, item = blockIdx.x, row = item / c.heads;
  const int head = (int)(item - row * c.heads);
  const float *const parts = c.part + item * c.d + tid, *const lse = c.part + (int64_t)c.splits * items * c.d + item;
  const float own = tid < c.splits ? lse[tid * items] : -INFINITY;
  float top = own;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  if (lane == 0) top_of[warp] = top;
  __syncthreads();
  top = fmaxf(fmaxf(top_of[0], top_of[1]), fmaxf(top_of[2], top_of[3]));
  const float w = expf(own - (top == -INFINITY ? 0.f : top));
  weight[tid] = w;
  const float part = warp_sum(w);
  if (lane == 0) sum_of[warp] = part;
  __syncthreads();
  const float sum = (sum_of[0] + sum_of[1]) + (sum_of[2] + sum_of[3]);
  if (tid < c.d) {
    float acc = 0.f;
#pragma unroll 8
    for (int s = 0; s < c.splits; ++s) acc += weight[s] * parts[s * items * c.d];  // (a part without keys is zero)
    const int64_t seq = c.q_offsets ? 0 : row / c.q_tokens, token = c.q_offsets ? row : row - seq * c.q_tokens;
    T *out = static_cast<T *>(c.out.p) + seq * c.out.seq + token * c.out.token + head * c.out.head;
    out[tid] = from_float<T>(sum == 0.f ? 0.f : acc / sum);
  }
  if (tid == 0) c.lse[(int64_t)head * c.rows + row] = sum == 0.f ? -INFINITY : top + logf(sum);
}

// ------------------------------------------------------------------ host

int64_t round_up(int64_t a, int64_t b) { return (a + b - 1) / b * b; }

bool dense_or_ragged(const int32_t *offsets, const int32_t *lengths) { return !(offsets && lengths); }

snack_status bad(const std::string &m) { return refuse(SNACK_ERR_INVALID_ARG, m); }

snack_status check_args(const snack_attention_args *a) {
  if (!a) return bad("args is NULL");
  if (!known_type(a->type)) return bad("unknown element type");
  if (a->head_size < 1 || a->head_size > 128) return bad("head_size must be 1 to 128");
  if (a->key_heads < 1 || a->heads < 1 || a->heads % a->key_heads)
    return bad("heads must be a positive multiple of key_heads");
  if (a->sequences < 0 || a->q_tokens < 0 || a->k_tokens < 0) return bad("negative sizes");
  if (a->causal != 0 && a->causal != 1) return bad("causal must be 0 or 1");
  if (!std::isfinite(a->scale)) return bad("scale must be finite");
  if (!(a->dropout >= 0.f && a->dropout < 1.f) || std::lround(a->dropout * 65536.0) > 65535)
    return bad("dropout must be at least 0 and below 1 - 2^-17");
  if (!dense_or_ragged(a->q_offsets, a->q_lengths) || !dense_or_ragged(a->k_offsets, a->k_lengths))
    return bad("a side has offsets or lengths, not both");
  const int64_t lim = (int64_t)1 << 31;
  const int64_t group = a->heads / a->key_heads;
  if (a->sequences > (1 << 24) || a->heads > (1 << 16)) return refuse(SNACK_ERR_UNSUPPORTED, "more than 2^24 sequences or 2^16 heads");
  if (a->k_tokens >= lim - 4096 || a->q_tokens >= lim || a->q_tokens * group >= lim - 4096)
    return refuse(SNACK_ERR_UNSUPPORTED, "tokens, and query tokens * group, must be below 2^31 - 4096");
  const int64_t rows = a->q_offsets ? a->q_tokens : a->sequences * a->q_tokens;
  const int64_t keys = a->k_offsets ? a->k_tokens : a->sequences * a->k_tokens;
  if (rows >= (int64_t)1 << 40 || keys >= (int64_t)1 << 40)
    return refuse(SNACK_ERR_UNSUPPORTED, "more than 2^40 tokens");
  if (a->dropout > 0.f && rows * a->heads >= (int64_t)1 << 34)
    return refuse(SNACK_ERR_UNSUPPORTED, "dropout takes fewer than 2^34 query rows (tokens * heads)");
  const auto tiles = [&](const int32_t *off, int64_t tokens, int64_t per) {
    return tiles_of(off != nullptr, a->sequences, tokens, per, 16) * a->key_heads;
  };
  if (a->sequences > (1 << 16) && (a->q_offsets || a->k_offsets))
    return refuse(SNACK_ERR_UNSUPPORTED, "a ragged side takes at most 2^16 sequences");  // every block looks for its own
  if (tiles(a->q_offsets, a->q_tokens, group) + tiles(a->k_offsets, a->k_tokens, 1) >= lim ||
      tiles_of(a->q_offsets != nullptr, a->sequences, a->q_tokens, 1, kTile) * a->heads >= lim ||
      rows * a->heads >= lim * 4)
    return refuse(SNACK_ERR_UNSUPPORTED, "too many rows for one launch");
  const int64_t strides[] = {a->q_stride[0], a->q_stride[1], a->q_stride[2], a->k_stride[0], a->k_stride[1],
                             a->k_stride[2], a->v_stride[0], a->v_stride[1], a->v_stride[2]};
  for (int64_t s : strides)
    if (s < 0) return bad("negative strides");
  if ((rows && !a->q) || (keys && (!a->k || !a->v))) return bad("q, k or v is NULL");
  return SNACK_OK;
}

Strided strided(const void *p, const int64_t *s) { return Strided{const_cast<void *>(p), s[0], s[1], s[2]}; }

AttnCall call_of(const snack_attention_args *a) {
  AttnCall c = {};
  c.q = strided(a->q, a->q_stride);
  c.k = strided(a->k, a->k_stride);
  c.v = strided(a->v, a->v_stride);
  c.rows = a->q_offsets ? a->q_tokens : a->sequences * a->q_tokens;
  c.sequences = (int)a->sequences;
  c.q_tokens = (int)a->q_tokens;
  c.k_tokens = (int)a->k_tokens;
  c.heads = a->heads;
  c.key_heads = a->key_heads;
  c.group = a->heads / a->key_heads;
  c.d = a->head_size;
  c.causal = a->causal;
  c.splits = 1;
  c.scale = a->scale;
  c.scale_log2 = a->scale * 1.4426950408889634f;
  c.q_offsets = a->q_offsets;
  c.k_offsets = a->k_offsets;
  c.q_lengths = a->q_lengths;
  c.k_lengths = a->k_lengths;
  c.drop = (uint32_t)std::lround(a->dropout * 65536.0);
  c.keep_scale = c.drop ? 65536.f / (float)(65536 - c.drop) : 1.f;
  c.seed = a->seed;
  c.seed_at = a->seed_at;
  c.polls = g_polls.load(std::memory_order_relaxed);
  return c;
}

// How a call is computed, and what of the workspace it takes.
struct Plan {
  bool tiles = false, few = false;  // on tcgen05; in blocks of 16 rows
  int splits = 1, chunk = 0, width = 0;  // width: columns of operands that are made; 0: none are
  bool halves = false;                   // bfloat16's, in float16
  size_t part = 0, parts[4] = {}, powers[4] = {}, bytes = 0;  // offsets (delta is at 0); parts: of q, k, v, dout
};

// Operands that are made first: those of 32-bit calls, and 16-bit tensors that TMA
// cannot bring as they lie (odd head sizes, addresses or strides): else mma.sync
// would take them, several times slower.
int part_width(const AttnCall &c, int type) {
  if (type == SNACK_F32) return 128;
  return tiles_read(c) ? 0 : c.d <= 64 ? 64 : 128;
}
void plan_parts(Plan *p, const AttnCall &c, int type, bool backward) {
  const int64_t keys = c.k_offsets ? c.k_tokens : (int64_t)c.sequences * c.k_tokens;
  const int64_t rows[4] = {c.rows * c.heads, keys * c.key_heads, keys * c.key_heads, backward ? c.rows * c.heads : 0};
  for (int i = 0; i < 4; ++i) {
    p->parts[i] = p->bytes;
    p->bytes += rows[i] * p->width * 2;
  }
  if (type != SNACK_F32 && !p->halves) return;
  int64_t q = tile_numbers(c.q_offsets, c.sequences, c.q_tokens) * c.heads;
  int64_t k = tile_numbers(c.k_offsets, c.sequences, c.k_tokens) * c.key_heads;
  if (p->halves) q = k = ((int64_t)c.sequences + 2) * c.key_heads;
  const int64_t tiles[4] = {q, k, k, backward ? q : 0};
  for (int i = 0; i < 4; ++i) {
    p->powers[i] = p->bytes;
    p->bytes += round_up(tiles[i] * (int64_t)sizeof(int32_t), 16);
  }
}

// The tiles take calls from 64 query tokens on, where there is work for them:
// X = query rows (tokens * heads) * keys.  12 heads of 64 (16 over 4 where it says so),
// tiles / mma.sync, us:
//   forward, bf16: 1 x 128 (X = 2e5) 8 / 7; 1 x 256 (8e5) 10 / 10, 16 over 4 10 / 10; 2 x 256
//   (1.6e6) 10 / 11; 4 x 256 (3e6) 10 / 17; 1 x 1024 (1.3e7) 18 / 41: from 1e6;
//   backward, bf16 and float16: 1 x 128 17 / 17, 18 / 17; 1 x 256 19 / 23, 19 / 25; 4 x 128
//   (8e5) 17 / 29, 19 / 29; 1 x 1024 28 / 97, 31 / 103: from 5e5;
//   fp32, where the operands are made first, forward: 1 x 256 19 / 15; 2 x 256 19 / 19; 4 x 256
//   21 / 31; 8 x 256 (6e6) 23 / 58; backward 1 x 256 26 / 34; 2 x 256 31 / 51; 4 x 256 33 / 99.  The
//   float16 parts leave gradients 1.5 times as far from 64 bits as the tf32 parts do
//   (6.2e-7, 4.2e-7 at 1 x 256), so: where they take less than about half the time, from 4e6
//   forward and 2e6 backward.
// Few rows over many keys are too few for the forward tiles even with the keys
// in parts.  A ragged side's lengths are not known here, only their mean; a tile holds
// one sequence's tokens.  Forward, bf16, 24 heads over 8 of 128, tiles / without, us:
// 128 x 1 over 500 keys each 228 / 56; 256 x 8 tokens 291 / 86; 128 x 16 139 / 56; but 1 x
// 2000 and 127 x 1 162 / 176, 1 x 4000 and 255 x 4 376 / 591 (mean 20; fp32, 12 heads of
// 64, 295 / 659): without below a mean of 16.  Backward, where the keys' side counts too,
// 128 x 1 over 500 619 / 720, 256 x 8 496 / 285, 1 x 2000 and 127 x 1 315 / 771: tiles.
bool worth_tiles(const AttnCall &c, int type, bool backward) {
  if (c.q_tokens < 64 || c.k_tokens < 64) return false;
  if (c.q_offsets && !backward && c.q_tokens < (int64_t)16 * c.sequences) return false;
  const double rows = (double)c.rows * c.heads, x = rows * c.k_tokens;
  if (backward) return x >= (type == SNACK_F32 ? 2e6 : 5e5);
  return x >= (type == SNACK_F32 ? 4e6 : 1e6) && rows >= 1024;
}

// Off the tiles, 16 rows to a block where blocks of 128 would leave SMs idle, and
// where a sequence has few rows for its key head (tokens * group; the mean on a ragged
// side), so that most of a block of 128 would be empty.  bf16, 128 rows / 16, us:
// decoding 128 requests over 500 keys, 24 heads over 8 of 128 (3 rows) 187 / 53; 512 over
// 1024 1358 / 307; 512 over 2048, 32 over 1 (32 rows) 396 / 186; fp32 256 over 4096, 64 over 2
// (32) 3341 / 1021; 256 x 32 tokens over 512, 12 heads of 64 (32) 259 / 162, but over 32 keys 37 / 44;
// 256 x 48 over 300 (48) 173 / 179; 16 tokens of a group of 3 over 64 keys (48) 29 / 35.  The
// keys in parts where the blocks still leave SMs idle.
Plan plan_forward(const AttnCall &c, int type) {
  Plan p;
  const int64_t sms = device_sms();
  p.tiles = worth_tiles(c, type, false) && tiles_take(c, type);
  int64_t blocks, least, want;  // least keys of a part: below that it starts and ends more than it reads
  if (p.tiles) {
    p.width = part_width(c, type);
    if (p.width) plan_parts(&p, c, type, false);
    blocks = tile_forward_blocks(c);
    least = 1024;
    want = blocks ? sms / blocks : 1;
  } else {
    const bool ragged = c.q_offsets != nullptr;
    p.few = tiles_of(ragged, c.sequences, c.q_tokens, c.group, 128) * c.key_heads < sms ||
            (int64_t)c.q_tokens * c.group <= (int64_t)32 * (ragged ? c.sequences : 1);
    if (!p.few) return p;
    blocks = tiles_of(ragged, c.sequences, c.q_tokens, c.group, 16) * c.key_heads;
    least = 512;
    want = blocks ? 16 * sms / blocks : 1;
  }
  const int64_t splits = std::min(std::min(want, c.k_tokens / least), (int64_t)kMostSplits);
  if (splits <= 1) return p;
  p.chunk = (int)round_up((c.k_tokens + splits - 1) / splits, 128);
  p.splits = (int)(((int64_t)c.k_tokens + p.chunk - 1) / p.chunk);
  if (p.splits > 1) {
    p.part = p.bytes;
    p.bytes += (size_t)p.splits * c.rows * c.heads * (c.d + 1) * sizeof(float);
  }
  return p;
}

// bfloat16 backward calls whose operands are made in float16 (attention_tiles_backward.cu):
// seven products instead of ten, for passes that make them.  X as above; heads of 128,
// made / as they lie, us: 2 x 2048 tokens, 16 over 4 heads (X = 1.3e8) 171 / 150; 1 x 4096
// (2.7e8) 284 / 271; 1 x 8192 (1.1e9) 691 / 750; 32 over 8 (2.1e9) 1375 / 1550; 4 x 4096 (2.1e9)
// 1618 / 1722.  At 64 columns exponentials bind, not products.  On a ragged side the mean of
// the keys counts: 500 x 40 tokens have few products however many tokens there are.
bool halves_take(const AttnCall &c) {
  const double keys = c.k_offsets ? (double)c.k_tokens / std::max(c.sequences, 1) : c.k_tokens;
  return c.d > 64 && (double)c.rows * c.heads * keys >= 6e8;
}

Plan plan_backward(const AttnCall &c, int type) {
  Plan p;
  p.bytes = round_up(std::max<int64_t>(c.rows * c.heads, 1) * (int64_t)sizeof(float), 256);
  p.tiles = worth_tiles(c, type, true) && tiles_take(c, type);
  p.halves = p.tiles && type == SNACK_BF16 && halves_take(c);
  p.width = !p.tiles ? 0 : p.halves ? 128 : part_width(c, type);
  if (p.width) plan_parts(&p, c, type, true);
  return p;
}

// q, k, v and dout of a call.
Sources sources_of(const AttnCall &c, const Plan &p, char *workspace) {
  Sources s;
  const int64_t keys = c.k_offsets ? c.k_tokens : (int64_t)c.sequences * c.k_tokens;
  const Strided *const from[4] = {&c.q, &c.k, &c.v, &c.dout};
  for (int i = 0; i < 4; ++i) {
    const bool own = i == 0 || i == 3;
    s.t[i] = Source{*from[i], own ? c.q_offsets : c.k_offsets, own ? c.q_lengths : c.k_lengths,
                    own ? c.q_tokens : c.k_tokens, own ? c.heads : c.key_heads, own ? c.rows : keys,
                    workspace + p.parts[i], reinterpret_cast<int32_t *>(workspace + p.powers[i])};
  }
  return s;
}

unsigned spread(int64_t rows) {  // a warp for each, or as many as are resident together
  return (unsigned)std::max<int64_t>(1, std::min<int64_t>((rows + 7) / 8, 8 * device_sms()));
}

// Makes a call's operands: q, k, v and, backward, dout.
template <typename T>
cudaError_t make_parts(AttnCall *c, const Plan &p, bool backward, char *workspace, SplitParts *parts, cudaStream_t s) {
  const Sources all = sources_of(*c, p, workspace);
  *parts = SplitParts{p.width, p.halves, all.t[0].made, all.t[1].made, all.t[2].made, all.t[3].made};
  const unsigned tensors = backward ? 4 : 3;
  c->q_power = all.t[0].power;
  c->k_power = all.t[1].power;
  c->v_power = all.t[2].power;
  c->dout_power = all.t[3].power;
  const int64_t q = tile_numbers(c->q_offsets, c->sequences, c->q_tokens) * c->heads;
  const int64_t k = tile_numbers(c->k_offsets, c->sequences, c->k_tokens) * c->key_heads;
  const dim3 tiles((unsigned)std::max(q, k), tensors);
  if constexpr (sizeof(T) == 4) {
    return launch_kernel(split_operands, tiles, 256, 0, false, s, all, c->sequences, c->d);
  } else {
    if (p.halves) {
      cudaError_t e = cudaMemsetAsync(all.t[0].power, 0, p.bytes - p.powers[0], s);
      if (e == cudaSuccess)
        e = launch_kernel(half_operands<false>, tiles, 256, 0, false, s, all, c->sequences, c->key_heads, c->d);
      if (e == cudaSuccess)
        e = launch_kernel(half_operands<true>, tiles, 256, 0, false, s, all, c->sequences, c->key_heads, c->d);
      return e;
    }
    const unsigned blocks = spread(std::max(all.t[0].rows, all.t[1].rows));
    return launch_kernel(p.width == 64 ? copy_operands<T, 64> : copy_operands<T, 128>, dim3(blocks, tensors), 256, 0,
                         false, s, all, c->sequences, c->d);
  }
}

template <typename T>
cudaError_t forward_typed(AttnCall c, const Plan &p, int type, char *workspace, cudaStream_t s) {
  if (!p.tiles && !p.few) return rows_forward_launch<T>(c, s);
  c.splits = p.splits;
  c.chunk = p.chunk;
  c.part = reinterpret_cast<float *>(workspace + p.part);
  cudaError_t e = cudaSuccess;
  if (p.tiles) {
    SplitParts parts = {};
    if (p.width) e = make_parts<T>(&c, p, false, workspace, &parts, s);
    if (e == cudaSuccess) e = tile_forward_launch(c, type, parts, s);
  } else {
    e = few_forward_launch(c, type, s);
  }
  if (e == cudaSuccess && c.splits > 1)
    e = launch_kernel(join_splits<T>, dim3((unsigned)(c.rows * c.heads)), 128, 0, true, s, c);
  return e;
}

template <typename T>
cudaError_t backward_typed(AttnCall c, const Plan &p, int type, char *workspace, cudaStream_t s) {
  cudaError_t e = c.rows ? delta_launch<T>(c, s) : cudaSuccess;
  if (e != cudaSuccess) return e;
  SplitParts parts = {};
  if (p.width) e = make_parts<T>(&c, p, true, workspace, &parts, s);
  if (e != cudaSuccess) return e;
  // (a 16-bit call whose dout alone lies badly was not planned for)
  if (p.tiles && (p.width || tiles_read(c))) return tile_backward_launch(c, type, parts, s);
  return rows_backward_launch<T>(c, s);
}

}  // namespace
}  // namespace snack

using namespace snack;

extern "C" size_t snack_attention_forward_workspace(const snack_attention_args *a) {
  if (!a || check_args(a) != SNACK_OK) return 0;
  return plan_forward(call_of(a), a->type).bytes;
}

extern "C" snack_status snack_attention_forward(const snack_attention_args *a, void *out, const int64_t *out_stride,
                                                float *lse, void *workspace, void *stream) {
  const snack_status st = check_args(a);
  if (st != SNACK_OK) return st;
  AttnCall c = call_of(a);
  if (c.rows == 0) return SNACK_OK;
  if (!out || !out_stride || !lse) return bad("out, its strides or lse is NULL");
  // the plan knows the arguments alone, so that it is the one the workspace was asked for
  const Plan p = plan_forward(c, a->type);
  if (p.bytes && (!workspace || !aligned_to(workspace, 16))) return bad("workspace is NULL or not 16-byte aligned");
  c.out = strided(out, out_stride);
  c.lse = lse;
  char *const ws = static_cast<char *>(workspace);
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t e = a->type == SNACK_F32    ? forward_typed<float>(c, p, a->type, ws, s)
                        : a->type == SNACK_BF16 ? forward_typed<__nv_bfloat16>(c, p, a->type, ws, s)
                                                : forward_typed<__half>(c, p, a->type, ws, s);
  return e == cudaSuccess ? SNACK_OK : cuda_status(e, "attention forward");
}

extern "C" snack_status snack_attention_error(int *flag, void *stream) {
  if (!flag) return bad("flag is NULL");
  *flag = 0;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e = tile_forward_failed(flag, s);
  if (e == cudaSuccess) e = tile_backward_failed(flag, s);
  return e == cudaSuccess ? SNACK_OK : cuda_status(e, "attention error flag");
}

extern "C" void snack_debug_attention_polls(int polls) {
  g_polls.store(polls < 0 ? tc::kPolls : polls, std::memory_order_relaxed);
}

extern "C" size_t snack_attention_backward_workspace(const snack_attention_args *a) {
  if (!a || check_args(a) != SNACK_OK) return 0;
  return plan_backward(call_of(a), a->type).bytes;
}

extern "C" snack_status snack_attention_backward(const snack_attention_args *a, const snack_attention_grads *g,
                                                 void *workspace, void *stream) {
  const snack_status st = check_args(a);
  if (st != SNACK_OK) return st;
  if (!g) return bad("grads is NULL");
  AttnCall c = call_of(a);
  if (!workspace || !aligned_to(workspace, 16)) return bad("workspace is NULL or not 16-byte aligned");
  if (c.rows && (!g->dout || !g->out || !g->lse)) return bad("dout, out or lse is NULL");
  const Plan p = plan_backward(c, a->type);  // before dout: the plan that the workspace was asked for
  c.dout = strided(g->dout, g->dout_stride);
  c.out = strided(g->out, g->out_stride);
  c.dq = strided(g->dq, g->dq_stride);
  c.dk = strided(g->dk, g->dk_stride);
  c.dv = strided(g->dv, g->dv_stride);
  c.lse = const_cast<float *>(g->lse);
  char *const ws = static_cast<char *>(workspace);
  c.delta = reinterpret_cast<float *>(ws);
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t e = a->type == SNACK_F32    ? backward_typed<float>(c, p, a->type, ws, s)
                        : a->type == SNACK_BF16 ? backward_typed<__nv_bfloat16>(c, p, a->type, ws, s)
                                                : backward_typed<__half>(c, p, a->type, ws, s);
  return e == cudaSuccess ? SNACK_OK : cuda_status(e, "attention backward");
}
