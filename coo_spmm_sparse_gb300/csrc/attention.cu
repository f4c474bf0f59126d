// Attention: argument checks, the choice of kernels, and what runs around
// them (delta, the joining of split calls).
#include <algorithm>
#include <cmath>

#include "attention.cuh"

namespace snack {
namespace {


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

__device__ __forceinline__ void block_peak(float v, uint32_t *peak) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const uint32_t other = __shfl_xor_sync(0xffffffffu, __float_as_uint(v), o);
    if (other > __float_as_uint(v)) v = __uint_as_float(other);  // magnitudes: their bits order as they do
  }
  if ((threadIdx.x & 31) == 0 && __float_as_uint(v) > 0) atomicMax(peak, __float_as_uint(v));
}
__device__ __forceinline__ float larger(float a, float b) {
  return __uint_as_float(max(__float_as_uint(a), __float_as_uint(fabsf(b))));
}

// delta = dout . out for every row and head; with `peak` also the largest
// |dout|.  A team of lanes takes a row with one 16-byte load of each tensor a
// lane, and kItems rows at a time, whose loads are in flight together.
constexpr int kItems = 4;
template <typename T, int TEAM, bool VEC>
__global__ void __launch_bounds__(256) attention_delta(const AttnCall c, uint32_t *peak) {
  constexpr int E = 16 / sizeof(T), kTeams = 256 / TEAM;
  const int lane = threadIdx.x % TEAM;
  const int64_t first = (int64_t)blockIdx.x * (kTeams * kItems) + threadIdx.x / TEAM;
  float sum[kItems] = {}, top = 0.f;
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
      for (int col = lane; col < c.d; col += TEAM) {
        const float v = to_float(d[col]);
        sum[i] += v * to_float(o[col]);
        top = larger(top, v);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < kItems; ++i) {
    if (VEC) {
      float a[E], b[E];
      unpack16<T>(x[i], a);
      unpack16<T>(y[i], b);
#pragma unroll
      for (int e = 0; e < E; ++e) {
        sum[i] += a[e] * b[e];
        top = larger(top, a[e]);
      }
    }
#pragma unroll
    for (int o = TEAM / 2; o > 0; o >>= 1) sum[i] += __shfl_xor_sync(0xffffffffu, sum[i], o);
    if (place[i] >= 0 && lane == 0) c.delta[place[i]] = sum[i];
  }
  if (peak) block_peak(top, peak);
}

template <typename T>
cudaError_t delta_launch(const AttnCall &c, bool vec, uint32_t *peak, cudaStream_t s) {
  const int lanes = vec ? (c.d * (int)sizeof(T) + 15) / 16 : 32;
  const int team = lanes <= 8 ? 8 : lanes <= 16 ? 16 : 32;
  const int64_t each = 256 / team * kItems;
  const dim3 grid((unsigned)((c.rows * c.heads + each - 1) / each));
  if (!vec) return launch_kernel(attention_delta<T, 32, false>, grid, 256, 0, false, s, c, peak);
  return team == 8    ? launch_kernel(attention_delta<T, 8, true>, grid, 256, 0, false, s, c, peak)
         : team == 16 ? launch_kernel(attention_delta<T, 16, true>, grid, 256, 0, false, s, c, peak)
                      : launch_kernel(attention_delta<T, 32, true>, grid, 256, 0, false, s, c, peak);
}

// One tensor of a call and what is made of it.
struct Source {
  Strided from;
  const int32_t *offsets, *lengths;
  int tokens, heads;
  int64_t rows;    // tokens of all sequences
  uint32_t *peak;  // receives the bits of the largest magnitude
  __half *parts;   // receives the float16 parts
};
struct Sources {
  Source t[4];
};

// A warp takes a token, a lane four columns of one of its heads at a time: one
// division a token, where one for every row of a head took longer than the
// memory does.  16 column places a head in the parts, as many as it has else.
__device__ __forceinline__ bool token_of(const Source &t, int sequences, int64_t row, int64_t *at) {
  int seq, token;
  const bool have = in_sequence(t.offsets, t.lengths, sequences, t.tokens, row, &seq, &token);
  *at = seq * t.from.seq + token * t.from.token;
  return have;
}

template <typename T>
__device__ __forceinline__ void load_four(const T *v, int left, float (&x)[4]) {
  if (left >= 4 && (reinterpret_cast<uintptr_t>(v) & (4 * sizeof(T) - 1)) == 0) {
    if constexpr (sizeof(T) == 4) {
      const float4 f = *reinterpret_cast<const float4 *>(v);
      x[0] = f.x, x[1] = f.y, x[2] = f.z, x[3] = f.w;
    } else {
      const uint2 u = *reinterpret_cast<const uint2 *>(v);
      unpack2<T>(u.x, x[0], x[1]);
      unpack2<T>(u.y, x[2], x[3]);
    }
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) x[e] = e < left ? to_float(v[e]) : 0.f;
  }
}

// The largest magnitude of each tensor, over the sequences' tokens.  Grid: y = tensor.
template <typename T>
__global__ void __launch_bounds__(256) attention_peak(const Sources all, int sequences, int d) {
  const Source &t = all.t[blockIdx.y];
  const int lane = threadIdx.x & 31, places = (d + 3) / 4, work = t.heads * places;
  float top = 0.f;
  for (int64_t row = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5); row < t.rows; row += (int64_t)gridDim.x * 8) {
    int64_t at;
    if (!token_of(t, sequences, row, &at)) continue;
    const T *const v = static_cast<const T *>(t.from.p) + at;
#pragma unroll 4
    for (int i = lane; i < work; i += 32) {
      const int head = i / places, col = (i - head * places) * 4;
      float x[4];
      load_four(v + head * t.from.head + col, d - col, x);
#pragma unroll
      for (int e = 0; e < 4; ++e) top = larger(top, x[e]);
    }
  }
  block_peak(top, t.peak);
}

// Every tensor as two float16 parts of its elements times the power of two that
// brings its largest to [2^14, 2^15): rows of 64 high and 64 low halves, zeros
// behind the head size and for tokens outside every sequence.  Grid: y = tensor.
__global__ void __launch_bounds__(256) split_parts(const Sources all, int sequences, int d) {
  const Source &t = all.t[blockIdx.y];
  const int lane = threadIdx.x & 31, work = t.heads * 16;
  const float by = exp2f((float)power_to_half(*t.peak));
  for (int64_t row = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5); row < t.rows; row += (int64_t)gridDim.x * 8) {
    int64_t at;
    const bool have = token_of(t, sequences, row, &at);
    const float *const v = static_cast<const float *>(t.from.p) + at;
    __half *const parts = t.parts + row * t.heads * 128;
#pragma unroll 4
    for (int i = lane; i < work; i += 32) {
      const int head = i / 16, col = i % 16 * 4;
      float x[4] = {};
      if (have && col < d) load_four(v + head * t.from.head + col, d - col, x);
      uint32_t hi[2], lo[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float a, b;
        const float u = x[2 * e] * by, w = x[2 * e + 1] * by;
        hi[e] = pack2<__half>(u, w);
        unpack2<__half>(hi[e], a, b);
        lo[e] = pack2<__half>(u - a, w - b);
      }
      __half *const to = parts + head * 128 + col;
      *reinterpret_cast<uint2 *>(to) = make_uint2(hi[0], hi[1]);
      *reinterpret_cast<uint2 *>(to + 64) = make_uint2(lo[0], lo[1]);
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
  if (a->dropout > 0.f && rows * a->heads >= (int64_t)1 << 34)
    return refuse(SNACK_ERR_UNSUPPORTED, "dropout takes fewer than 2^34 query rows (tokens * heads)");
  const auto tiles = [&](const int32_t *off, int64_t tokens, int64_t per) {
    return tiles_of(off != nullptr, a->sequences, tokens, per, 16) * a->key_heads;
  };
  if (tiles(a->q_offsets, a->q_tokens, group) + tiles(a->k_offsets, a->k_tokens, 1) >= lim ||
      rows * a->heads >= lim * 8)
    return refuse(SNACK_ERR_UNSUPPORTED, "too many rows for one launch");
  const int64_t strides[] = {a->q_stride[0], a->q_stride[1], a->q_stride[2], a->k_stride[0], a->k_stride[1],
                             a->k_stride[2], a->v_stride[0], a->v_stride[1], a->v_stride[2]};
  for (int64_t s : strides)
    if (s < 0) return bad("negative strides");
  const int64_t keys = a->k_offsets ? a->k_tokens : a->sequences * a->k_tokens;
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
  return c;
}

// How a call is computed, and what of the workspace it takes.
struct Plan {
  bool tiles = false, few = false;  // on tcgen05; in blocks of 16 rows
  int splits = 1, chunk = 0;
  size_t delta = 0, parts[4] = {}, bytes = 0;  // offsets: after the peaks; q, k, v, dout
};
constexpr size_t kPeaks = 256;

// The parts of 32-bit operands.
void plan_parts(Plan *p, const AttnCall &c, bool backward) {
  const int64_t keys = c.k_offsets ? c.k_tokens : (int64_t)c.sequences * c.k_tokens;
  const int64_t rows[4] = {c.rows * c.heads, keys * c.key_heads, keys * c.key_heads, backward ? c.rows * c.heads : 0};
  for (int i = 0; i < 4; ++i) {
    p->parts[i] = p->bytes;
    p->bytes += rows[i] * 128 * sizeof(__half);
  }
}

constexpr double kTilesFrom32 = 4e6;
// 16-bit calls go to the tiles from 64 query tokens on.  32-bit ones pay for
// making the parts first (two launches, three or four tensors read twice).
bool worth_tiles(const AttnCall &c, int type) {
  if (c.q_tokens < 64 || c.k_tokens < 64) return false;
  return type != SNACK_F32 || (double)c.rows * c.heads * c.k_tokens >= kTilesFrom32;
}

// Few rows (16 to a block) where blocks of 128 would leave SMs idle, and the
// keys in parts where even those do.
Plan plan_forward(const AttnCall &c, int type) {
  Plan p;
  p.tiles = worth_tiles(c, type) && tile_forward_fits(c, type);
  if (p.tiles) {
    if (type == SNACK_F32) {
      p.bytes = kPeaks;
      plan_parts(&p, c, false);
    }
    return p;
  }
  const bool ragged = c.q_offsets != nullptr;
  const int64_t sms = device_sms();
  p.few = tiles_of(ragged, c.sequences, c.q_tokens, c.group, 128) * c.key_heads < sms;
  if (!p.few) return p;
  const int64_t blocks = tiles_of(ragged, c.sequences, c.q_tokens, c.group, 16) * c.key_heads;
  // chunks of 512 keys at least: below that a block starts and ends more than it reads
  const int64_t want = blocks ? 16 * sms / blocks : 1, most = c.k_tokens / 512;
  const int64_t splits = std::max<int64_t>(1, std::min(std::min(want, most), (int64_t)kMostSplits));
  if (splits == 1) return p;
  p.chunk = (int)round_up((c.k_tokens + splits - 1) / splits, 64);
  p.splits = (int)((c.k_tokens + p.chunk - 1) / p.chunk);
  if (p.splits > 1) p.bytes = (size_t)p.splits * c.rows * c.heads * (c.d + 1) * sizeof(float);
  return p;
}

Plan plan_backward(const AttnCall &c, int type) {
  Plan p;
  p.bytes = kPeaks;
  p.delta = p.bytes;
  p.bytes += round_up(c.rows * c.heads * (int64_t)sizeof(float), 256);
  p.tiles = worth_tiles(c, type) && tile_backward_fits(c, type);
  if (p.tiles && type == SNACK_F32) plan_parts(&p, c, true);
  return p;
}

// q, k, v and dout of a call; peaks in the order that AttnCall has them in.
Sources sources_of(const AttnCall &c, const Plan &p, char *workspace) {
  Sources s;
  uint32_t *const peak = reinterpret_cast<uint32_t *>(workspace);
  const int64_t keys = c.k_offsets ? c.k_tokens : (int64_t)c.sequences * c.k_tokens;
  const Strided *const from[4] = {&c.q, &c.k, &c.v, &c.dout};
  const int at[4] = {2, 3, 1, 0};
  for (int i = 0; i < 4; ++i) {
    const bool own = i == 0 || i == 3;
    s.t[i] = Source{*from[i], own ? c.q_offsets : c.k_offsets, own ? c.q_lengths : c.k_lengths,
                    own ? c.q_tokens : c.k_tokens, own ? c.heads : c.key_heads, own ? c.rows : keys, peak + at[i],
                    reinterpret_cast<__half *>(workspace + p.parts[i])};
  }
  return s;
}

unsigned spread(int64_t rows) {  // a warp for each, or as many as are resident together
  return (unsigned)std::max<int64_t>(1, std::min<int64_t>((rows + 7) / 8, 8 * device_sms()));
}

// Makes the parts of 32-bit operands; `tensors`: 3 (forward) or 4.
cudaError_t make_parts(AttnCall *c, const Plan &p, int tensors, char *workspace, SplitParts *parts, cudaStream_t s) {
  const Sources all = sources_of(*c, p, workspace);
  cudaError_t e = cudaMemsetAsync(workspace, 0, 4 * sizeof(uint32_t), s);
  int64_t most = 0;
  for (int i = 0; i < tensors; ++i) most = std::max(most, all.t[i].rows);
  const dim3 grid(spread(most), (unsigned)tensors);
  if (e == cudaSuccess) e = launch_kernel(attention_peak<float>, grid, 256, 0, false, s, all, c->sequences, c->d);
  if (e == cudaSuccess) e = launch_kernel(split_parts, grid, 256, 0, false, s, all, c->sequences, c->d);
  c->peak = reinterpret_cast<const uint32_t *>(workspace);
  *parts = SplitParts{all.t[0].parts, all.t[1].parts, all.t[2].parts, all.t[3].parts};
  return e;
}

template <typename T>
cudaError_t forward_typed(AttnCall c, const Plan &p, int type, char *workspace, cudaStream_t s) {
  if (p.tiles) {
    SplitParts parts = {};
    if (type == SNACK_F32) {
      const cudaError_t e = make_parts(&c, p, 3, workspace, &parts, s);
      if (e != cudaSuccess) return e;
    }
    return tile_forward_launch(c, type, parts, s);
  }
  if (!p.few) return rows_forward_launch<T>(c, s);
  c.splits = p.splits;
  c.chunk = p.chunk;
  c.part = reinterpret_cast<float *>(workspace);
  cudaError_t e = few_forward_launch(c, type, s);
  if (e == cudaSuccess && c.splits > 1)
    e = launch_kernel(join_splits<T>, dim3((unsigned)(c.rows * c.heads)), 128, 0, true, s, c);
  return e;
}

template <typename T>
cudaError_t backward_typed(AttnCall c, const Plan &p, int type, char *workspace, cudaStream_t s) {
  constexpr int E = 16 / sizeof(T);
  cudaError_t e = cudaSuccess;
  SplitParts parts = {};
  uint32_t *peak = nullptr;  // where delta leaves the largest |dout|
  if (p.tiles && type == SNACK_F32) {
    e = make_parts(&c, p, 4, workspace, &parts, s);
  } else if (type == SNACK_F16) {
    peak = reinterpret_cast<uint32_t *>(workspace);
    c.peak = peak;
    e = cudaMemsetAsync(peak, 0, 2 * sizeof(uint32_t), s);
    Sources v = sources_of(c, p, workspace);
    v.t[0] = v.t[2];
    if (e == cudaSuccess && v.t[0].rows)
      e = launch_kernel(attention_peak<T>, dim3(spread(v.t[0].rows)), 256, 0, false, s, v, c.sequences, c.d);
  }
  if (e != cudaSuccess) return e;
  if (c.rows) {
    const auto even = [](const Strided &t) {
      return aligned_to(t.p, 16) && t.seq % E == 0 && t.token % E == 0 && t.head % E == 0;
    };
    e = delta_launch<T>(c, c.d % E == 0 && even(c.dout) && even(c.out), peak, s);
    if (e != cudaSuccess) return e;
  }
  return p.tiles ? tile_backward_launch(c, type, parts, s) : rows_backward_launch<T>(c, s);
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
  if (p.bytes && !workspace) return bad("workspace is NULL");
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
  if (!workspace) return bad("workspace is NULL");
  if (c.rows && (!g->dout || !g->out || !g->lse)) return bad("dout, out or lse is NULL");
  c.dout = strided(g->dout, g->dout_stride);
  // (what dout decides, whether a 16-bit call can go to the tiles, takes no workspace)
  const Plan p = plan_backward(c, a->type);
  c.out = strided(g->out, g->out_stride);
  c.dq = strided(g->dq, g->dq_stride);
  c.dk = strided(g->dk, g->dk_stride);
  c.dv = strided(g->dv, g->dv_stride);
  c.lse = const_cast<float *>(g->lse);
  char *const ws = static_cast<char *>(workspace);
  c.delta = reinterpret_cast<float *>(ws + p.delta);
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t e = a->type == SNACK_F32    ? backward_typed<float>(c, p, a->type, ws, s)
                        : a->type == SNACK_BF16 ? backward_typed<__nv_bfloat16>(c, p, a->type, ws, s)
                                                : backward_typed<__half>(c, p, a->type, ws, s);
  return e == cudaSuccess ? SNACK_OK : cuda_status(e, "attention backward");
}
