// Attention: argument checks, the choice of kernels, and what runs around
// them (delta, the joining of split calls).
#include <algorithm>
#include <cmath>

#include "attention.cuh"

namespace snack {
namespace {

constexpr int kTeam = 16;  // lanes that share a row of v

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
  *seq = (int)(row / tokens);
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
    const int64_t item = first + i * kTeams, row = item / c.heads;
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

// The largest |v| of the sequences' keys.
template <typename T>
__global__ void __launch_bounds__(256) attention_peak(const AttnCall c, int64_t rows, uint32_t *peak) {
  const int lane = threadIdx.x % kTeam;
  float top = 0.f;
  const int64_t items = rows * c.key_heads;
  for (int64_t item = (int64_t)blockIdx.x * (256 / kTeam) + threadIdx.x / kTeam; item < items;
       item += (int64_t)gridDim.x * (256 / kTeam)) {
    const int64_t row = item / c.key_heads;
    int seq, token;
    if (!in_sequence(c.k_offsets, c.k_lengths, c.sequences, c.k_tokens, row, &seq, &token)) continue;
    const T *v = static_cast<const T *>(c.v.p) + seq * c.v.seq + token * c.v.token +
                 (item - row * c.key_heads) * c.v.head;
    for (int col = lane; col < c.d; col += kTeam) top = larger(top, to_float(v[col]));
  }
  block_peak(top, peak);
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

// How a forward call is cut: few rows (16 to a block) where blocks of 128
// would leave SMs idle, and its keys in parts where even those do.
struct Cut {
  bool tiles = false, few = false;
  int splits = 1, chunk = 0;
};
Cut cut_of(const AttnCall &c, int type) {
  Cut cut;
  cut.tiles = c.q_tokens >= 64 && tile_forward_fits(c, type);
  if (cut.tiles) return cut;
  const bool ragged = c.q_offsets != nullptr;
  const int64_t sms = device_sms();
  cut.few = tiles_of(ragged, c.sequences, c.q_tokens, c.group, 128) * c.key_heads < sms;
  if (!cut.few) return cut;
  const int64_t blocks = tiles_of(ragged, c.sequences, c.q_tokens, c.group, 16) * c.key_heads;
  // chunks of 512 keys at least: below that a block starts and ends more than it reads
  const int64_t want = blocks ? 16 * sms / blocks : 1, most = c.k_tokens / 512;
  const int64_t splits = std::max<int64_t>(1, std::min(std::min(want, most), (int64_t)kMostSplits));
  if (splits == 1) return cut;
  cut.chunk = (int)round_up((c.k_tokens + splits - 1) / splits, 64);
  cut.splits = (int)((c.k_tokens + cut.chunk - 1) / cut.chunk);
  return cut;
}

template <typename T>
cudaError_t forward_typed(const AttnCall &c, const Cut &cut, int type, cudaStream_t s) {
  if (cut.tiles) return tile_forward_launch(c, type, s);
  if (!cut.few) return rows_forward_launch<T>(c, s);
  cudaError_t e = few_forward_launch(c, type, s);
  if (e == cudaSuccess && c.splits > 1)
    e = launch_kernel(join_splits<T>, dim3((unsigned)(c.rows * c.heads)), 128, 0, true, s, c);
  return e;
}

template <typename T>
cudaError_t backward_typed(AttnCall c, int type, uint32_t *peak, cudaStream_t s) {
  constexpr int E = 16 / sizeof(T);
  cudaError_t e = cudaSuccess;
  if (peak) {
    if ((e = cudaMemsetAsync(peak, 0, 2 * sizeof(uint32_t), s)) != cudaSuccess) return e;
    const int64_t rows = c.k_offsets ? c.k_tokens : (int64_t)c.sequences * c.k_tokens;
    if (rows) {
      const int64_t blocks = std::min<int64_t>((rows * c.key_heads + 15) / 16, 8 * device_sms());
      e = launch_kernel(attention_peak<T>, dim3((unsigned)blocks), 256, 0, false, s, c, rows, peak + 1);
      if (e != cudaSuccess) return e;
    }
    c.peak = peak;
  }
  if (c.rows) {
    const auto even = [](const Strided &t) {
      return aligned_to(t.p, 16) && t.seq % E == 0 && t.token % E == 0 && t.head % E == 0;
    };
    e = delta_launch<T>(c, c.d % E == 0 && even(c.dout) && even(c.out), peak, s);
    if (e != cudaSuccess) return e;
  }
  if (c.q_tokens >= 64 && c.k_tokens >= 64 && tile_backward_fits(c, type)) return tile_backward_launch(c, type, s);
  return rows_backward_launch<T>(c, s);
}

}  // namespace
}  // namespace snack

using namespace snack;

extern "C" size_t snack_attention_forward_workspace(const snack_attention_args *a) {
  if (!a || check_args(a) != SNACK_OK) return 0;
  const AttnCall c = call_of(a);
  const Cut cut = cut_of(c, a->type);
  return cut.splits > 1 ? (size_t)cut.splits * c.rows * c.heads * (c.d + 1) * sizeof(float) : 0;
}

extern "C" snack_status snack_attention_forward(const snack_attention_args *a, void *out, const int64_t *out_stride,
                                                float *lse, void *workspace, void *stream) {
  const snack_status st = check_args(a);
  if (st != SNACK_OK) return st;
  AttnCall c = call_of(a);
  if (c.rows == 0) return SNACK_OK;
  if (!out || !out_stride || !lse) return bad("out, its strides or lse is NULL");
  c.out = strided(out, out_stride);
  c.lse = lse;
  const Cut cut = cut_of(c, a->type);
  c.splits = cut.splits;
  c.chunk = cut.chunk;
  if (cut.splits > 1) {
    if (!workspace) return bad("workspace is NULL");
    c.part = static_cast<float *>(workspace);
  }
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t e = a->type == SNACK_F32    ? forward_typed<float>(c, cut, a->type, s)
                        : a->type == SNACK_BF16 ? forward_typed<__nv_bfloat16>(c, cut, a->type, s)
                                                : forward_typed<__half>(c, cut, a->type, s);
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
  const AttnCall c = call_of(a);
  return (size_t)c.rows * c.heads * sizeof(float) + (a->type == SNACK_F16 ? 16 : 0);
}

extern "C" snack_status snack_attention_backward(const snack_attention_args *a, const snack_attention_grads *g,
                                                 void *workspace, void *stream) {
  const snack_status st = check_args(a);
  if (st != SNACK_OK) return st;
  if (!g) return bad("grads is NULL");
  AttnCall c = call_of(a);
  if (c.rows && (!g->dout || !g->out || !g->lse || !workspace)) return bad("dout, out, lse or workspace is NULL");
  c.dout = strided(g->dout, g->dout_stride);
  c.out = strided(g->out, g->out_stride);
  c.dq = strided(g->dq, g->dq_stride);
  c.dk = strided(g->dk, g->dk_stride);
  c.dv = strided(g->dv, g->dv_stride);
  c.lse = const_cast<float *>(g->lse);
  uint32_t *peak = nullptr;
  if (a->type == SNACK_F16) {
    if (!workspace) return bad("workspace is NULL");
    peak = static_cast<uint32_t *>(workspace);
  }
  c.delta = reinterpret_cast<float *>(static_cast<char *>(workspace) + (peak ? 16 : 0));
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t e = a->type == SNACK_F32    ? backward_typed<float>(c, a->type, peak, s)
                        : a->type == SNACK_BF16 ? backward_typed<__nv_bfloat16>(c, a->type, peak, s)
                                                : backward_typed<__half>(c, a->type, peak, s);
  return e == cudaSuccess ? SNACK_OK : cuda_status(e, "attention backward");
}
