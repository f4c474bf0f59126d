// The norms before and after a block, with its gate and residual scales:
//
//   u = P(y) or y;   r = a x + b g u;   h = N(r)
//
// and, with D the whole gradient of r (that of the residual path plus what
// comes back through N), t = dh * w:
//
//   D  = dr + rho_r (t - mean(t) - rhat mean(t rhat))      (no mean(t) for the rms norm)
//   dx = a D;   dz = b g D;   dg = b u D;   dy the same rule as D's second term, on p = dz * w_post
//   dw_next = sum_rows dh rhat, db_next = sum_rows dh, dw_post = sum_rows dz yhat, db_post = sum_rows dz
//
// Memory bound: some 20 to 40 operations for every element read.  The
// backward reads x and y again rather than r: r can be had from them exactly
// as the forward computed it, before its rounding, and so the gradients do
// not carry the rounding of r to 16 bits.
#include <algorithm>

#include "residual_norm.cuh"

namespace snack {
namespace {

constexpr int kThreads = 256;

// Column sums of the backward: the gradients of weights, biases and of a
// gate that rows share.
constexpr int kCols = 5;
enum { kNextW = 0, kNextB = 1, kPostW = 2, kPostB = 3, kGate = 4 };

// One row's view of the inputs.
template <typename TS, typename TB>
struct Row {
  const snack_norm_args &a;
  const TS *x;
  const TB *y;
  const TB *gate;  // full or sequence gate row, channel gate, or null
  float token_gate;
  float ym, yr;    // statistics of y
  __device__ __forceinline__ Row(const snack_norm_args &a_, int64_t row) : a(a_), ym(0.f), yr(1.f) {
    x = static_cast<const TS *>(a.x) + row * a.x_stride;
    y = a.y ? static_cast<const TB *>(a.y) + row * a.y_stride : nullptr;
    gate = nullptr;
    token_gate = 1.f;
    const TB *g = static_cast<const TB *>(a.gate);
    if (a.gate_kind == SNACK_GATE_CHANNEL) gate = g;
    if (a.gate_kind == SNACK_GATE_SEQUENCE) gate = g + (row / a.group_rows) * a.width;
    if (a.gate_kind == SNACK_GATE_FULL) gate = g + row * a.gate_stride;
    if (a.gate_kind == SNACK_GATE_TOKEN) token_gate = to_float(g[row]);
  }
  __device__ __forceinline__ float gate_at(int64_t i) const { return gate ? to_float(gate[i]) : token_gate; }
  __device__ __forceinline__ float yhat(int64_t i) const { return (to_float(y[i]) - ym) * yr; }
  __device__ __forceinline__ float u(int64_t i) const {
    if (!a.post_norm) return to_float(y[i]);
    float v = yhat(i);
    if (a.post_weight) v *= load_as_float(a.post_weight, a.param_type, i);
    if (a.post_bias) v += load_as_float(a.post_bias, a.param_type, i);
    return v;
  }
  __device__ __forceinline__ float r(int64_t i) const {
    const float v = a.residual_scale * to_float(x[i]);
    return y ? fmaf(a.branch_scale * gate_at(i), u(i), v) : v;
  }
};

// Mean and 1/deviation of f(i) over the row, in every thread.
template <typename F>
__device__ __forceinline__ void row_stats(const snack_norm_args &a, F f, float *red, float &mean, float &rstd) {
  float s[1] = {0.f};
  mean = 0.f;
  if (a.norm_kind == SNACK_NORM_LAYER) {
    for (int64_t i = threadIdx.x; i < a.width; i += blockDim.x) s[0] += f(i);
    block_sum(s, red);
    mean = s[0] / (float)a.width;
    s[0] = 0.f;
  }
  for (int64_t i = threadIdx.x; i < a.width; i += blockDim.x) {
    const float d = f(i) - mean;
    s[0] = fmaf(d, d, s[0]);
  }
  block_sum(s, red);
  rstd = 1.f / sqrtf(s[0] / (float)a.width + a.eps);
}

template <typename TS, typename TB>
__global__ void __launch_bounds__(kThreads) norm_forward_rows(const __grid_constant__ NormArgs n) {
  __shared__ float red[64];
  dependency_wait();
  const snack_norm_args &a = n.a;
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    Row<TS, TB> c(a, row);
    float mean = 0.f, rstd = 1.f;
    if (a.y && a.post_norm) row_stats(a, [&](int64_t i) { return to_float(c.y[i]); }, red, c.ym, c.yr);
    if (a.next_norm) row_stats(a, [&](int64_t i) { return c.r(i); }, red, mean, rstd);
    for (int64_t i = threadIdx.x; i < a.width; i += kThreads) {
      const float r = c.r(i);
      if (n.r) static_cast<TS *>(n.r)[row * a.width + i] = from_float<TS>(r);
      if (a.next_norm) {
        float h = (r - mean) * rstd;
        if (a.next_weight) h *= load_as_float(a.next_weight, a.param_type, i);
        if (a.next_bias) h += load_as_float(a.next_bias, a.param_type, i);
        static_cast<TB *>(n.h)[row * a.width + i] = from_float<TB>(h);
      }
    }
    if (a.stats && threadIdx.x == 0)
      reinterpret_cast<float4 *>(a.stats)[row] = make_float4(c.ym, c.yr, mean, rstd);
  }
}

// t = dh * w and the gradient of r, from the row's two means.
template <typename TS, typename TB>
struct BackRow : Row<TS, TB> {
  const TS *dr;
  const TB *dh;
  float mean, rstd, c1, c2;
  __device__ __forceinline__ BackRow(const NormArgs &n, int64_t row) : Row<TS, TB>(n.a, row), c1(0.f), c2(0.f) {
    dr = n.g.dr ? static_cast<const TS *>(n.g.dr) + row * n.g.dr_stride : nullptr;
    dh = n.g.dh && n.a.next_norm ? static_cast<const TB *>(n.g.dh) + row * n.g.dh_stride : nullptr;
    const float4 s = reinterpret_cast<const float4 *>(n.a.stats)[row];
    this->ym = s.x;
    this->yr = s.y;
    mean = s.z;
    rstd = s.w;
  }
  __device__ __forceinline__ float t(int64_t i) const {
    const float v = to_float(dh[i]);
    return this->a.next_weight ? v * load_as_float(this->a.next_weight, this->a.param_type, i) : v;
  }
  __device__ __forceinline__ float rhat(int64_t i) const { return (this->r(i) - mean) * rstd; }
  __device__ __forceinline__ float D(int64_t i) const {
    float v = dr ? to_float(dr[i]) : 0.f;
    if (dh) v += rstd * (t(i) - c1 - rhat(i) * c2);
    return v;
  }
};

template <typename TS, typename TB>
__global__ void __launch_bounds__(kThreads) norm_backward_rows(const __grid_constant__ NormArgs n) {
  __shared__ float red[64];
  dependency_wait();
  const snack_norm_args &a = n.a;
  const bool layer = a.norm_kind == SNACK_NORM_LAYER;
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    BackRow<TS, TB> c(n, row);
    if (c.dh) {
      float s[2] = {0.f, 0.f};
      for (int64_t i = threadIdx.x; i < a.width; i += kThreads) {
        const float t = c.t(i);
        s[0] += t;
        s[1] = fmaf(t, c.rhat(i), s[1]);
      }
      block_sum(s, red);
      c.c1 = layer ? s[0] / (float)a.width : 0.f;
      c.c2 = s[1] / (float)a.width;
    }
    float e1 = 0.f, e2 = 0.f;
    const bool post = a.y && a.post_norm;
    const auto p_at = [&](int64_t i, float D) {
      const float dz = a.branch_scale * c.gate_at(i) * D;
      return post && a.post_weight ? dz * load_as_float(a.post_weight, a.param_type, i) : dz;
    };
    if (post) {
      float s[2] = {0.f, 0.f};
      for (int64_t i = threadIdx.x; i < a.width; i += kThreads) {
        const float p = p_at(i, c.D(i));
        s[0] += p;
        s[1] = fmaf(p, c.yhat(i), s[1]);
      }
      block_sum(s, red);
      e1 = layer ? s[0] / (float)a.width : 0.f;
      e2 = s[1] / (float)a.width;
    }
    float dg[1] = {0.f};
    for (int64_t i = threadIdx.x; i < a.width; i += kThreads) {
      const float D = c.D(i);
      if (n.g.dx) static_cast<TS *>(n.g.dx)[row * a.width + i] = from_float<TS>(a.residual_scale * D);
      if (!a.y) continue;
      if (n.g.dy) {
        float p = p_at(i, D);
        if (post) p = c.yr * (p - e1 - c.yhat(i) * e2);
        static_cast<TB *>(n.g.dy)[row * a.width + i] = from_float<TB>(p);
      }
      if (n.g.dgate && a.gate_kind >= SNACK_GATE_TOKEN) {
        const float v = a.branch_scale * c.u(i) * D;
        if (a.gate_kind == SNACK_GATE_FULL)
          static_cast<TB *>(n.g.dgate)[row * a.width + i] = from_float<TB>(v);
        dg[0] += v;
      }
    }
    if (n.g.dgate && a.gate_kind == SNACK_GATE_TOKEN) {
      block_sum(dg, red);
      if (threadIdx.x == 0) static_cast<TB *>(n.g.dgate)[row] = from_float<TB>(dg[0]);
    }
    if (threadIdx.x == 0) {
      n.row_scalars[2 * row] = c.c1;
      n.row_scalars[2 * row + 1] = c.c2;
    }
  }
}

constexpr int kColThreads = 32, kRowThreads = 8;

// Column sums over one slab of rows (all of one group): block (column tile, slab).
template <typename TS, typename TB>
__global__ void __launch_bounds__(kColThreads *kRowThreads) norm_backward_columns(
    const __grid_constant__ NormArgs n) {
  __shared__ float red[kRowThreads][kColThreads + 1];
  dependency_wait();
  const snack_norm_args &a = n.a;
  const int tx = threadIdx.x % kColThreads, ty = threadIdx.x / kColThreads;
  const int64_t i = (int64_t)blockIdx.x * kColThreads + tx;
  for (int64_t slab = blockIdx.y; slab < n.slabs; slab += gridDim.y) {
    const int64_t group = slab / n.slabs_per_group, k = slab % n.slabs_per_group;
    const int64_t r0 = group * n.group_len + k * n.slab_rows;
    const int64_t r1 = min((group + 1) * n.group_len, r0 + n.slab_rows);
    float acc[kCols] = {};
    if (i < a.width)
      for (int64_t row = r0 + ty; row < r1; row += kRowThreads) {
        BackRow<TS, TB> c(n, row);
        c.c1 = n.row_scalars[2 * row];
        c.c2 = n.row_scalars[2 * row + 1];
        if (c.dh) {
          const float dh = to_float(c.dh[i]);
          acc[kNextW] = fmaf(dh, c.rhat(i), acc[kNextW]);
          acc[kNextB] += dh;
        }
        if (a.y) {
          const float D = c.D(i), dz = a.branch_scale * c.gate_at(i) * D;
          if (a.post_norm) {
            acc[kPostW] = fmaf(dz, c.yhat(i), acc[kPostW]);
            acc[kPostB] += dz;
          }
          acc[kGate] = fmaf(a.branch_scale * c.u(i), D, acc[kGate]);
        }
      }
#pragma unroll
    for (int k2 = 0; k2 < kCols; ++k2) {
      red[ty][tx] = acc[k2];
      __syncthreads();
      if (ty == 0) {
        float s = 0.f;
#pragma unroll
        for (int j = 0; j < kRowThreads; ++j) s += red[j][tx];
        if (i < a.width) n.parts[(slab * kCols + k2) * a.width + i] = s;
      }
      __syncthreads();
    }
  }
}

// The slabs' sums, added in their order.  blockIdx.y: a column array, or
// kGate + group.
__global__ void __launch_bounds__(kThreads) norm_backward_finish(const __grid_constant__ NormArgs n) {
  dependency_wait();
  const snack_norm_args &a = n.a;
  const int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  if (i >= a.width) return;
  for (int64_t what = blockIdx.y; what < kGate + n.groups; what += gridDim.y) {
    void *out = nullptr;
    int64_t s0 = 0, s1 = n.slabs, at = i;
    int k = (int)what, type = a.param_type;
    if (what == kNextW) out = n.g.dnext_weight;
    if (what == kNextB) out = n.g.dnext_bias;
    if (what == kPostW) out = n.g.dpost_weight;
    if (what == kPostB) out = n.g.dpost_bias;
    if (what >= kGate) {
      const int64_t group = what - kGate;
      k = kGate;
      out = a.gate_kind == SNACK_GATE_CHANNEL || a.gate_kind == SNACK_GATE_SEQUENCE ? n.g.dgate : nullptr;
      s0 = group * n.slabs_per_group;
      s1 = s0 + n.slabs_per_group;
      at = group * a.width + i;
      type = a.branch_type;
    }
    if (!out) continue;
    float s = 0.f;
    for (int64_t slab = s0; slab < s1; ++slab) s += n.parts[(slab * kCols + k) * a.width + i];
    store_from_float(out, type, at, s);
  }
}

bool wants_columns(const snack_norm_args &a, const snack_norm_grads &g) {
  return g.dnext_weight || g.dnext_bias || g.dpost_weight || g.dpost_bias ||
         (g.dgate && (a.gate_kind == SNACK_GATE_CHANNEL || a.gate_kind == SNACK_GATE_SEQUENCE));
}

// Rows are summed in slabs, each within one group: as many in all as there
// are teams to take them (or two rounds of the any-shape kernel's blocks).
void plan_slabs(NormArgs *n, int64_t teams) {
  const snack_norm_args &a = n->a;
  const bool seq = a.gate_kind == SNACK_GATE_SEQUENCE;
  n->groups = seq ? a.rows / a.group_rows : 1;
  n->group_len = seq ? a.group_rows : a.rows;
  int64_t want = teams / std::max<int64_t>(1, n->groups);
  if (teams == 0) {
    const int64_t tiles = (a.width + kColThreads - 1) / kColThreads;
    want = (int64_t)device_sms() * 16 / std::max<int64_t>(1, tiles * n->groups);
    want = std::min<int64_t>(want, (n->group_len + 31) / 32);
  }
  want = std::max<int64_t>(1, want);
  n->slab_rows = std::max<int64_t>(1, (n->group_len + want - 1) / want);
  n->slabs_per_group = (n->group_len + n->slab_rows - 1) / n->slab_rows;  // 0 without rows
  n->slabs = n->slabs_per_group * n->groups;
}

int64_t align16(int64_t b) { return (b + 15) / 16 * 16; }

const char *bad_args(const snack_norm_args *a) {
  if (!a) return "args is NULL";
  if (a->rows < 0 || a->width < 1 || a->width > 0x7fffffffLL) return "rows must be >= 0 and width in [1, 2^31)";
  if (a->rows > (int64_t(1) << 62) / a->width) return "rows * width is too large";
  if (a->norm_kind != SNACK_NORM_LAYER && a->norm_kind != SNACK_NORM_RMS) return "norm_kind is not one of snack_norm_kind";
  if (a->gate_kind < SNACK_GATE_NONE || a->gate_kind > SNACK_GATE_FULL) return "gate_kind is not one of snack_gate_kind";
  if (!known_type(a->stream_type) || !known_type(a->branch_type) || !known_type(a->param_type))
    return "a type is not one of snack_dtype";
  if (a->stream_type != a->branch_type && a->stream_type != SNACK_F32)
    return "stream_type must be branch_type or SNACK_F32";
  if (a->param_type != SNACK_F32 && a->param_type != a->branch_type)
    return "param_type must be SNACK_F32 or branch_type";
  if (a->gate_kind == SNACK_GATE_SEQUENCE && (a->group_rows < 1 || a->rows % a->group_rows != 0))
    return "group_rows must divide rows";
  if (!(a->eps >= 0.f)) return "eps must be >= 0";
  if (!a->post_norm && (a->post_weight || a->post_bias)) return "post_weight or post_bias without post_norm";
  if (!a->next_norm && (a->next_weight || a->next_bias)) return "next_weight or next_bias without next_norm";
  if (a->rows == 0) return nullptr;
  if (!a->x) return "x is NULL";
  if ((a->gate_kind != SNACK_GATE_NONE) && (!a->gate || !a->y)) return "a gate needs gate and y";
  if (a->post_norm && !a->y) return "post_norm needs y";
  if (a->rows > 1 && (a->x_stride < a->width || (a->y && a->y_stride < a->width) ||
                      (a->gate_kind == SNACK_GATE_FULL && a->gate_stride < a->width)))
    return "a row stride is below width";
  const int64_t ts = type_bytes(a->stream_type), tb = type_bytes(a->branch_type), tp = type_bytes(a->param_type);
  if (!aligned_to(a->x, ts) || !aligned_to(a->y, tb) || !aligned_to(a->gate, tb) ||
      !aligned_to(a->post_weight, tp) || !aligned_to(a->post_bias, tp) || !aligned_to(a->next_weight, tp) ||
      !aligned_to(a->next_bias, tp))
    return "a pointer is not aligned to its elements";
  if (a->stats && !aligned_to(a->stats, 16)) return "stats must be 16-byte aligned";
  return nullptr;
}

// Gradients of what the call does not have.
const char *bad_grads(const snack_norm_args &a, const snack_norm_grads &g) {
  if (!a.post_norm && (g.dpost_weight || g.dpost_bias)) return "dpost_weight or dpost_bias without post_norm";
  if (!a.next_norm && (g.dh || g.dnext_weight || g.dnext_bias)) return "dh, dnext_weight or dnext_bias without next_norm";
  if (a.gate_kind == SNACK_GATE_NONE && g.dgate) return "dgate without a gate";
  if (a.rows > 0 && !a.y && g.dy) return "dy without y";
  return nullptr;
}

cudaError_t launch_forward(const NormArgs &n, cudaStream_t s) {
  const snack_norm_args &a = n.a;
  const int64_t grid = std::min<int64_t>(a.rows, (int64_t)device_sms() * 8);
#define SNACK_CALL(TS, TB) return launch_kernel(norm_forward_rows<TS, TB>, dim3((unsigned)grid), kThreads, 0, true, s, n);
  SNACK_NORM_TYPES(SNACK_CALL)
#undef SNACK_CALL
}

cudaError_t launch_backward_rows(const NormArgs &n, cudaStream_t s) {
  const snack_norm_args &a = n.a;
  const int64_t grid = std::min<int64_t>(a.rows, (int64_t)device_sms() * 8);
#define SNACK_CALL(TS, TB) return launch_kernel(norm_backward_rows<TS, TB>, dim3((unsigned)grid), kThreads, 0, true, s, n);
  SNACK_NORM_TYPES(SNACK_CALL)
#undef SNACK_CALL
}

cudaError_t launch_backward_columns(const NormArgs &n, cudaStream_t s) {
  const snack_norm_args &a = n.a;
  const dim3 grid((unsigned)((a.width + kColThreads - 1) / kColThreads), (unsigned)std::min<int64_t>(n.slabs, 65535));
#define SNACK_CALL(TS, TB) return launch_kernel(norm_backward_columns<TS, TB>, grid, kColThreads * kRowThreads, 0, true, s, n);
  SNACK_NORM_TYPES(SNACK_CALL)
#undef SNACK_CALL
}

cudaError_t launch_backward_finish(const NormArgs &n, cudaStream_t s) {
  const dim3 grid((unsigned)((n.a.width + kThreads - 1) / kThreads),
                  (unsigned)std::min<int64_t>(kGate + n.groups, 65535));
  return launch_kernel(norm_backward_finish, grid, kThreads, 0, true, s, n);
}

}  // namespace
}  // namespace snack

extern "C" snack_status snack_residual_norm_forward(const snack_norm_args *args, void *r, void *h,
                                                    void *stream) {
  using namespace snack;
  if (const char *bad = bad_args(args)) return refuse(SNACK_ERR_INVALID_ARG, bad);
  if (args->rows == 0) return SNACK_OK;
  if (args->next_norm && !h) return refuse(SNACK_ERR_INVALID_ARG, "h is NULL");
  if (!aligned_to(r, type_bytes(args->stream_type)) || !aligned_to(h, type_bytes(args->branch_type)))
    return refuse(SNACK_ERR_INVALID_ARG, "a pointer is not aligned to its elements");
  NormArgs n = {};
  n.a = *args;
  n.r = r;
  n.h = h;
  const TeamPlan p = team_forward(n);
  plan_slabs(&n, p.teams);
  const cudaError_t e = p.threads ? launch_team_forward(n, p, static_cast<cudaStream_t>(stream))
                                  : launch_forward(n, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? SNACK_OK : cuda_status(e, "residual norm launch");
}

extern "C" size_t snack_residual_norm_workspace(const snack_norm_args *args) {
  using namespace snack;
  if (bad_args(args)) return 16;
  // enough for either way of summing the columns, whatever the gradients' alignment
  NormArgs n = {};
  n.a = *args;
  plan_slabs(&n, 0);
  int64_t floats = n.slabs * kCols;
  const TeamPlan p = team_backward(n);
  if (p.threads) {
    plan_slabs(&n, p.teams);
    floats = std::max(floats, 2 * (p.teams + n.slabs));
  }
  return (size_t)(align16(args->rows * 8) + floats * args->width * 4 + 16);
}

extern "C" snack_status snack_residual_norm_backward(const snack_norm_args *args,
                                                     const snack_norm_grads *grads, void *workspace,
                                                     void *stream) {
  using namespace snack;
  if (const char *bad = bad_args(args)) return refuse(SNACK_ERR_INVALID_ARG, bad);
  if (!grads) return refuse(SNACK_ERR_INVALID_ARG, "grads is NULL");
  if (const char *bad = bad_grads(*args, *grads)) return refuse(SNACK_ERR_INVALID_ARG, bad);
  const snack_norm_args &a = *args;
  const snack_norm_grads &g = *grads;
  const int64_t ts = type_bytes(a.stream_type), tb = type_bytes(a.branch_type), tp = type_bytes(a.param_type);
  if (!workspace || !aligned_to(workspace, 16))
    return refuse(SNACK_ERR_INVALID_ARG, "workspace must be 16-byte aligned device memory");
  if (a.rows > 0 && !a.stats) return refuse(SNACK_ERR_INVALID_ARG, "stats is NULL");
  if (a.rows > 1 && ((g.dr && g.dr_stride < a.width) || (g.dh && g.dh_stride < a.width)))
    return refuse(SNACK_ERR_INVALID_ARG, "a row stride is below width");
  if (!aligned_to(g.dr, ts) || !aligned_to(g.dh, tb) || !aligned_to(g.dx, ts) || !aligned_to(g.dy, tb) ||
      !aligned_to(g.dgate, tb) || !aligned_to(g.dpost_weight, tp) || !aligned_to(g.dpost_bias, tp) ||
      !aligned_to(g.dnext_weight, tp) || !aligned_to(g.dnext_bias, tp))
    return refuse(SNACK_ERR_INVALID_ARG, "a pointer is not aligned to its elements");
  NormArgs n = {};
  n.a = a;
  n.g = g;
  const TeamPlan p = team_backward(n);
  plan_slabs(&n, p.teams);
  n.row_scalars = static_cast<float *>(workspace);
  n.parts = reinterpret_cast<float *>(static_cast<char *>(workspace) + align16(a.rows * 8));
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e = cudaSuccess;
  if (p.threads && a.rows > 0) {
    e = launch_team_backward(n, p, s);
    return e == cudaSuccess ? SNACK_OK : cuda_status(e, "residual norm backward launch");
  }
  if (a.rows > 0 && (e = launch_backward_rows(n, s)) != cudaSuccess)
    return cuda_status(e, "residual norm backward launch");
  if (wants_columns(a, g)) {
    if (a.rows > 0 && (e = launch_backward_columns(n, s)) != cudaSuccess)
      return cuda_status(e, "residual norm column sums launch");
    if ((e = launch_backward_finish(n, s)) != cudaSuccess)
      return cuda_status(e, "residual norm column sums launch");
  }
  return SNACK_OK;
}
