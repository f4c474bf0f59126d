// Residual norm, rows held in registers: every input is read once, every
// output written once.
//
// A team of threads takes one row after another; each thread holds 8 columns
// of it, always the same ones, and so the column sums of the backward (the
// gradients of weights, biases and shared gates) stay in its registers over
// all of the team's rows and leave once per team.  Rows to come are copied
// asynchronously into slots of shared memory that only the copying thread
// reads; the team meets only for its sums.  Rows of more than 4096 columns
// are held by a cluster of blocks that exchange their sums through each
// other's shared memory.
//
// The column sums kept are  sum dh rhat, sum dh, sum G D yhat, sum G D, with
// G = 1 where the gate belongs to the column (then it is a factor of the
// whole sum and is multiplied in at the end) and the gate itself where it
// belongs to the row:
//   dw_post = b sum g D yhat,  db_post = b sum g D,
//   dg = b (w_post sum D yhat + b_post sum D).
#include <cooperative_groups.h>

#include <algorithm>

#include "residual_norm.cuh"

namespace snack {
namespace {

namespace cg = cooperative_groups;

constexpr int C = kTeamCols;

struct TeamArgs {
  NormArgs n;
  int block_cols;
  float *next_parts;  // [teams][2][width]
  float *post_parts;  // [slabs][2][width]
};

// Slots of 16 bytes that C elements of T take.
template <typename T>
__host__ __device__ constexpr int slots_of() { return C * (int)sizeof(T) / 16; }

// The columns of a thread: with vectors, runs of U columns a block's width
// of runs apart, else single columns a block's threads apart.
template <typename TS, typename TB, bool VEC>
struct Columns {
  static constexpr int U = sizeof(TB) == 4 ? 4 : 8;
  int64_t c0, width;  // the block's first column; columns of the row
  int64_t end;        // the block's last column + 1
  __device__ __forceinline__ Columns(const TeamArgs &q, int rank) {
    width = q.n.a.width;
    c0 = (int64_t)rank * q.block_cols;
    end = min(width, c0 + q.block_cols);
  }
  __device__ __forceinline__ int64_t at(int j) const {  // column of element j
    if (VEC) return c0 + ((j / U) * (int64_t)blockDim.x + threadIdx.x) * U + j % U;
    return c0 + (int64_t)j * blockDim.x + threadIdx.x;
  }
  __device__ __forceinline__ bool in(int j) const { return at(j) < end; }
};

// C elements of a row from memory (no vectors) ...
template <typename T, typename CO>
__device__ __forceinline__ void load_plain(const T *row, const CO &co, float (&v)[C]) {
  T raw[C];
#pragma unroll
  for (int j = 0; j < C; ++j) raw[j] = co.in(j) ? row[co.at(j)] : from_float<T>(0.f);
#pragma unroll
  for (int j = 0; j < C; ++j) v[j] = to_float(raw[j]);
}

// ... copied ahead into the thread's slots (`slot` apart by `step`) ...
template <typename T, typename CO>
__device__ __forceinline__ void copy_row(uint4 *slot, int step, const T *row, const CO &co) {
  constexpr int E = 16 / sizeof(T);
#pragma unroll
  for (int k = 0; k < slots_of<T>(); ++k)
    if (co.in(k * E)) copy_async16(slot + k * step, row + co.at(k * E));
}

// ... and taken from there.
template <typename T>
__device__ __forceinline__ void take_row(const uint4 *slot, int step, float (&v)[C]) {
  constexpr int E = 16 / sizeof(T);
#pragma unroll
  for (int k = 0; k < slots_of<T>(); ++k) {
    const uint4 raw = slot[k * step];
#pragma unroll
    for (int e = 0; e < E; ++e) v[k * E + e] = to_float(reinterpret_cast<const T *>(&raw)[e]);
  }
}

template <typename T, bool VEC, typename CO>
__device__ __forceinline__ void store_row(T *row, const CO &co, const float (&v)[C]) {
  if (VEC) {
    constexpr int E = 16 / sizeof(T);
#pragma unroll
    for (int k = 0; k < slots_of<T>(); ++k) {
      if (!co.in(k * E)) continue;
      uint4 raw;
#pragma unroll
      for (int e = 0; e < E; ++e) reinterpret_cast<T *>(&raw)[e] = from_float<T>(v[k * E + e]);
      *reinterpret_cast<uint4 *>(row + co.at(k * E)) = raw;
    }
  } else {
#pragma unroll
    for (int j = 0; j < C; ++j)
      if (co.in(j)) row[co.at(j)] = from_float<T>(v[j]);
  }
}

// Parameters of the thread's columns (`other` where there is no vector).
template <typename CO>
__device__ __forceinline__ void load_params(const void *p, int type, const CO &co, float other, float (&v)[C]) {
#pragma unroll
  for (int j = 0; j < C; ++j) v[j] = p && co.in(j) ? load_as_float(p, type, co.at(j)) : other;
}

// Sums over the team.  One barrier each: consecutive sums use alternate
// halves of `red`, [2][N * cluster * 16] floats.
template <bool CL>
struct Team {
  float *red;
  int flip = 0;
  int rank = 0, size = 1;
  static constexpr int kFloats = 2 * 3 * kTeamCluster * 16;

  template <int N>
  __device__ __forceinline__ void sum(float (&v)[N]) {
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, nw = blockDim.x >> 5;
#pragma unroll
    for (int k = 0; k < N; ++k) v[k] = warp_sum(v[k]);
    if (!CL && nw == 1) return;
    float *buf = red + flip * (kFloats / 2);
    flip ^= 1;
    const int all = nw * size;
    if (CL) {
      // every warp's sums to every block of the team
      cg::cluster_group cl = cg::this_cluster();
      if (lane < size) {
        float *to = cl.map_shared_rank(buf, lane);
#pragma unroll
        for (int k = 0; k < N; ++k) to[k * all + rank * nw + w] = v[k];
      }
      cl.sync();
    } else {
      if (lane == 0)
#pragma unroll
        for (int k = 0; k < N; ++k) buf[k * all + w] = v[k];
      __syncthreads();
    }
#pragma unroll
    for (int k = 0; k < N; ++k) {
      float s = 0.f;
      for (int i = lane; i < all; i += 32) s += buf[k * all + i];
      v[k] = warp_sum(s);
    }
  }

  // Mean and 1/deviation of the row.
  template <typename CO>
  __device__ __forceinline__ void stats(const snack_norm_args &a, const CO &co, const float (&v)[C], float &mean,
                                        float &rstd) {
    const float inv = 1.f / (float)a.width;
    float s[1] = {0.f};
    mean = 0.f;
    if (a.norm_kind == SNACK_NORM_LAYER) {
#pragma unroll
      for (int j = 0; j < C; ++j) s[0] += v[j];  // 0 beyond the row
      sum(s);
      mean = s[0] * inv;
      s[0] = 0.f;
    }
#pragma unroll
    for (int j = 0; j < C; ++j) {
      const float d = co.in(j) ? v[j] - mean : 0.f;
      s[0] = fmaf(d, d, s[0]);
    }
    sum(s);
    rstd = 1.f / sqrtf(fmaf(s[0], inv, a.eps));
  }
};

template <bool CL>
__device__ __forceinline__ Team<CL> make_team(float *red) {
  Team<CL> t;
  t.red = red;
  if (CL) {
    cg::cluster_group cl = cg::this_cluster();
    t.rank = (int)cl.block_rank();
    t.size = (int)cl.num_blocks();
    cl.sync();  // the team's blocks are all there before one writes to another
  }
  return t;
}

// The gate's vector for a row, or null where the gate is one number.
template <typename TB>
__device__ __forceinline__ const TB *gate_row(const snack_norm_args &a, int64_t row) {
  const TB *g = static_cast<const TB *>(a.gate);
  if (a.gate_kind == SNACK_GATE_CHANNEL) return g;
  if (a.gate_kind == SNACK_GATE_SEQUENCE) return g + (row / a.group_rows) * a.width;
  if (a.gate_kind == SNACK_GATE_FULL) return g + row * a.gate_stride;
  return nullptr;
}

template <typename TS, typename TB, int S, bool VEC, bool CL>
__global__ void __launch_bounds__(kTeamThreads) norm_team_forward(const __grid_constant__ TeamArgs q) {
  extern __shared__ uint4 smem4[];
  __shared__ float red[Team<CL>::kFloats];
  const snack_norm_args &a = q.n.a;
  dependency_wait();
  dependency_launch();
  Team<CL> team = make_team<CL>(red);
  const Columns<TS, TB, VEC> co(q, team.rank);
  const int64_t first = blockIdx.x / team.size, step = gridDim.x / team.size;
  constexpr int XS = slots_of<TS>(), BS = slots_of<TB>();
  const int threads = blockDim.x;
  const bool has_y = a.y != nullptr, full = a.gate_kind == SNACK_GATE_FULL;
  const int per = XS + BS + (full ? BS : 0);  // slots of a row
  uint4 *const mine = smem4 + threadIdx.x;

  const auto fetch = [&](int64_t row, int stage) {
    if (!VEC) return;
    if (row < a.rows) {
      uint4 *slot = mine + stage * per * threads;
      copy_row(slot, threads, static_cast<const TS *>(a.x) + row * a.x_stride, co);
      if (has_y) copy_row(slot + XS * threads, threads, static_cast<const TB *>(a.y) + row * a.y_stride, co);
      if (full) copy_row(slot + (XS + BS) * threads, threads, gate_row<TB>(a, row), co);
    }
    copies_commit();
  };
#pragma unroll
  for (int i = 0; i < S - 1; ++i) fetch(first + i * step, i);

  float nw[C], nb[C], pw[C], pb[C];
  load_params(a.next_weight, a.param_type, co, 1.f, nw);
  load_params(a.next_bias, a.param_type, co, 0.f, nb);
  load_params(a.post_weight, a.param_type, co, 1.f, pw);
  load_params(a.post_bias, a.param_type, co, 0.f, pb);
  float gate[C];
#pragma unroll
  for (int j = 0; j < C; ++j) gate[j] = 1.f;
  if (a.gate_kind == SNACK_GATE_CHANNEL) load_plain(gate_row<TB>(a, 0), co, gate);

  int stage = 0;
  int64_t group = -1;
  for (int64_t row = first; row < a.rows; row += step) {
    float x[C], y[C];
    if (VEC) {
      copies_wait<S - 2>();
      const uint4 *slot = mine + stage * per * threads;
      take_row<TS>(slot, threads, x);
      if (has_y) take_row<TB>(slot + XS * threads, threads, y);
      if (full) take_row<TB>(slot + (XS + BS) * threads, threads, gate);
      fetch(row + (S - 1) * step, stage == 0 ? S - 1 : stage - 1);
      stage = stage == S - 1 ? 0 : stage + 1;
    } else {
      load_plain(static_cast<const TS *>(a.x) + row * a.x_stride, co, x);
      if (has_y) load_plain(static_cast<const TB *>(a.y) + row * a.y_stride, co, y);
      if (full) load_plain(gate_row<TB>(a, row), co, gate);
    }
    if (VEC) {  // slots beyond the row were never written
#pragma unroll
      for (int j = 0; j < C; ++j) {
        x[j] = co.in(j) ? x[j] : 0.f;
        if (has_y) y[j] = co.in(j) ? y[j] : 0.f;
      }
    }
    if (a.gate_kind == SNACK_GATE_SEQUENCE && row / a.group_rows != group) {
      group = row / a.group_rows;
      load_plain(gate_row<TB>(a, row), co, gate);
    }
    float ym = 0.f, yr = 1.f, mean = 0.f, rstd = 1.f;
    if (has_y) {
      if (a.post_norm) team.stats(a, co, y, ym, yr);
      const float b = a.branch_scale * (a.gate_kind == SNACK_GATE_TOKEN
                                            ? to_float(static_cast<const TB *>(a.gate)[row])
                                            : 1.f);
#pragma unroll
      for (int j = 0; j < C; ++j) {
        const float u = fmaf((y[j] - ym) * yr, pw[j], pb[j]);
        x[j] = co.in(j) ? fmaf(b * gate[j], u, a.residual_scale * x[j]) : 0.f;
      }
    } else {
#pragma unroll
      for (int j = 0; j < C; ++j) x[j] *= a.residual_scale;
    }
    if (q.n.r) store_row<TS, VEC>(static_cast<TS *>(q.n.r) + row * a.width, co, x);
    if (a.next_norm) {
      team.stats(a, co, x, mean, rstd);
#pragma unroll
      for (int j = 0; j < C; ++j) x[j] = fmaf((x[j] - mean) * rstd, nw[j], nb[j]);
      store_row<TB, VEC>(static_cast<TB *>(q.n.h) + row * a.width, co, x);
    }
    if (a.stats && team.rank == 0 && threadIdx.x == 0)
      reinterpret_cast<float4 *>(a.stats)[row] = make_float4(ym, yr, mean, rstd);
  }
  copies_wait<0>();
  if (CL) cg::this_cluster().sync();  // no block leaves while another may still write to it
}

// A team takes slabs of rows, each within one group; sum dh rhat and sum dh
// leave once per team, sum G D yhat and sum G D once per slab.
template <typename TS, typename TB, int S, bool VEC, bool CL>
__global__ void __launch_bounds__(kTeamThreads) norm_team_backward(const __grid_constant__ TeamArgs q) {
  extern __shared__ uint4 smem4[];
  __shared__ float red[Team<CL>::kFloats];
  const snack_norm_args &a = q.n.a;
  const snack_norm_grads &g = q.n.g;
  dependency_wait();
  dependency_launch();
  Team<CL> team = make_team<CL>(red);
  const Columns<TS, TB, VEC> co(q, team.rank);
  const int64_t me = blockIdx.x / team.size, teams = gridDim.x / team.size;
  constexpr int XS = slots_of<TS>(), BS = slots_of<TB>();
  const int threads = blockDim.x;
  const bool layer = a.norm_kind == SNACK_NORM_LAYER, has_y = a.y != nullptr, post = has_y && a.post_norm;
  const bool full = a.gate_kind == SNACK_GATE_FULL, token = a.gate_kind == SNACK_GATE_TOKEN;
  const bool has_dh = g.dh && a.next_norm, has_dr = g.dr != nullptr;
  const int per = 2 * XS + (2 + (full ? 1 : 0)) * BS;
  const float inv = 1.f / (float)a.width;
  uint4 *const mine = smem4 + threadIdx.x;

  const auto fetch = [&](int64_t row, int64_t end, int stage) {
    if (!VEC) return;
    if (row < end) {
      uint4 *slot = mine + stage * per * threads;
      copy_row(slot, threads, static_cast<const TS *>(a.x) + row * a.x_stride, co);
      if (has_dr) copy_row(slot + XS * threads, threads, static_cast<const TS *>(g.dr) + row * g.dr_stride, co);
      slot += 2 * XS * threads;
      if (has_y) copy_row(slot, threads, static_cast<const TB *>(a.y) + row * a.y_stride, co);
      if (has_dh) copy_row(slot + BS * threads, threads, static_cast<const TB *>(g.dh) + row * g.dh_stride, co);
      if (full) copy_row(slot + 2 * BS * threads, threads, gate_row<TB>(a, row), co);
    }
    copies_commit();
  };

  float nw[C], k1[C], k0[C];  // next weight; b g w_post and b g b_post (without a gate that belongs to the row)
  float s0[C], s1[C];         // sum dh rhat, sum dh
  load_params(a.next_weight, a.param_type, co, 1.f, nw);
#pragma unroll
  for (int j = 0; j < C; ++j) s0[j] = s1[j] = 0.f;

  for (int64_t slab = me; slab < q.n.slabs; slab += teams) {
    const int64_t group = slab / q.n.slabs_per_group, k = slab % q.n.slabs_per_group;
    const int64_t r0 = group * q.n.group_len + k * q.n.slab_rows;
    const int64_t r1 = min((group + 1) * q.n.group_len, r0 + q.n.slab_rows);
#pragma unroll
    for (int i = 0; i < S - 1; ++i) fetch(r0 + i, r1, i);
    if (has_y) {
      load_params(a.post_weight, a.param_type, co, 1.f, k1);
      load_params(a.post_bias, a.param_type, co, 0.f, k0);
      float gate[C];
#pragma unroll
      for (int j = 0; j < C; ++j) gate[j] = 1.f;
      if (a.gate_kind == SNACK_GATE_CHANNEL || a.gate_kind == SNACK_GATE_SEQUENCE)
        load_plain(gate_row<TB>(a, r0), co, gate);
#pragma unroll
      for (int j = 0; j < C; ++j) {
        const float bg = a.branch_scale * gate[j];
        k1[j] *= bg;
        k0[j] *= bg;
      }
    }
    float s2[C], s3[C];  // sum G D yhat, sum G D
#pragma unroll
    for (int j = 0; j < C; ++j) s2[j] = s3[j] = 0.f;

    int stage = 0;
    float4 st = r0 < r1 ? reinterpret_cast<const float4 *>(a.stats)[r0] : make_float4(0.f, 0.f, 0.f, 0.f);
    for (int64_t row = r0; row < r1; ++row) {
      // rhat, D (first t), yhat and the row's gate
      float rh[C], D[C], yh[C], dr[C], gate[C];
      const float ym = st.x, yr = st.y, mean = st.z, rstd = st.w;
      const uint4 *slot = mine + stage * per * threads;
      if (VEC) {
        copies_wait<S - 2>();
        take_row<TS>(slot, threads, rh);
        if (has_y) take_row<TB>(slot + 2 * XS * threads, threads, yh);
        if (has_dh) take_row<TB>(slot + (2 * XS + BS) * threads, threads, D);
        if (has_dr) take_row<TS>(slot + XS * threads, threads, dr);
        if (full) take_row<TB>(slot + (2 * XS + 2 * BS) * threads, threads, gate);
        fetch(row + S - 1, r1, stage == 0 ? S - 1 : stage - 1);
        stage = stage == S - 1 ? 0 : stage + 1;
      } else {
        load_plain(static_cast<const TS *>(a.x) + row * a.x_stride, co, rh);
        if (has_y) load_plain(static_cast<const TB *>(a.y) + row * a.y_stride, co, yh);
        if (has_dh) load_plain(static_cast<const TB *>(g.dh) + row * g.dh_stride, co, D);
        if (has_dr) load_plain(static_cast<const TS *>(g.dr) + row * g.dr_stride, co, dr);
        if (full) load_plain(gate_row<TB>(a, row), co, gate);
      }
      if (row + 1 < r1) st = reinterpret_cast<const float4 *>(a.stats)[row + 1];
      const float tg = token ? to_float(static_cast<const TB *>(a.gate)[row]) : 1.f;
#pragma unroll
      for (int j = 0; j < C; ++j) gate[j] = full ? (co.in(j) ? gate[j] : 0.f) : tg;
      float c[2] = {0.f, 0.f};
#pragma unroll
      for (int j = 0; j < C; ++j) {
        const bool in = co.in(j);
        float r = a.residual_scale * rh[j];
        if (has_y) {
          yh[j] = in ? (yh[j] - ym) * yr : 0.f;
          r = fmaf(gate[j], fmaf(k1[j], yh[j], k0[j]), r);
        }
        rh[j] = in ? (r - mean) * rstd : 0.f;
        if (has_dh) {
          const float dh = in ? D[j] : 0.f;
          s0[j] = fmaf(dh, rh[j], s0[j]);
          s1[j] += dh;
          D[j] = dh * nw[j];
          c[0] += D[j];
          c[1] = fmaf(D[j], rh[j], c[1]);
        }
      }
      if (has_dh) {
        team.sum(c);
        const float c1 = layer ? c[0] * inv : 0.f, c2 = c[1] * inv;
#pragma unroll
        for (int j = 0; j < C; ++j) D[j] = rstd * (D[j] - fmaf(rh[j], c2, c1));
      } else {
#pragma unroll
        for (int j = 0; j < C; ++j) D[j] = 0.f;
      }
#pragma unroll
      for (int j = 0; j < C; ++j) D[j] = co.in(j) ? D[j] + (has_dr ? dr[j] : 0.f) : 0.f;
      if (g.dx) {
        float v[C];
#pragma unroll
        for (int j = 0; j < C; ++j) v[j] = a.residual_scale * D[j];
        store_row<TS, VEC>(static_cast<TS *>(g.dx) + row * a.width, co, v);
      }
      if (!has_y) continue;
      float e[3] = {0.f, 0.f, 0.f};
      if ((full || token) && g.dgate) {
        float u[C], w[C];
        load_params(a.post_weight, a.param_type, co, 1.f, w);
        load_params(a.post_bias, a.param_type, co, 0.f, u);
#pragma unroll
        for (int j = 0; j < C; ++j) {
          u[j] = a.branch_scale * fmaf(yh[j], w[j], u[j]) * D[j];
          e[2] += u[j];
        }
        if (full) store_row<TB, VEC>(static_cast<TB *>(g.dgate) + row * a.width, co, u);
      }
#pragma unroll
      for (int j = 0; j < C; ++j) {
        D[j] *= gate[j];
        s2[j] = fmaf(D[j], yh[j], s2[j]);
        s3[j] += D[j];
        D[j] *= k1[j];
        e[0] += D[j];
        e[1] = fmaf(D[j], yh[j], e[1]);
      }
      if (post || (token && g.dgate)) {
        team.sum(e);
        if (token && g.dgate && team.rank == 0 && threadIdx.x == 0)
          static_cast<TB *>(g.dgate)[row] = from_float<TB>(e[2]);
      }
      if (g.dy) {
        if (post) {
          const float e1 = layer ? e[0] * inv : 0.f, e2 = e[1] * inv;
#pragma unroll
          for (int j = 0; j < C; ++j) D[j] = yr * (D[j] - fmaf(yh[j], e2, e1));
        }
        store_row<TB, VEC>(static_cast<TB *>(g.dy) + row * a.width, co, D);
      }
    }
    copies_wait<0>();
    if (q.post_parts) {
      float *out = q.post_parts + slab * 2 * a.width;
#pragma unroll
      for (int j = 0; j < C; ++j)
        if (co.in(j)) {
          out[co.at(j)] = s2[j];
          out[a.width + co.at(j)] = s3[j];
        }
    }
  }
  if (q.next_parts) {
    float *out = q.next_parts + me * 2 * a.width;
#pragma unroll
    for (int j = 0; j < C; ++j)
      if (co.in(j)) {
        out[co.at(j)] = s0[j];
        out[a.width + co.at(j)] = s1[j];
      }
  }
  if (CL) cg::this_cluster().sync();
}

// The parts, added in their order.  blockIdx.y: 0 next weight and bias, 1
// post weight and bias, 2 + group: the gate.
constexpr int kFinX = 32, kFinY = 16;
template <typename TB>
__global__ void __launch_bounds__(kFinX *kFinY) norm_team_finish(const __grid_constant__ TeamArgs q, int64_t teams) {
  __shared__ float red[2][kFinY][kFinX + 1];
  dependency_wait();
  dependency_launch();
  const snack_norm_args &a = q.n.a;
  const snack_norm_grads &g = q.n.g;
  const int tx = threadIdx.x % kFinX, ty = threadIdx.x / kFinX;
  const int64_t i = (int64_t)blockIdx.x * kFinX + tx;
  const bool seq = a.gate_kind == SNACK_GATE_SEQUENCE, channel = a.gate_kind == SNACK_GATE_CHANNEL;
  for (int64_t what = blockIdx.y; what < 2 + q.n.groups; what += gridDim.y) {
    const float *parts = what == 0 ? q.next_parts : q.post_parts;
    int64_t p0 = 0, p1 = what == 0 ? teams : q.n.slabs;
    if (what >= 2) {
      p0 = (what - 2) * q.n.slabs_per_group;
      p1 = p0 + q.n.slabs_per_group;
    }
    if (what == 0 && !g.dnext_weight && !g.dnext_bias) continue;
    if (what == 1 && !g.dpost_weight && !g.dpost_bias) continue;
    if (what >= 2 && !(g.dgate && (seq || channel))) continue;
    float v[2] = {0.f, 0.f};
    if (i < a.width) {
#pragma unroll 4
      for (int64_t p = p0 + ty; p < p1; p += kFinY) {
        float f = 1.f;
        if (what == 1 && seq)
          f = to_float(static_cast<const TB *>(a.gate)[(p / q.n.slabs_per_group) * a.width + i]);
        v[0] = fmaf(f, parts[p * 2 * a.width + i], v[0]);
        v[1] = fmaf(f, parts[p * 2 * a.width + a.width + i], v[1]);
      }
    }
    red[0][ty][tx] = v[0];
    red[1][ty][tx] = v[1];
    __syncthreads();
    if (ty == 0 && i < a.width) {
      v[0] = v[1] = 0.f;
#pragma unroll
      for (int k = 0; k < kFinY; ++k) {
        v[0] += red[0][k][tx];
        v[1] += red[1][k][tx];
      }
      if (what == 0) {
        if (g.dnext_weight) store_from_float(g.dnext_weight, a.param_type, i, v[0]);
        if (g.dnext_bias) store_from_float(g.dnext_bias, a.param_type, i, v[1]);
      } else if (what == 1) {
        const float f = a.branch_scale * (channel ? to_float(static_cast<const TB *>(a.gate)[i]) : 1.f);
        if (g.dpost_weight) store_from_float(g.dpost_weight, a.param_type, i, f * v[0]);
        if (g.dpost_bias) store_from_float(g.dpost_bias, a.param_type, i, f * v[1]);
      } else {
        const float w = a.post_weight ? load_as_float(a.post_weight, a.param_type, i) : 1.f;
        const float b = a.post_bias ? load_as_float(a.post_bias, a.param_type, i) : 0.f;
        static_cast<TB *>(g.dgate)[(what - 2) * a.width + i] =
            from_float<TB>(a.branch_scale * fmaf(w, v[0], b * v[1]));
      }
    }
    __syncthreads();
  }
}

bool rows16(const void *p, int64_t stride, int type) {
  return !p || (aligned_to(p, 16) && stride * type_bytes(type) % 16 == 0);
}

// The smallest team that holds a row.
TeamPlan team_shape(const snack_norm_args &a) {
  TeamPlan p;
  const int64_t most = (int64_t)kTeamThreads * kTeamCols;
  int cluster = 1;
  while (cluster < kTeamCluster && a.width > most * cluster) cluster *= 2;
  if (a.width > most * cluster) return p;
  const int64_t cols = (a.width + cluster - 1) / cluster;
  p.threads = (int)((cols + 32 * kTeamCols - 1) / (32 * kTeamCols)) * 32;
  p.cluster = cluster;
  p.block_cols = p.threads * kTeamCols;
  // a narrow remainder must not leave a block of the cluster without columns
  if ((int64_t)(cluster - 1) * p.block_cols >= a.width) p.block_cols = (int)((cols + 7) / 8 * 8);
  return p;
}

// Rows ahead: two, or one where two do not fit.
void team_ring(TeamPlan *p, int slots) {
  if (!p->vec) {
    p->stages = 2;
    p->smem = 0;
    return;
  }
  const size_t row = (size_t)slots * 16 * p->threads;
  p->stages = 3 * row <= 200 * 1024 ? 3 : 2;
  p->smem = p->stages * row;
}

template <typename K>
cudaError_t launch_team(K kern, const TeamPlan &p, int64_t teams, const TeamArgs &q, cudaStream_t s) {
  cudaError_t e = allow_smem(kern, p.smem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(teams * p.cluster));
  cfg.blockDim = dim3((unsigned)p.threads);
  cfg.dynamicSmemBytes = p.smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)p.cluster;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = p.cluster > 1 ? 2 : 1;
  e = cudaLaunchKernelEx(&cfg, kern, q);
  if (e == cudaSuccess) count_launches(1);
  return e;
}

// CALL(kernel) for the plan's variant.
#define SNACK_TEAM(KERNEL, TS, TB, CALL)                                                       \
  {                                                                                            \
    if (p.cluster > 1) {                                                                       \
      if (!p.vec) CALL((KERNEL<TS, TB, 2, false, true>))                                       \
      else if (p.stages == 3) CALL((KERNEL<TS, TB, 3, true, true>))                            \
      else CALL((KERNEL<TS, TB, 2, true, true>))                                               \
    } else {                                                                                   \
      if (!p.vec) CALL((KERNEL<TS, TB, 2, false, false>))                                      \
      else if (p.stages == 3) CALL((KERNEL<TS, TB, 3, true, false>))                           \
      else CALL((KERNEL<TS, TB, 2, true, false>))                                              \
    }                                                                                          \
  }

// Teams that the GPU holds at once: 512 threads of 128 registers on each SM.
int64_t team_limit(const TeamPlan &p) {
  return std::max<int64_t>(1, (int64_t)device_sms() * (kTeamThreads / p.threads) / p.cluster);
}

int slots_for(int type) { return C * (int)type_bytes(type) / 16; }

}  // namespace

TeamPlan team_forward(const NormArgs &n) {
  const snack_norm_args &a = n.a;
  TeamPlan p = team_shape(a);
  if (p.threads == 0) return p;
  const bool full = a.gate_kind == SNACK_GATE_FULL;
  p.vec = a.width % 8 == 0 && rows16(a.x, a.x_stride, a.stream_type) && rows16(a.y, a.y_stride, a.branch_type) &&
          (!full || rows16(a.gate, a.gate_stride, a.branch_type)) && aligned_to(n.r, 16) && aligned_to(n.h, 16);
  team_ring(&p, slots_for(a.stream_type) + (full ? 2 : 1) * slots_for(a.branch_type));
  p.teams = std::min<int64_t>(a.rows, team_limit(p));
  return p;
}

// One team for every two rows (a part of the column sums for each team, all
// read again at the end) as long as the GPU has room for them.
TeamPlan team_backward(const NormArgs &n) {
  const snack_norm_args &a = n.a;
  const snack_norm_grads &g = n.g;
  TeamPlan p = team_shape(a);
  if (p.threads == 0) return p;
  const bool full = a.gate_kind == SNACK_GATE_FULL;
  p.vec = a.width % 8 == 0 && rows16(a.x, a.x_stride, a.stream_type) && rows16(a.y, a.y_stride, a.branch_type) &&
          (!full || rows16(a.gate, a.gate_stride, a.branch_type)) && rows16(g.dr, g.dr_stride, a.stream_type) &&
          rows16(g.dh, g.dh_stride, a.branch_type) && aligned_to(g.dx, 16) && aligned_to(g.dy, 16) &&
          (!full || aligned_to(g.dgate, 16));
  team_ring(&p, 2 * slots_for(a.stream_type) + (full ? 3 : 2) * slots_for(a.branch_type));
  p.teams = std::max<int64_t>(1, std::min<int64_t>((a.rows + 1) / 2, team_limit(p)));
  return p;
}

cudaError_t launch_team_forward(const NormArgs &n, const TeamPlan &p, cudaStream_t s) {
  const snack_norm_args &a = n.a;
  const TeamArgs q = {n, p.block_cols, nullptr, nullptr};
#define SNACK_LAUNCH(K) return launch_team(K, p, p.teams, q, s);
#define SNACK_CALL(TS, TB) SNACK_TEAM(norm_team_forward, TS, TB, SNACK_LAUNCH)
  SNACK_NORM_TYPES(SNACK_CALL)
#undef SNACK_CALL
#undef SNACK_LAUNCH
}

cudaError_t launch_team_backward(const NormArgs &n, const TeamPlan &p, cudaStream_t s) {
  const snack_norm_args &a = n.a;
  const snack_norm_grads &g = n.g;
  TeamArgs q = {n, p.block_cols, nullptr, nullptr};
  const bool next = g.dnext_weight || g.dnext_bias;
  const bool post = g.dpost_weight || g.dpost_bias ||
                    (g.dgate && (a.gate_kind == SNACK_GATE_CHANNEL || a.gate_kind == SNACK_GATE_SEQUENCE));
  const int64_t teams = std::min<int64_t>(p.teams, n.slabs);
  if (next) q.next_parts = n.parts;
  if (post) q.post_parts = n.parts + teams * 2 * a.width;
  const auto main = [&]() -> cudaError_t {
#define SNACK_CALL(TS, TB) \
  { SNACK_TEAM(norm_team_backward, TS, TB, SNACK_LAUNCH2) }
#define SNACK_LAUNCH2(K) return launch_team(K, p, teams, q, s);
    SNACK_NORM_TYPES(SNACK_CALL)
#undef SNACK_CALL
#undef SNACK_LAUNCH2
  };
  const cudaError_t e = main();
  if (e != cudaSuccess || !(next || post)) return e;
  const dim3 grid((unsigned)((a.width + kFinX - 1) / kFinX),
                  (unsigned)std::min<int64_t>(2 + (post && g.dgate ? n.groups : 0), 65535));
  const auto finish = a.branch_type == SNACK_F32    ? norm_team_finish<float>
                      : a.branch_type == SNACK_BF16 ? norm_team_finish<__nv_bfloat16>
                                                    : norm_team_finish<__half>;
  return launch_kernel(finish, grid, kFinX * kFinY, 0, true, s, q, teams);
}

}  // namespace snack
