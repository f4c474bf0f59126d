// Residual norm backward, rows held in registers (norm_team.cuh).
//
// The column sums (the gradients of weights, biases and shared gates) stay
// in the registers of the threads that hold the columns, over all of a
// team's rows, and leave once per team.  Those kept are  sum dh rhat, sum dh,
// sum G D yhat, sum G D, with G = 1 where the gate belongs to the column
// (then it is a factor of the whole sum and is multiplied in at the end) and
// the gate itself where it belongs to the row:
//   dw_post = b sum g D yhat,  db_post = b sum g D,
//   dg = b (w_post sum D yhat + b_post sum D).
#include "norm_team.cuh"

namespace snack {
namespace {

using namespace team;

// The teams of a block take slabs of rows, each within one group, row by row
// in turn; sum dh rhat and sum dh leave once per block, sum G D yhat and sum
// G D once per slab.
template <typename TS, typename TB, int S, bool VEC, bool CL, bool LAYER, Form F>
__global__ void __launch_bounds__(kTeamThreads) norm_team_backward(const __grid_constant__ TeamArgs q) {
  extern __shared__ uint4 smem4[];
  __shared__ float red[Team<CL, !CL>::kFloats];
  const snack_norm_args &a = q.n.a;
  const snack_norm_grads &g = q.n.g;
  dependency_wait();
  dependency_launch();
  Team<CL, !CL> team = make_team<CL, !CL>(red, q.threads);
  const Columns<TS, TB, VEC> co(q, team.rank, (int)threadIdx.x - team.index() * q.threads, q.threads);
  const int per_block = (int)blockDim.x / q.threads;
  const int64_t me = blockIdx.x / team.size, teams = gridDim.x / team.size;
  const bool has_y = F || a.y, post = F ? F == kFastPost : has_y && a.post_norm;
  const bool full = !F && a.gate_kind == SNACK_GATE_FULL, token = !F && a.gate_kind == SNACK_GATE_TOKEN;
  const bool has_dh = F || (g.dh && a.next_norm), has_dr = F || g.dr, want_dx = F || g.dx, want_dy = F || g.dy;
  // a bias: the layer norms' own, or one given to an rms norm
  const bool post_bias = LAYER || (!F && a.post_bias);
  const bool dbias = LAYER || (!F && (g.dnext_bias || g.dpost_bias || a.post_bias));
  const int xb = row_bytes<TS, VEC>(q, q.threads), bb = row_bytes<TB, VEC>(q, q.threads), per = 2 * xb + (2 + (full ? 1 : 0)) * bb;
  const float inv = 1.f / (float)a.width;
  char *const whole = reinterpret_cast<char *>(smem4), *const ring = whole + team.index() * S * per;
  if (VEC && co.count < q.threads * C) clear_slots(whole, per_block * S * per);
  // the sums of the block's teams, added in their order through the ring
  const auto join = [&](float (&u)[C], float (&v)[C], float *out) {
    float *buf = reinterpret_cast<float *>(smem4);
    for (int k = 0; k + 1 < per_block; ++k) {
      __syncthreads();
      if (team.index() == k)
#pragma unroll
        for (int j = 0; j < C; ++j) {
          float *at = buf + (j * q.threads + co.tid) * 2;
          at[0] = u[j];
          at[1] = v[j];
        }
      __syncthreads();
      if (team.index() == k + 1)
#pragma unroll
        for (int j = 0; j < C; ++j) {
          const float *at = buf + (j * q.threads + co.tid) * 2;
          u[j] += at[0];
          v[j] += at[1];
        }
    }
    if (team.index() == per_block - 1)
#pragma unroll
      for (int j = 0; j < C; ++j)
        if (co.in(j)) {
          out[co.at(j)] = u[j];
          out[a.width + co.at(j)] = v[j];
        }
    __syncthreads();  // the ring is the rows' again
    if (VEC && per_block > 1 && co.count < q.threads * C) clear_slots(whole, per_block * S * per);
  };

  const auto x_row = [&](int64_t r) { return static_cast<const TS *>(a.x) + r * a.x_stride; };
  const auto y_row = [&](int64_t r) { return static_cast<const TB *>(a.y) + r * a.y_stride; };
  const auto dr_row = [&](int64_t r) { return static_cast<const TS *>(g.dr) + r * g.dr_stride; };
  const auto dh_row = [&](int64_t r) { return static_cast<const TB *>(g.dh) + r * g.dh_stride; };
  const auto fetch = [&](int64_t row, int64_t end, int stage) {
    if (row < end) {
      char *to = ring + stage * per;
      copy_row<TS, VEC>(to, x_row(row), co);
      if (has_dr) copy_row<TS, VEC>(to + xb, dr_row(row), co);
      to += 2 * xb;
      if (has_y) copy_row<TB, VEC>(to, y_row(row), co);
      if (has_dh) copy_row<TB, VEC>(to + bb, dh_row(row), co);
      if (full) copy_row<TB, VEC>(to + 2 * bb, gate_row<TB>(a, row), co);
    }
    copies_commit();
  };

  float nw[C], k1[C], k0[C];  // next weight; b g w_post and b g b_post (without a gate that belongs to the row)
  float s0[C], s1[C];         // sum dh rhat, sum dh
  load_params(a.next_weight, a.param_type, co, 1.f, nw);
#pragma unroll
  for (int j = 0; j < C; ++j) s0[j] = s1[j] = 0.f;

  for (int64_t slab = me; slab < q.n.slabs; slab += teams) {
    // every step-th row of the group: all teams together sweep the rows in
    // their order
    const int64_t spg = q.n.slabs_per_group, step = spg * per_block, group = slab / spg;
    const int64_t r0 = group * q.n.group_len + slab % spg + team.index() * spg, r1 = (group + 1) * q.n.group_len;
    if (!VEC) team.barrier();  // the slab before has been read by all
#pragma unroll
    for (int i = 0; i < S - 1; ++i) fetch(r0 + i * step, r1, i);
    if (has_y) {
      load_params(a.post_weight, a.param_type, co, 1.f, k1);
      load_params(a.post_bias, a.param_type, co, 0.f, k0);
#pragma unroll
      for (int j = 0; j < C; ++j) {
        float f = a.branch_scale;
        if (a.gate_kind == SNACK_GATE_CHANNEL || a.gate_kind == SNACK_GATE_SEQUENCE)
          f *= co.in(j) ? to_float(gate_row<TB>(a, group * q.n.group_len)[co.at(j)]) : 0.f;
        k1[j] *= f;
        k0[j] *= f;
      }
    }
    float s2[C], s3[C];  // sum G D yhat, sum G D
#pragma unroll
    for (int j = 0; j < C; ++j) s2[j] = s3[j] = 0.f;

    int stage = 0;
    float4 st = r0 < r1 ? reinterpret_cast<const float4 *>(a.stats)[r0] : make_float4(0.f, 0.f, 0.f, 0.f);
    for (int64_t row = r0; row < r1; row += step) {
      // A column beyond the row holds zeros and zero parameters: whatever
      // its hats are, it adds 0 to the row's sums, and nothing of it is stored.
      float rh[C], D[C], yh[C], gate[C];
      const float ym = st.x, yr = st.y, mean = st.z, rstd = st.w;
      copies_wait<S - 2>();
      if (!VEC) team.barrier();
      const char *from = ring + stage * per;
      take_row<TS, VEC>(from, x_row(row), co, rh);
      if (row + step < r1) st = reinterpret_cast<const float4 *>(a.stats)[row + step];
      const float tg = token ? to_float(static_cast<const TB *>(a.gate)[row]) : 1.f;
      if (full) take_row<TB, VEC>(from + 2 * xb + 2 * bb, gate_row<TB>(a, row), co, gate);
      if (has_y) {
        take_row<TB, VEC>(from + 2 * xb, y_row(row), co, yh);
#pragma unroll
        for (int j = 0; j < C; ++j) {
          if (post) yh[j] = (LAYER ? yh[j] - ym : yh[j]) * yr;
          float u = post_bias ? fmaf(k1[j], yh[j], k0[j]) : k1[j] * yh[j];
          if (full) u *= gate[j];
          if (token) u *= tg;
          rh[j] = fmaf(a.residual_scale, rh[j], u);
        }
      } else {
#pragma unroll
        for (int j = 0; j < C; ++j) rh[j] *= a.residual_scale;
      }
      float c[2] = {0.f, 0.f};
      if (has_dh) {
        take_row<TB, VEC>(from + 2 * xb + bb, dh_row(row), co, D);
#pragma unroll
        for (int j = 0; j < C; ++j) {
          rh[j] = (LAYER ? rh[j] - mean : rh[j]) * rstd;
          s0[j] = fmaf(D[j], rh[j], s0[j]);
          if (dbias) s1[j] += D[j];
          D[j] *= nw[j];
          if (LAYER) c[0] += D[j];
          c[1] = fmaf(D[j], rh[j], c[1]);
        }
        if (LAYER) {
          team.sum(c);
        } else {
          float c1[1] = {c[1]};
          team.sum(c1);
          c[1] = c1[0];
        }
        const float m1 = c[0] * inv, m2 = c[1] * inv;
#pragma unroll
        for (int j = 0; j < C; ++j) D[j] = fmaf(-rh[j], m2, LAYER ? D[j] - m1 : D[j]);
      } else {
#pragma unroll
        for (int j = 0; j < C; ++j) D[j] = 0.f;
      }
      if (has_dr) {
        take_row<TS, VEC>(from + xb, dr_row(row), co, rh);  // rhat is done with
#pragma unroll
        for (int j = 0; j < C; ++j) D[j] = fmaf(D[j], rstd, rh[j]);
      } else {
#pragma unroll
        for (int j = 0; j < C; ++j) D[j] *= rstd;
      }
      // vectors: into the slots that this thread read for the row before; else
      // all have read that row, for they have passed this row's barrier
      fetch(row + (S - 1) * step, r1, stage == 0 ? S - 1 : stage - 1);
      stage = stage == S - 1 ? 0 : stage + 1;
      if (want_dx) {
        float v[C];
#pragma unroll
        for (int j = 0; j < C; ++j) v[j] = a.residual_scale * D[j];
        store_row<TS, VEC>(static_cast<TS *>(g.dx) + row * a.width, co, v);
      }
      if (!has_y) continue;
      float dg = 0.f;
      if ((full || token) && g.dgate) {
        float u[C], w[C];
        load_params(a.post_weight, a.param_type, co, 1.f, w);
        load_params(a.post_bias, a.param_type, co, 0.f, u);
#pragma unroll
        for (int j = 0; j < C; ++j) {
          u[j] = a.branch_scale * fmaf(yh[j], w[j], u[j]) * D[j];
          dg += u[j];
        }
        if (full) store_row<TB, VEC>(static_cast<TB *>(g.dgate) + row * a.width, co, u);
      }
      float e[2] = {0.f, 0.f};
#pragma unroll
      for (int j = 0; j < C; ++j) {
        if (full) D[j] *= gate[j];
        if (token) D[j] *= tg;
        s2[j] = fmaf(D[j], yh[j], s2[j]);
        if (dbias) s3[j] += D[j];
        D[j] *= k1[j];
        if (LAYER) e[0] += D[j];
        e[1] = fmaf(D[j], yh[j], e[1]);
      }
      if (token && g.dgate) {
        float all[3] = {e[0], e[1], dg};
        team.sum(all);
        e[0] = all[0];
        e[1] = all[1];
        if (team.rank == 0 && co.tid == 0) static_cast<TB *>(g.dgate)[row] = from_float<TB>(all[2]);
      } else if (post) {
        if (LAYER) {
          team.sum(e);
        } else {
          float e1[1] = {e[1]};
          team.sum(e1);
          e[1] = e1[0];
        }
      }
      if (want_dy) {
        if (post) {
          const float m1 = LAYER ? e[0] * inv : 0.f, m2 = e[1] * inv;
#pragma unroll
          for (int j = 0; j < C; ++j) D[j] = yr * fmaf(-yh[j], m2, LAYER ? D[j] - m1 : D[j]);
        }
        store_row<TB, VEC>(static_cast<TB *>(g.dy) + row * a.width, co, D);
      }
    }
    copies_wait<0>();
    if (q.post_parts) join(s2, s3, q.post_parts + slab * 2 * a.width);
  }
  if (q.next_parts) join(s0, s1, q.next_parts + me * 2 * a.width);
  if (CL) cg::this_cluster().sync();
}

// The parts, added in their order.  blockIdx.y: 0 next weight and bias, 1
// post weight and bias (and a channel gate, which has the same sums), 2 +
// group: a sequence's gate.
constexpr int kFinX = 32, kFinY = 32;
template <typename TB>
__global__ void __launch_bounds__(kFinX *kFinY) norm_team_finish(const __grid_constant__ TeamArgs q, int teams) {
  __shared__ float red[2][kFinY][kFinX + 1];
  dependency_wait();
  dependency_launch();
  const snack_norm_args &a = q.n.a;
  const snack_norm_grads &g = q.n.g;
  const int tx = threadIdx.x % kFinX, ty = threadIdx.x / kFinX;
  const int64_t i = (int64_t)blockIdx.x * kFinX + tx;
  const bool seq = a.gate_kind == SNACK_GATE_SEQUENCE, channel = a.gate_kind == SNACK_GATE_CHANNEL;
  const TB *gate = static_cast<const TB *>(a.gate);
  const int spg = (int)q.n.slabs_per_group;
  for (int64_t what = blockIdx.y; what < 2 + q.n.groups; what += gridDim.y) {
    const float *parts = what == 0 ? q.next_parts : q.post_parts;
    int64_t p0 = 0, p1 = what == 0 ? teams : q.n.slabs;
    if (what >= 2) {
      p0 = (what - 2) * spg;
      p1 = p0 + spg;
    }
    if (!parts || (what >= 2 && !(g.dgate && seq))) continue;
    float v[2] = {0.f, 0.f};
    if (i < a.width) {
#pragma unroll 8
      for (int64_t p = p0 + ty; p < p1; p += kFinY) {
        const float f = what == 1 && seq ? to_float(gate[(int)p / spg * a.width + i]) : 1.f;
        v[0] = fmaf(f, parts[p * 2 * a.width + i], v[0]);
        v[1] = fmaf(f, parts[p * 2 * a.width + a.width + i], v[1]);
      }
    }
    red[0][ty][tx] = v[0];
    red[1][ty][tx] = v[1];
    __syncthreads();
    // warp w sums one of the two for columns w, w + 16: all of a column's
    // rows lie in the warp's lanes
    {
      const int w = ty, lane = tx, which = w & 1;
      for (int c = w >> 1; c < kFinX; c += kFinY / 2) {
        const float s = warp_sum(red[which][lane][c]);
        if (lane == 0) red[which][0][c] = s;  // lane 0 read its own value before
      }
    }
    __syncthreads();
    if (ty == 0 && i < a.width) {
      v[0] = red[0][0][tx];
      v[1] = red[1][0][tx];
      const float w = a.post_weight ? load_as_float(a.post_weight, a.param_type, i) : 1.f;
      const float b = a.post_bias ? load_as_float(a.post_bias, a.param_type, i) : 0.f;
      const float dgate = a.branch_scale * fmaf(w, v[0], b * v[1]);
      if (what == 0) {
        if (g.dnext_weight) store_from_float(g.dnext_weight, a.param_type, i, v[0]);
        if (g.dnext_bias) store_from_float(g.dnext_bias, a.param_type, i, v[1]);
      } else if (what == 1) {
        const float f = a.branch_scale * (channel ? to_float(gate[i]) : 1.f);
        if (g.dpost_weight) store_from_float(g.dpost_weight, a.param_type, i, f * v[0]);
        if (g.dpost_bias) store_from_float(g.dpost_bias, a.param_type, i, f * v[1]);
        if (g.dgate && channel) static_cast<TB *>(g.dgate)[i] = from_float<TB>(dgate);
      } else {
        static_cast<TB *>(g.dgate)[(what - 2) * a.width + i] = from_float<TB>(dgate);
      }
    }
    __syncthreads();
  }
}

template <typename TS, typename TB>
cudaError_t launch(const TeamPlan &p, int64_t teams, const TeamArgs &q, Form form, cudaStream_t s) {
  SNACK_TEAM(norm_team_backward, TS, TB)
}

}  // namespace

// One team for every two rows, at most what 512 threads of 128 registers on
// each SM hold at once; on each SM they are one block, which leaves one part
// of the column sums (a part for each of 585 teams of 128 threads, 4095 x
// 1001: 9 MB, and 14 us to add them up).
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
  const int64_t sms = device_sms(), fit = kTeamThreads / p.threads;
  const int64_t group = a.gate_kind == SNACK_GATE_SEQUENCE ? a.group_rows : a.rows;  // rows that a block's teams share
  const int64_t teams = std::max<int64_t>(1, std::min<int64_t>((a.rows + 1) / 2, std::max<int64_t>(1, sms * fit / p.cluster)));
  if (p.cluster == 1) p.per_block = (int)std::max<int64_t>(1, std::min(std::min(fit, teams / sms), group));
  team_ring(&p, a, 2, full ? 3 : 2);
  p.teams = (teams + p.per_block - 1) / p.per_block;
  return p;
}

cudaError_t launch_team_backward(const NormArgs &n, const TeamPlan &p, cudaStream_t s) {
  const snack_norm_args &a = n.a;
  const snack_norm_grads &g = n.g;
  TeamArgs q = {n, p.block_cols, p.threads, nullptr, nullptr};
  const bool seq = a.gate_kind == SNACK_GATE_SEQUENCE;
  const bool next = g.dnext_weight || g.dnext_bias;
  const bool post = g.dpost_weight || g.dpost_bias || (g.dgate && (a.gate_kind == SNACK_GATE_CHANNEL || seq));
  const int64_t teams = std::min<int64_t>(p.teams, n.slabs);
  if (next) q.next_parts = n.parts;
  if (post) q.post_parts = n.parts + teams * 2 * a.width;
  // an rms norm's forms of their own keep no sums for biases
  const bool dbias = a.norm_kind == SNACK_NORM_RMS && (g.dnext_bias || g.dpost_bias);
  const Form form = !plain_options(a) || dbias || !g.dr || !g.dh || !g.dx || !g.dy
                        ? kAny
                        : (a.post_norm ? kFastPost : kFast);
  const auto main = [&]() -> cudaError_t {
#define SNACK_CALL(TS, TB) return launch<TS, TB>(p, teams, q, form, s);
    SNACK_NORM_TYPES(SNACK_CALL)
#undef SNACK_CALL
  };
  const cudaError_t e = main();
  if (e != cudaSuccess || !(next || post)) return e;
  const dim3 grid((unsigned)((a.width + kFinX - 1) / kFinX),
                  (unsigned)std::min<int64_t>((post ? 2 : 1) + (g.dgate && seq ? n.groups : 0), 65535));
  const auto finish = a.branch_type == SNACK_F32    ? norm_team_finish<float>
                      : a.branch_type == SNACK_BF16 ? norm_team_finish<__nv_bfloat16>
                                                    : norm_team_finish<__half>;
  return launch_kernel(finish, grid, kFinX * kFinY, 0, true, s, q, (int)teams);
}

}  // namespace snack
