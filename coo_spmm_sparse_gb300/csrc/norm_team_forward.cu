// Residual norm forward, rows held in registers (norm_team.cuh).
#include "norm_team.cuh"

namespace snack {
namespace {

using namespace team;

template <typename TS, typename TB, int S, bool VEC, bool CL, bool LAYER, Form F>
__global__ void __launch_bounds__(kTeamThreads, 2) norm_team_forward(const __grid_constant__ TeamArgs q) {
  extern __shared__ uint4 smem4[];
  __shared__ float red[Team<CL, false>::kFloats];
  char *const ring = reinterpret_cast<char *>(smem4);
  const snack_norm_args &a = q.n.a;
  dependency_wait();
  dependency_launch();
  Team<CL, false> team = make_team<CL, false>(red, blockDim.x);
  const Columns<TS, TB, VEC> co(q, team.rank, threadIdx.x, blockDim.x);
  const int64_t me = blockIdx.x / team.size, teams = gridDim.x / team.size, step = q.n.slabs_per_group;
  const bool has_y = F || a.y, full = !F && a.gate_kind == SNACK_GATE_FULL;
  const bool token = !F && a.gate_kind == SNACK_GATE_TOKEN, post = F ? F == kFastPost : has_y && a.post_norm;
  const bool next = F || a.next_norm, has_k0 = LAYER || (!F && a.post_bias);
  const int xb = row_bytes<TS, VEC>(q, blockDim.x), bb = row_bytes<TB, VEC>(q, blockDim.x), per = xb + bb + (full ? bb : 0);
  if (VEC && co.count < (int)blockDim.x * C) clear_slots(ring, S * per);

  const auto fetch = [&](int64_t row, int64_t end, int stage) {
    if (row < end) {
      char *to = ring + stage * per;
      copy_row<TS, VEC>(to, static_cast<const TS *>(a.x) + row * a.x_stride, co);
      if (has_y) copy_row<TB, VEC>(to + xb, static_cast<const TB *>(a.y) + row * a.y_stride, co);
      if (full) copy_row<TB, VEC>(to + xb + bb, gate_row<TB>(a, row), co);
    }
    copies_commit();
  };
  // h = hat nw + nb;  r = a x + gate (hat k1 + k0), where k1 and k0 take in
  // the branch's scale and a gate that belongs to the column
  float nw[C], nb[C], k1[C], k0[C];
  load_params(a.next_weight, a.param_type, co, 1.f, nw);
  if (LAYER) load_params(a.next_bias, a.param_type, co, 0.f, nb);
  const auto fold = [&](int64_t row) {
    load_params(a.post_weight, a.param_type, co, 1.f, k1);
    if (has_k0) load_params(a.post_bias, a.param_type, co, 0.f, k0);
#pragma unroll
    for (int j = 0; j < C; ++j) {
      float f = a.branch_scale;
      if (a.gate_kind == SNACK_GATE_CHANNEL || a.gate_kind == SNACK_GATE_SEQUENCE)
        f *= co.in(j) ? to_float(gate_row<TB>(a, row)[co.at(j)]) : 0.f;
      k1[j] *= f;
      if (has_k0) k0[j] *= f;
    }
  };
  // The team's rows: every step-th of one group after another.  All teams
  // together sweep the rows in their order (each its own run of rows
  // measured the same).
  for (int64_t slab = me; slab < q.n.slabs; slab += teams) {
    const int64_t group = slab / step, first = group * q.n.group_len + slab % step, end = (group + 1) * q.n.group_len;
    if (!VEC) __syncthreads();  // the slab before has been read by all
#pragma unroll
    for (int i = 0; i < S - 1; ++i) fetch(first + i * step, end, i);
    if (has_y) fold(first);
    int stage = 0;
    for (int64_t row = first; row < end; row += step) {
      float x[C];
      float ym = 0.f, yr = 1.f, mean = 0.f, rstd = 1.f;
      copies_wait<S - 2>();
      if (!VEC) __syncthreads();
      const char *from = ring + stage * per;
      take_row<TS, VEC>(from, static_cast<const TS *>(a.x) + row * a.x_stride, co, x);
      if (has_y) {
        float y[C];
        take_row<TB, VEC>(from + xb, static_cast<const TB *>(a.y) + row * a.y_stride, co, y);
        if (post) team.template stats<LAYER>(a, co, y, ym, yr);
        const float tg = token ? to_float(static_cast<const TB *>(a.gate)[row]) : 1.f;
        float gate[C];
        if (full) take_row<TB, VEC>(from + xb + bb, gate_row<TB>(a, row), co, gate);
#pragma unroll
        for (int j = 0; j < C; ++j) {
          float u = post ? (LAYER ? y[j] - ym : y[j]) * yr : y[j];
          u = has_k0 ? fmaf(u, k1[j], k0[j]) : u * k1[j];
          if (full) u *= gate[j];
          if (token) u *= tg;
          x[j] = fmaf(a.residual_scale, x[j], u);
        }
      } else {
#pragma unroll
        for (int j = 0; j < C; ++j) x[j] *= a.residual_scale;
      }
      // vectors: into the slots that this thread read for the row before; else
      // all have read that row, for they have passed this row's barrier
      fetch(row + (S - 1) * step, end, stage == 0 ? S - 1 : stage - 1);
      stage = stage == S - 1 ? 0 : stage + 1;
      if (F || q.n.r) store_row<TS, VEC>(static_cast<TS *>(q.n.r) + row * a.width, co, x);
      if (next) {
        team.template stats<LAYER>(a, co, x, mean, rstd);
#pragma unroll
        for (int j = 0; j < C; ++j) {
          const float hat = (LAYER ? x[j] - mean : x[j]) * rstd;
          x[j] = LAYER ? fmaf(hat, nw[j], nb[j]) : hat * nw[j];
        }
        if (!F && !LAYER && a.next_bias) {
          load_params(a.next_bias, a.param_type, co, 0.f, k0);
#pragma unroll
          for (int j = 0; j < C; ++j) x[j] += k0[j];
          if (has_y && a.post_bias) fold(row);
        }
        store_row<TB, VEC>(static_cast<TB *>(q.n.h) + row * a.width, co, x);
      }
      if ((F || a.stats) && team.rank == 0 && threadIdx.x == 0)
        reinterpret_cast<float4 *>(a.stats)[row] = make_float4(ym, yr, mean, rstd);
    }
    copies_wait<0>();
  }
  if (CL) cg::this_cluster().sync();  // no block leaves while another may still write to it
}

template <typename TS, typename TB>
cudaError_t launch(const TeamPlan &p, int64_t teams, const TeamArgs &q, Form form, cudaStream_t s) {
  SNACK_TEAM(norm_team_forward, TS, TB)
}

}  // namespace

TeamPlan team_forward(const NormArgs &n) {
  const snack_norm_args &a = n.a;
  TeamPlan p = team_shape(a);
  if (p.threads == 0) return p;
  const bool full = a.gate_kind == SNACK_GATE_FULL;
  p.vec = a.width % 8 == 0 && rows16(a.x, a.x_stride, a.stream_type) && rows16(a.y, a.y_stride, a.branch_type) &&
          (!full || rows16(a.gate, a.gate_stride, a.branch_type)) && aligned_to(n.r, 16) && aligned_to(n.h, 16);
  team_ring(&p, a, 1, full ? 2 : 1);
  p.teams = std::min<int64_t>(a.rows, std::max<int64_t>(1, (int64_t)device_sms() * (2 * kTeamThreads / p.threads) / p.cluster));
  return p;
}

cudaError_t launch_team_forward(const NormArgs &n, const TeamPlan &p, cudaStream_t s) {
  const snack_norm_args &a = n.a;
  const TeamArgs q = {n, p.block_cols, p.threads, nullptr, nullptr};
  const Form form = !plain_options(a) || !n.r || !a.stats ? kAny : (a.post_norm ? kFastPost : kFast);
#define SNACK_CALL(TS, TB) return launch<TS, TB>(p, p.teams, q, form, s);
  SNACK_NORM_TYPES(SNACK_CALL)
#undef SNACK_CALL
}

}  // namespace snack
