// Shared by the residual norm's kernels: residual_norm.cu (checks, any shape)
// and norm_team_*.cu (rows held in registers).
#pragma once

#include "dense_ops.cuh"

namespace snack {

struct NormArgs {
  snack_norm_args a;
  snack_norm_grads g;
  void *r, *h;
  float *row_scalars;         // [rows][2]: mean(t), mean(t rhat)
  float *parts;               // column sums of the backward (see each kernel)
  int64_t groups, group_len;  // rows that share a gate row lie in one group of group_len rows
  int64_t slabs, slab_rows, slabs_per_group;
};

// One team of threads for each row; the team's blocks (one, or a cluster for
// wide rows) hold the row in registers, kTeamCols columns in each thread.
constexpr int kTeamCols = 8;
constexpr int kTeamThreads = 512;  // most threads of one block
constexpr int kTeamCluster = 8;    // most blocks of one team

struct TeamPlan {
  int threads = 0;   // of a team in one block; 0: the row is too wide for a team
  int per_block = 1; // teams of one block
  int cluster = 1;
  int block_cols = 0;  // columns of one block
  bool vec = false;    // rows can be read and written in 16-byte vectors
  int stages = 0;      // rows in the ring: one held, the others copied ahead
  size_t smem = 0;
  int64_t teams = 0;  // blocks (or clusters) in all
};

TeamPlan team_forward(const NormArgs &n);
TeamPlan team_backward(const NormArgs &n);
cudaError_t launch_team_forward(const NormArgs &n, const TeamPlan &p, cudaStream_t s);
cudaError_t launch_team_backward(const NormArgs &n, const TeamPlan &p, cudaStream_t s);

// F(TS, TB) for the types of a.
#define SNACK_NORM_TYPES(F)                                                                   \
  if (a.stream_type == SNACK_F32 && a.branch_type == SNACK_F32) F(float, float)               \
  else if (a.stream_type == SNACK_F32 && a.branch_type == SNACK_BF16) F(float, __nv_bfloat16) \
  else if (a.stream_type == SNACK_F32) F(float, __half)                                       \
  else if (a.stream_type == SNACK_BF16) F(__nv_bfloat16, __nv_bfloat16)                       \
  else F(__half, __half)

}  // namespace snack
