// Tile shapes of attention on mma.sync; included once for each type.
#pragma once

#include "attention_rows.cuh"

namespace snack {

// Backward, many rows: 64 of one side in a block of eight warps.  Few rows,
// which would leave most of the GPU idle so: 16 of them, and four warps that
// share every step; one stage, so that all blocks are resident together and
// one computes while another waits for its copies.  What the steps of many rows
// hold is what two stages of them leave of the 227 KB.
template <typename T>
struct Shapes {
  static constexpr bool kWide = sizeof(T) == 4;
  static constexpr int kBackward = 32, kFewBackward = kWide ? 16 : 32;
};

template <typename T, int DP>
cudaError_t rows_forward_size(const AttnCall &c, cudaStream_t s) {
  constexpr int kKeys = sizeof(T) == 4 ? 32 : 64;
  const auto kern = rows_forward<T, DP, 8, kKeys>;
  constexpr size_t smem = rows_forward_smem<T, DP, 8, kKeys>();
  const int64_t blocks = tiles_of(c.q_offsets != nullptr, c.sequences, c.q_tokens, c.group, 128) * c.key_heads;
  if (blocks == 0) return cudaSuccess;
  const cudaError_t e = allow_smem(kern, smem);
  if (e != cudaSuccess) return e;
  return launch_kernel(kern, dim3((unsigned)blocks), 256, smem, false, s, c);
}

template <typename T, int DP, int WM, int WN, int BN, int ST, int ONLY>
cudaError_t rows_backward_blocks(const AttnCall &c, int64_t keys, int64_t queries, cudaStream_t s) {
  if (keys + queries == 0) return cudaSuccess;
  const auto kern = rows_backward<T, DP, WM, WN, BN, ST, ONLY>;
  constexpr size_t smem = rows_backward_smem<T, DP, WM, WN, BN, ST>();
  const cudaError_t e = allow_smem(kern, smem);
  if (e != cudaSuccess) return e;
  return launch_kernel(kern, dim3((unsigned)(keys + queries)), 32 * WM * WN, smem, false, s, c, (int)keys);
}

// Few rows: keys and queries in one launch, side by side (256 tokens of 12
// heads of 64 in 32 bits took 49 us in two).  Many: one after the other, each
// with the registers that it needs.
template <typename T, int DP>
cudaError_t rows_backward_size(const AttnCall &c, cudaStream_t s) {
  using S = Shapes<T>;
  const auto keys = [&](int rows) {
    return c.dk.p || c.dv.p ? tiles_of(c.k_offsets != nullptr, c.sequences, c.k_tokens, 1, rows) * c.key_heads : 0;
  };
  const auto queries = [&](int rows) {
    return c.dq.p ? tiles_of(c.q_offsets != nullptr, c.sequences, c.q_tokens, c.group, rows) * c.key_heads : 0;
  };
  if (keys(64) + queries(64) < 2 * device_sms())
    return rows_backward_blocks<T, DP, 1, 4, S::kFewBackward, 1, 0>(c, keys(16), queries(16), s);
  const cudaError_t e = rows_backward_blocks<T, DP, 4, 2, S::kBackward, 2, 1>(c, keys(64), 0, s);
  return e != cudaSuccess ? e : rows_backward_blocks<T, DP, 4, 2, S::kBackward, 2, 2>(c, 0, queries(64), s);
}

template <typename T>
cudaError_t rows_forward_launch(const AttnCall &c, cudaStream_t s) {
  return c.d <= 64 ? rows_forward_size<T, 64>(c, s) : rows_forward_size<T, 128>(c, s);
}
template <typename T>
cudaError_t rows_backward_launch(const AttnCall &c, cudaStream_t s) {
  return c.d <= 64 ? rows_backward_size<T, 64>(c, s) : rows_backward_size<T, 128>(c, s);
}

}  // namespace snack
