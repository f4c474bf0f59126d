// Tile shapes of attention on mma.sync; included once for each type.
#pragma once

#include "attention_rows.cuh"

namespace snack {

// Backward, many rows: 64 of one side in a block of eight warps.  Few rows,
// which would leave most of the GPU idle so: 16 of them, and four warps that
// share every step.  What the steps hold is what two stages of them leave of
// the 227 KB.
template <typename T>
struct Shapes {
  static constexpr bool kWide = sizeof(T) == 4;
  static constexpr int kBackward = 32, kFewBackward = kWide ? 16 : 32;
};

template <typename K>
inline cudaError_t launch_rows(K kern, int64_t blocks, int threads, size_t smem, const AttnCall &c,
                               cudaStream_t s) {
  if (blocks == 0) return cudaSuccess;
  const cudaError_t e = allow_smem(kern, smem);
  if (e != cudaSuccess) return e;
  return launch_kernel(kern, dim3((unsigned)blocks), threads, smem, false, s, c);
}

template <typename T, int DP>
cudaError_t rows_forward_size(const AttnCall &c, cudaStream_t s) {
  constexpr int kKeys = sizeof(T) == 4 ? 32 : 64;
  return launch_rows(rows_forward<T, DP, 8, kKeys>,
                     tiles_of(c.q_offsets != nullptr, c.sequences, c.q_tokens, c.group, 128) * c.key_heads, 256,
                     rows_forward_smem<T, DP, 8, kKeys>(), c, s);
}

template <typename T, int DP>
cudaError_t rows_backward_size(const AttnCall &c, cudaStream_t s) {
  using S = Shapes<T>;
  cudaError_t e = cudaSuccess;
  if (c.dk.p || c.dv.p) {
    const bool ragged = c.k_offsets != nullptr;
    const int64_t many = tiles_of(ragged, c.sequences, c.k_tokens, 1, 64) * c.key_heads;
    if (many < device_sms())
      e = launch_rows(rows_backward_keys<T, DP, 1, 4, S::kFewBackward>,
                      tiles_of(ragged, c.sequences, c.k_tokens, 1, 16) * c.key_heads, 128,
                      rows_backward_smem<T, DP, 1, 4, S::kFewBackward>(), c, s);
    else
      e = launch_rows(rows_backward_keys<T, DP, 4, 2, S::kBackward>, many, 256,
                      rows_backward_smem<T, DP, 4, 2, S::kBackward>(), c, s);
  }
  if (e == cudaSuccess && c.dq.p) {
    const bool ragged = c.q_offsets != nullptr;
    const int64_t many = tiles_of(ragged, c.sequences, c.q_tokens, c.group, 64) * c.key_heads;
    if (many < device_sms())
      e = launch_rows(rows_backward_queries<T, DP, 1, 4, S::kFewBackward>,
                      tiles_of(ragged, c.sequences, c.q_tokens, c.group, 16) * c.key_heads, 128,
                      rows_backward_smem<T, DP, 1, 4, S::kFewBackward>(), c, s);
    else
      e = launch_rows(rows_backward_queries<T, DP, 4, 2, S::kBackward>, many, 256,
                      rows_backward_smem<T, DP, 4, 2, S::kBackward>(), c, s);
  }
  return e;
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
