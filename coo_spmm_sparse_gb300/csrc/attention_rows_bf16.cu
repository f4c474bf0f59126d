#include "attention_rows_launch.cuh"

namespace snack {
template cudaError_t rows_forward_launch<__nv_bfloat16>(const AttnCall &, cudaStream_t);
template cudaError_t rows_backward_launch<__nv_bfloat16>(const AttnCall &, cudaStream_t);
}  // namespace snack
