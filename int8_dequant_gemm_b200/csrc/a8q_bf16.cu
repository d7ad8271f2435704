// The 8-bit row operators on bf16 tensors; see a8q.cuh.
#include "a8q.cuh"

namespace rtq {

template cudaError_t row_operator<__nv_bfloat16>(int, int, const RowArgs &, cudaStream_t);
template cudaError_t row_values<__nv_bfloat16>(int, const uint8_t *, const float *, void *, int, int,
                                     cudaStream_t);

}  // namespace rtq
