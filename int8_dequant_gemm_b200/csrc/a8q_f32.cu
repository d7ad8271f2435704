// The 8-bit row operators on fp32 tensors; see a8q.cuh.
#include "a8q.cuh"

namespace rtq {

template cudaError_t row_operator<float>(int, int, const RowArgs &, cudaStream_t);
template cudaError_t row_values<float>(int, const uint8_t *, const float *, void *, int, int,
                                     cudaStream_t);

}  // namespace rtq
