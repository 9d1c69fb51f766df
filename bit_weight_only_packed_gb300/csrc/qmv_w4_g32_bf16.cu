// qmv_w4_g32_bf16.cu -- the 4-bit matvec for groups of 32 with scales in bf16.
#include "qmv_w4_gemv.cuh"

namespace qmv {
namespace w4 {
template cudaError_t launch_group<32, true>(const GemvArgs4& a, cudaStream_t s);
template cudaError_t read_error<32, true>(int clear, int* out);
}  // namespace w4
}  // namespace qmv
