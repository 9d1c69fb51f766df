// qmv_w4_g64_bf16.cu -- the 4-bit matvec for groups of 64 with scales in bf16.
#include "qmv_w4_gemv.cuh"

namespace qmv {
namespace w4 {
template cudaError_t launch_group<64, true>(const GemvArgs4& a, cudaStream_t s);
template cudaError_t read_error<64, true>(int clear, int* out);
}  // namespace w4
}  // namespace qmv
