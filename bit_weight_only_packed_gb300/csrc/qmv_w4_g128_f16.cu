// qmv_w4_g128_f16.cu -- the 4-bit matvec for groups of 128 with scales in fp16.
#include "qmv_w4_gemv.cuh"

namespace qmv {
namespace w4 {
template cudaError_t launch_group<128, false>(const GemvArgs4& a, cudaStream_t s);
template cudaError_t read_error<128, false>(int clear, int* out);
}  // namespace w4
}  // namespace qmv
