// qmv_experts_g128.cu -- the experts' products with groups of 128.
#include "qmv_experts.cuh"

namespace qmv {
namespace w4 {
template cudaError_t run_experts<128>(const ExpertsArgs&, const ExpertsPlan&, cudaStream_t);
template cudaError_t read_x_error<128>(int, int*);
}  // namespace w4
}  // namespace qmv
