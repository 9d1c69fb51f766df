// qmv_experts_g64.cu -- the experts' products with groups of 64.
#include "qmv_experts.cuh"

namespace qmv {
namespace w4 {
template cudaError_t run_experts<64>(const ExpertsArgs&, const ExpertsPlan&, cudaStream_t);
template cudaError_t read_x_error<64>(int, int*);
}  // namespace w4
}  // namespace qmv
