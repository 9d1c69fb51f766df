// qmv_experts_g32.cu -- the experts' products with groups of 32.
#include "qmv_experts.cuh"

namespace qmv {
namespace w4 {
template cudaError_t run_experts<32>(const ExpertsArgs&, const ExpertsPlan&, cudaStream_t);
template cudaError_t read_x_error<32>(int, int*);
}  // namespace w4
}  // namespace qmv
