// qmv_token.cuh -- declarations of the decode-step operators around the matvecs: norms and
// rotation of heads (qmv_rope.cu), routing to experts (qmv_route.cu), the experts' products
// (qmv_experts.cu) and the next token (qmv_draw.cu).  Arguments are checked in qmv_token_abi.cu.
#pragma once
#include "qmv_step.cuh"

namespace qmv {

// What is read before the wait for the kernel before (see launch_step): from L2, past lines of L1 that
// may be older than a write two kernels back.
__device__ __forceinline__ int ld_early(const int* p) {
  int v;
  asm volatile("ld.relaxed.gpu.global.s32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
  return v;
}
__device__ __forceinline__ float ld_early(const float* p) {
  float v;
  asm volatile("ld.relaxed.gpu.global.f32 %0, [%1];" : "=f"(v) : "l"(p) : "memory");
  return v;
}

struct RopeArgs {
  int M, nq, nk, D;
  const void* x;
  int ld, x_dtype;
  const int* positions;
  const int64_t* turns;
  int rot, layout;
  float amplitude;
  const void *gamma_q, *gamma_k;
  float goff, eps;
  void* q;
  int ldq;
  void* k;
  int ldk;
  int bf16;
};
cudaError_t launch_rope(const RopeArgs& a, cudaStream_t s);

struct RouteArgs {
  int M, E, T;
  const void* x;
  int ldx, dtype, score;
  const float* bias;
  int groups, group_k, group_top, renorm;
  float scale;
  int* ids;
  float* w;
  int per;                      // experts a group
  uint32_t per_inv;             // above 1: e / per is the upper half of e * per_inv, for e below 1024
};
cudaError_t launch_route(const RouteArgs& a, cudaStream_t s);

struct ExpertsArgs {
  const uint8_t* packed;
  int K, scale_bf16, group, zeros;
  int E, R, M, T;
  const int* ids;
  const float* weights;
  const void* x;
  int ldx, per_pair, x_bf16, act;
  void* y;
  int ldy, y_dtype;
  void* ws;
};
// One column of the longest row fits twice beside the rings; strips of all tasks are counted in int.
constexpr int EXPERTS_MAX_K = 16384, EXPERTS_MAX_PAIRS = 32768, EXPERTS_MAX_E = 1024, EXPERTS_MAX_R = 1 << 20;
static_assert((int64_t)EXPERTS_MAX_PAIRS * (EXPERTS_MAX_R / 32) <= (int64_t)1 << 30, "strips");
// Scratch of any call of these sizes, and of the one call (ids, y and the scratch itself do not count).
size_t experts_workspace(int K, int R, int M, int T);
size_t experts_workspace(const ExpertsArgs& a);
cudaError_t launch_experts(const ExpertsArgs& a, cudaStream_t s);
// The device error word of the experts' products (bounded waits, ids out of range).
int read_experts_error(int clear, int* out);

struct DrawArgs {
  int rows, V;
  const void* x;
  int ldx, dtype;
  const float* t;
  float t0;
  const int* k;
  int k0;
  const float* p;
  float p0;
  const float* m;
  float m0;
  const float* u;
  int* tokens;
};
cudaError_t launch_draw(const DrawArgs& a, cudaStream_t s);

}  // namespace qmv
