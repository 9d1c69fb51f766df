// qmv_norm.cu -- the norms after and before a block with its gate and residual
// scale (qmv_block_norm):
//   u = gate * (y / sqrt(mean y^2 + eps) * g_post),  h = round(a r + b u),
//   z = round(h / sqrt(mean h^2 + eps) * g_pre).
#include "qmv_step.cuh"

namespace qmv {
namespace {

constexpr int NT = 256;

__device__ __forceinline__ float block_sum(float v, float* red) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(~0u, v, o);
  __syncthreads();                 // red may still be read from the last sum
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  v = 0.0f;
#pragma unroll
  for (int w = 0; w < NT / 32; ++w) v += red[w];
  return v;
}

// One CTA a row; h waits in shared memory for its own norm.
template <typename Y, typename T>
__global__ void __launch_bounds__(NT) norm_kernel(NormArgs a) {
  extern __shared__ uint4 dyn[];
  T* hs = reinterpret_cast<T*>(dyn);
  __shared__ float red[NT / 32];
  const int64_t m = blockIdx.x;
  const Y* y = (const Y*)a.y + m * a.ldy;
  const T* r = (const T*)a.r + m * a.ldr;
  const T* gate = a.gate ? (const T*)a.gate + m * a.ldg : nullptr;
  const T *gpo = (const T*)a.gamma_post, *gpr = (const T*)a.gamma_pre;
  T* h = a.h ? (T*)a.h + m * a.ldh : nullptr;
  T* out = (T*)a.out + m * a.ldo;
  float inv = 1.0f;
  if (gpo) {
    float ss = 0.0f;
    for (int i = threadIdx.x; i < a.D; i += NT) {
      const float v = to_f<Y>(y[i]);
      ss = fmaf(v, v, ss);
    }
    inv = 1.0f / sqrtf(block_sum(ss, red) / (float)a.D + a.eps);
  }
  float ss = 0.0f;
  for (int i = threadIdx.x; i < a.D; i += NT) {
    float u = to_f<Y>(y[i]);
    if (gpo) u = u * inv * (to_f<T>(gpo[i]) + a.goff);
    if (gate) u *= to_f<T>(gate[i]);
    const T hv = from_f<T>(fmaf(a.rs, to_f<T>(r[i]), a.bs * u));
    hs[i] = hv;
    const float f = to_f<T>(hv);
    ss = fmaf(f, f, ss);
  }
  const float inv2 = 1.0f / sqrtf(block_sum(ss, red) / (float)a.D + a.eps);
  for (int i = threadIdx.x; i < a.D; i += NT) {
    if (h) h[i] = hs[i];
    out[i] = from_f<T>(to_f<T>(hs[i]) * inv2 * (to_f<T>(gpr[i]) + a.goff));
  }
}

template <typename Y, typename T>
cudaError_t run(const NormArgs& a, cudaStream_t s) {
  static thread_local KernCache c;
  const size_t smem = (size_t)a.D * sizeof(T);
  const cudaError_t e = prep_kernel(norm_kernel<Y, T>, c, NT, smem, nullptr);
  if (e != cudaSuccess) return e;
  norm_kernel<Y, T><<<a.M, NT, smem, s>>>(a);
  return cudaGetLastError();
}

template <typename T>
cudaError_t run_y(const NormArgs& a, cudaStream_t s) {
  if (a.y_dtype == QMV_F32) return run<float, T>(a, s);
  if (a.y_dtype == QMV_F16) return run<__half, T>(a, s);
  return run<__nv_bfloat16, T>(a, s);
}

}  // namespace

cudaError_t launch_block_norm(const NormArgs& a, cudaStream_t s) {
  return a.bf16 ? run_y<__nv_bfloat16>(a, s) : run_y<__half>(a, s);
}

}  // namespace qmv
