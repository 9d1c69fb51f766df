// qmv_norm.cu -- the norms after and before a block with its gate and residual
// scale (qmv_block_norm):
//   u = gate * (y / sqrt(mean y^2 + eps) * g_post),  h = round(a r + b u),
//   z = round(h / sqrt(mean h^2 + eps) * g_pre).
#include "qmv_step.cuh"

namespace qmv {
namespace {

// The sum of v over a CTA, the same in every thread; red: one float a warp,
// a buffer of its own for each sum of a kernel.
__device__ __forceinline__ float block_sum(float v, float* red) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(~0u, v, o);
  const int nw = blockDim.x >> 5;
  if (nw == 1) return v;
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  v = (threadIdx.x & 31) < nw ? red[threadIdx.x & 31] : 0.0f;
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(~0u, v, o);
  return v;
}

// Eight elements of a row as fp32.  VEC: eight neighbours, aligned to their
// total size; otherwise every blockDim.x-th one, so that neighbouring threads
// read neighbouring elements whatever the alignment.
template <typename T, bool VEC>
struct Eight {
  alignas(16) T v[8];
  __device__ __forceinline__ void load(const T* p, int i0, int step, int D) {
    if (VEC) {
#pragma unroll
      for (int q = 0; q < (int)sizeof(v) / 16; ++q)
        reinterpret_cast<uint4*>(v)[q] = reinterpret_cast<const uint4*>(p + i0)[q];
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (i0 + e * step < D) v[e] = p[i0 + e * step];
    }
  }
  __device__ __forceinline__ void store(T* p, int i0, int step, int D) const {
    if (VEC) {
#pragma unroll
      for (int q = 0; q < (int)sizeof(v) / 16; ++q)
        reinterpret_cast<uint4*>(p + i0)[q] = reinterpret_cast<const uint4*>(v)[q];
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (i0 + e * step < D) p[i0 + e * step] = v[e];
    }
  }
};

// One CTA a row, the row in registers: 8 * P elements a thread, read once.
template <typename Y, typename T, bool VEC, int P>
__global__ void __launch_bounds__(1024) norm_kernel(NormArgs a) {
  __shared__ float red[2][32];
  const int64_t m = blockIdx.x;
  const int D = a.D, NT = blockDim.x, tid = threadIdx.x;
  const T *gpo = (const T*)a.gamma_post, *gpr = (const T*)a.gamma_pre;
  int i0[P];
  bool on[P];                    // VEC: whether these eight are inside the row
#pragma unroll
  for (int p = 0; p < P; ++p) {
    i0[p] = VEC ? (p * NT + tid) * 8 : p * 8 * NT + tid;
    on[p] = i0[p] < D;
  }
  const int step = NT;
  pdl_begin();
  Eight<Y, VEC> y[P];
  Eight<T, VEC> r[P], gt[P];
#pragma unroll
  for (int p = 0; p < P; ++p)
    if (on[p]) {
      y[p].load((const Y*)a.y + m * a.ldy, i0[p], step, D);
      r[p].load((const T*)a.r + m * a.ldr, i0[p], step, D);
      if (a.gate) gt[p].load((const T*)a.gate + m * a.ldg, i0[p], step, D);
    }
  float inv = 1.0f;
  if (gpo) {
    float ss = 0.0f;
#pragma unroll
    for (int p = 0; p < P; ++p)
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (VEC ? on[p] : i0[p] + e * step < D) {
          const float v = to_f<Y>(y[p].v[e]);
          ss = fmaf(v, v, ss);
        }
    inv = 1.0f / sqrtf(block_sum(ss, red[0]) / (float)D + a.eps);
  }
  float ss = 0.0f;
#pragma unroll
  for (int p = 0; p < P; ++p)
    if (on[p]) {
      Eight<T, VEC> go;
      if (gpo) go.load(gpo, i0[p], step, D);
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (VEC || i0[p] + e * step < D) {
          float u = to_f<Y>(y[p].v[e]);
          if (gpo) u = u * inv * (to_f<T>(go.v[e]) + a.goff);
          if (a.gate) u *= to_f<T>(gt[p].v[e]);
          const T hv = from_f<T>(fmaf(a.rs, to_f<T>(r[p].v[e]), a.bs * u));
          r[p].v[e] = hv;
          const float f = to_f<T>(hv);
          ss = fmaf(f, f, ss);
        }
      if (a.h) r[p].store((T*)a.h + m * a.ldh, i0[p], step, D);
    }
  const float inv2 = 1.0f / sqrtf(block_sum(ss, red[1]) / (float)D + a.eps);
#pragma unroll
  for (int p = 0; p < P; ++p)
    if (on[p]) {
      Eight<T, VEC> g;
      g.load(gpr, i0[p], step, D);
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (VEC || i0[p] + e * step < D) r[p].v[e] = from_f<T>(to_f<T>(r[p].v[e]) * inv2 * (to_f<T>(g.v[e]) + a.goff));
      r[p].store((T*)a.out + m * a.ldo, i0[p], step, D);
    }
}

// Rows too long for registers: h waits in shared memory for its own norm.
template <typename Y, typename T>
__global__ void __launch_bounds__(1024) norm_long_kernel(NormArgs a) {
  extern __shared__ uint4 dyn[];
  T* hs = reinterpret_cast<T*>(dyn);
  __shared__ float red[2][32];
  const int64_t m = blockIdx.x;
  const int NT = blockDim.x;
  const Y* y = (const Y*)a.y + m * a.ldy;
  const T* r = (const T*)a.r + m * a.ldr;
  const T* gate = a.gate ? (const T*)a.gate + m * a.ldg : nullptr;
  const T *gpo = (const T*)a.gamma_post, *gpr = (const T*)a.gamma_pre;
  T* h = a.h ? (T*)a.h + m * a.ldh : nullptr;
  T* out = (T*)a.out + m * a.ldo;
  pdl_begin();
  float inv = 1.0f;
  if (gpo) {
    float ss = 0.0f;
    for (int i = threadIdx.x; i < a.D; i += NT) {
      const float v = to_f<Y>(y[i]);
      ss = fmaf(v, v, ss);
    }
    inv = 1.0f / sqrtf(block_sum(ss, red[0]) / (float)a.D + a.eps);
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
  const float inv2 = 1.0f / sqrtf(block_sum(ss, red[1]) / (float)a.D + a.eps);
  for (int i = threadIdx.x; i < a.D; i += NT) {
    if (h) h[i] = hs[i];
    out[i] = from_f<T>(to_f<T>(hs[i]) * inv2 * (to_f<T>(gpr[i]) + a.goff));
  }
}

template <typename Y, typename T>
cudaError_t run(const NormArgs& a, cudaStream_t s) {
  const auto ok = [&](const void* p, int ld, size_t size) {
    return (uintptr_t)p % 16 == 0 && ((size_t)ld * size) % 16 == 0;
  };
  const bool vec = a.D % 8 == 0 && ok(a.y, a.ldy, sizeof(Y)) && ok(a.r, a.ldr, 2) && ok(a.gamma_post, 0, 2) &&
                   ok(a.gate, a.ldg, 2) && ok(a.gamma_pre, 0, 2) && ok(a.h, a.ldh, 2) && ok(a.out, a.ldo, 2);
  const int need = (a.D + 7) / 8;              // threads at eight elements each
  const dim3 grid(a.M);
  if (need <= 1024) {
    const int nt = (need + 31) / 32 * 32;
    return vec ? launch_step(norm_kernel<Y, T, true, 1>, grid, nt, 0, s, 1, a)
               : launch_step(norm_kernel<Y, T, false, 1>, grid, nt, 0, s, 1, a);
  }
  if (need <= 2048 && vec) {
    const int nt = ((need + 1) / 2 + 31) / 32 * 32;
    return launch_step(norm_kernel<Y, T, true, 2>, grid, nt, 0, s, 1, a);
  }
  static thread_local KernCache c;
  const size_t smem = (size_t)a.D * sizeof(T);
  const cudaError_t e = prep_kernel(norm_long_kernel<Y, T>, c, 1024, smem, nullptr);
  if (e != cudaSuccess) return e;
  return launch_step(norm_long_kernel<Y, T>, grid, 1024, smem, s, 1, a);
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
