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

// Two neighbouring 16-bit elements as fp32 and back (one instruction for the pair).
template <typename T>
__device__ __forceinline__ float2 unpack(uint32_t v);
template <>
__device__ __forceinline__ float2 unpack<__half>(uint32_t v) {
  return __half22float2(*reinterpret_cast<const __half2*>(&v));
}
template <>
__device__ __forceinline__ float2 unpack<__nv_bfloat16>(uint32_t v) {
  return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xffff0000u));
}
template <typename T>
__device__ __forceinline__ uint32_t pack(float a, float b);
template <>
__device__ __forceinline__ uint32_t pack<__half>(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
template <>
__device__ __forceinline__ uint32_t pack<__nv_bfloat16>(float a, float b) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// Eight elements of a row, kept as they are stored.  VEC: eight neighbours,
// aligned to 16 bytes; otherwise every `step`-th one, so that neighbouring
// threads read neighbouring elements whatever the alignment.
template <typename T, bool VEC>
struct Eight {
  alignas(16) uint32_t w[2 * sizeof(T)];
  __device__ __forceinline__ void load(const T* p, int i0, int step, int D) {
    if (VEC) {
#pragma unroll
      for (int q = 0; q < (int)sizeof(w) / 16; ++q)
        reinterpret_cast<uint4*>(w)[q] = reinterpret_cast<const uint4*>(p + i0)[q];
    } else if (sizeof(T) == 4) {
#pragma unroll
      for (int e = 0; e < 8; ++e) w[e] = i0 + e * step < D ? reinterpret_cast<const uint32_t*>(p)[i0 + e * step] : 0u;
    } else {
      const uint16_t* s = reinterpret_cast<const uint16_t*>(p);
#pragma unroll
      for (int e = 0; e < 8; e += 2) {
        const uint32_t a = i0 + e * step < D ? s[i0 + e * step] : 0u, b = i0 + (e + 1) * step < D ? s[i0 + (e + 1) * step] : 0u;
        w[e >> 1] = a | b << 16;
      }
    }
  }
  __device__ __forceinline__ float2 pair(int e) const {      // elements e and e + 1
    if constexpr (sizeof(T) == 4)
      return make_float2(__uint_as_float(w[e]), __uint_as_float(w[e + 1]));
    else
      return unpack<T>(w[e >> 1]);
  }
  __device__ __forceinline__ void set(int e, float a, float b) { w[e >> 1] = pack<T>(a, b); }
  __device__ __forceinline__ void store(T* p, int i0, int step, int D) const {
    if (VEC) {
      *reinterpret_cast<uint4*>(p + i0) = *reinterpret_cast<const uint4*>(w);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (i0 + e * step < D) reinterpret_cast<uint16_t*>(p)[i0 + e * step] = (uint16_t)(w[e >> 1] >> (16 * (e & 1)));
    }
  }
};

// One CTA a row, the row in registers: 8 * P elements a thread, read once.
// Elements past the row's end are zeros, which add nothing to either sum.
// MAXT: the most threads of a launch; below 1024 the registers are held to what
// 1536 threads (1280 with fp32 y) a streaming multiprocessor leave.
template <typename Y, typename T, bool VEC, int P, int MAXT>
__global__ void __launch_bounds__(MAXT, MAXT < 1024 ? (sizeof(Y) == 4 ? 1280 : 1536) / MAXT : 1) norm_kernel(NormArgs a) {
  __shared__ float red[2][32];
  const int64_t m = blockIdx.x;
  const int D = a.D, NT = blockDim.x, tid = threadIdx.x;
  const T *gpo = (const T*)a.gamma_post, *gpr = (const T*)a.gamma_pre;
  pdl_begin();
  Eight<Y, VEC> y[P] = {};
  Eight<T, VEC> r[P] = {}, gt[P] = {};
#pragma unroll
  for (int p = 0; p < P; ++p) {
    const int i0 = VEC ? (p * NT + tid) * 8 : p * 8 * NT + tid;
    if (i0 < D) {
      y[p].load((const Y*)a.y + m * a.ldy, i0, NT, D);
      r[p].load((const T*)a.r + m * a.ldr, i0, NT, D);
      if (a.gate) gt[p].load((const T*)a.gate + m * a.ldg, i0, NT, D);
    }
  }
  float inv = a.bs;                      // branch scale and first norm as one factor
  if (gpo) {
    float ss = 0.0f;
#pragma unroll
    for (int p = 0; p < P; ++p)
#pragma unroll
      for (int e = 0; e < 8; e += 2) {
        const float2 v = y[p].pair(e);
        ss = fmaf(v.x, v.x, fmaf(v.y, v.y, ss));
      }
    inv = a.bs / sqrtf(block_sum(ss, red[0]) / (float)D + a.eps);
  }
  float ss = 0.0f;
#pragma unroll
  for (int p = 0; p < P; ++p) {
    const int i0 = VEC ? (p * NT + tid) * 8 : p * 8 * NT + tid;
    if (i0 >= D) continue;
    Eight<T, VEC> go;
    if (gpo) go.load(gpo, i0, NT, D);
#pragma unroll
    for (int e = 0; e < 8; e += 2) {
      float2 u = y[p].pair(e);
      u.x *= inv, u.y *= inv;
      if (gpo) {
        const float2 g = go.pair(e);
        u.x *= g.x + a.goff, u.y *= g.y + a.goff;
      }
      if (a.gate) {
        const float2 g = gt[p].pair(e);
        u.x *= g.x, u.y *= g.y;
      }
      const float2 v = r[p].pair(e);
      r[p].set(e, fmaf(a.rs, v.x, u.x), fmaf(a.rs, v.y, u.y));
      const float2 h = r[p].pair(e);
      ss = fmaf(h.x, h.x, fmaf(h.y, h.y, ss));
    }
    if (a.h) r[p].store((T*)a.h + m * a.ldh, i0, NT, D);
  }
  const float inv2 = 1.0f / sqrtf(block_sum(ss, red[1]) / (float)D + a.eps);
#pragma unroll
  for (int p = 0; p < P; ++p) {
    const int i0 = VEC ? (p * NT + tid) * 8 : p * 8 * NT + tid;
    if (i0 >= D) continue;
    Eight<T, VEC> g;
    g.load(gpr, i0, NT, D);
#pragma unroll
    for (int e = 0; e < 8; e += 2) {
      const float2 h = r[p].pair(e), q = g.pair(e);
      r[p].set(e, h.x * inv2 * (q.x + a.goff), h.y * inv2 * (q.y + a.goff));
    }
    r[p].store((T*)a.out + m * a.ldo, i0, NT, D);
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
  const int one = (need + 31) / 32 * 32, two = ((need + 1) / 2 + 31) / 32 * 32;
  // Few rows: more threads, for the latency of one.  Many rows: twice the elements a
  // thread, since the sums' steps are shared by them, and more rows at once (4096 rows
  // of 4096 in bf16 with a gate: 33.0 us at eight elements a thread, 30.5 us at
  // sixteen, 28.8 us with six rows a streaming multiprocessor).
  const bool many = vec && need >= 128 && a.M >= 2 * dev_info().sms;
  if (many && two <= 256) return launch_step(norm_kernel<Y, T, true, 2, 256>, grid, two, 0, s, 1, a);
  if (many && two <= 512) return launch_step(norm_kernel<Y, T, true, 2, 512>, grid, two, 0, s, 1, a);
  if (need <= 1024)
    return vec ? launch_step(norm_kernel<Y, T, true, 1, 1024>, grid, one, 0, s, 1, a)
               : launch_step(norm_kernel<Y, T, false, 1, 1024>, grid, one, 0, s, 1, a);
  if (need <= 2048 && vec) return launch_step(norm_kernel<Y, T, true, 2, 1024>, grid, two, 0, s, 1, a);
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
