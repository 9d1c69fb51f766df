// qmv_norm.cu -- the norms after and before a block with its gate and residual
// scale (qmv_block_norm):
//   u = gate * (y / sqrt(mean y^2 + eps) * g_post),  h = round(a r + b u),
//   z = round(h / sqrt(mean h^2 + eps) * g_pre).
#include <algorithm>

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

// How a thread takes its eights of a row:
//   ALIGNED  eight neighbours, 16-byte aligned everywhere;
//   SHIFTED  the same, but every row begins somewhere past such an alignment (an odd D
//            shifts every row; all [M][D] tensors alike).  The elements before its first
//            aligned eight and after its last, at most seven each, go one to a thread
//            of the first sixteen; the vectors [D] lie another way;
//   APART    every NT-th element, whatever the alignments.
enum Mode { ALIGNED, SHIFTED, APART };

// Eight 16-bit elements from p on, whatever p's alignment: the two aligned 16-byte words
// that hold them, moved into place; both are the caller's to read.  Against eight loads, for
// 3000 rows of 5381: 40.2 for 44.1 us in bf16, 39.4 for 49.9 with y in fp32; where one warp
// takes a row, which then goes both ways, it costs (160000 x 99: 106 for 93 us).
__device__ __forceinline__ void load_across(const uint16_t* p, uint32_t* w) {
  const uint32_t off = (uint32_t)(uintptr_t)p & 15;            // the same in a whole row
  const uint4* q = reinterpret_cast<const uint4*>((uintptr_t)p - off);
  const uint4 lo = q[0], hi = q[1];
  uint32_t v[7] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z};
  if (off & 8) v[0] = v[2], v[1] = v[3], v[2] = v[4], v[3] = v[5], v[4] = v[6], v[5] = hi.w;
  if (off & 4) v[0] = v[1], v[1] = v[2], v[2] = v[3], v[3] = v[4], v[4] = v[5];
#pragma unroll
  for (int k = 0; k < 4; ++k) w[k] = __funnelshift_r(v[k], v[k + 1], (off & 2) * 8);
}

// Eight elements of a row from i0 on, kept as they are stored; those outside the
// row are zeros.
template <typename T, Mode MODE>
struct Eight {
  alignas(16) uint32_t w[2 * sizeof(T)];
  // vector: a [D] vector, aligned as it is, by load_across where that pays.
  __device__ __forceinline__ void load(const T* p, int i0, int step, int D, bool vector, bool across) {
    if (MODE == ALIGNED || (MODE == SHIFTED && !vector)) {
#pragma unroll
      for (int q = 0; q < (int)sizeof(w) / 16; ++q)
        reinterpret_cast<uint4*>(w)[q] = reinterpret_cast<const uint4*>(p + i0)[q];
    } else if (sizeof(T) == 4) {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int i = i0 + e * step;
        w[e] = i < D ? reinterpret_cast<const uint32_t*>(p)[i] : 0u;
      }
    } else {
      const uint16_t* s = reinterpret_cast<const uint16_t*>(p);
      if (MODE == SHIFTED && vector && across && i0 >= 8 && i0 + 16 <= D) {     // both words inside
        load_across(s + i0, w);
        return;
      }
#pragma unroll
      for (int e = 0; e < 8; e += 2) {
        const int i = i0 + e * step, j = i + step;
        const uint32_t a = MODE == SHIFTED || i < D ? s[i] : 0u, b = MODE == SHIFTED || j < D ? s[j] : 0u;
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
    if (MODE != APART) {
      *reinterpret_cast<uint4*>(p + i0) = *reinterpret_cast<const uint4*>(w);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (i0 + e * step < D)
          reinterpret_cast<uint16_t*>(p)[i0 + e * step] = (uint16_t)(w[e >> 1] >> (16 * (e & 1)));
    }
  }
};

// One row by NT threads, in registers: 8 * P elements a thread, read once.  Elements
// past the row's end are zeros, which add nothing to either sum.
template <typename Y, typename T, Mode MODE, int P, bool WARP, typename Sum>
__device__ __forceinline__ void norm_row(const NormArgs& a, int64_t m, int tid, int NT, const Sum& sum) {
  const int D = a.D, step = MODE == APART ? NT : 1;
  const T *gpo = (const T*)a.gamma_post, *gpr = (const T*)a.gamma_pre;
  const T *rr = (const T*)a.r + m * a.ldr, *gg = (const T*)a.gate + m * a.ldg;
  const Y* yy = (const Y*)a.y + m * a.ldy;
  const bool per_row = a.ldg != 0;            // a gate of one row [D] is a vector
  // SHIFTED: the first aligned eight, what follows the last, and this thread's element of
  // the row's ends (-1: none)
  const int lead = MODE == SHIFTED ? min((int)(-(uintptr_t)rr / sizeof(T) % 8), D) : 0, behind = lead + (D - lead) / 8 * 8;
  int end = -1;
  if (MODE == SHIFTED) {
    if (tid < lead) end = tid;
    if (tid >= 8 && tid < 8 + D - behind) end = behind + tid - 8;
  }
  int i0[P];
  bool on[P];
#pragma unroll
  for (int p = 0; p < P; ++p) {
    i0[p] = MODE == APART ? p * 8 * NT + tid : lead + (p * NT + tid) * 8;
    on[p] = i0[p] < (MODE == SHIFTED ? behind : D);
  }
  Eight<Y, MODE> y[P] = {};
  Eight<T, MODE> r[P] = {}, gt[P] = {};
#pragma unroll
  for (int p = 0; p < P; ++p)
    if (on[p]) {
      y[p].load(yy, i0[p], step, D, false, false);
      r[p].load(rr, i0[p], step, D, false, false);
      if (a.gate) gt[p].load(gg, i0[p], step, D, !per_row, !WARP);
    }
  float ye = 0.0f, he = 0.0f;
  if (MODE == SHIFTED && end >= 0) ye = to_f<Y>(yy[end]), he = to_f<T>(rr[end]);
  float inv = a.bs;                      // branch scale and first norm as one factor
  if (gpo) {
    float ss = ye * ye;
#pragma unroll
    for (int p = 0; p < P; ++p)
#pragma unroll
      for (int e = 0; e < 8; e += 2) {
        const float2 v = y[p].pair(e);
        ss = fmaf(v.x, v.x, fmaf(v.y, v.y, ss));
      }
    inv = a.bs / sqrtf(sum(ss, 0) / (float)D + a.eps);
  }
  float ss = 0.0f;
  if (MODE == SHIFTED && end >= 0) {
    float u = ye * inv;
    if (gpo) u *= to_f<T>(gpo[end]) + a.goff;
    if (a.gate) u *= to_f<T>(gg[end]);
    const T h = from_f<T>(fmaf(a.rs, he, u));
    he = to_f<T>(h);
    ss = he * he;
    if (a.h) ((T*)a.h + m * a.ldh)[end] = h;
  }
#pragma unroll
  for (int p = 0; p < P; ++p) {
    if (!on[p]) continue;
    Eight<T, MODE> go;
    if (gpo) go.load(gpo, i0[p], step, D, true, !WARP);
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
    if (a.h) r[p].store((T*)a.h + m * a.ldh, i0[p], step, D);
  }
  const float inv2 = 1.0f / sqrtf(sum(ss, 1) / (float)D + a.eps);
  if (MODE == SHIFTED && end >= 0) ((T*)a.out + m * a.ldo)[end] = from_f<T>(he * inv2 * (to_f<T>(gpr[end]) + a.goff));
#pragma unroll
  for (int p = 0; p < P; ++p) {
    if (!on[p]) continue;
    Eight<T, MODE> g;
    g.load(gpr, i0[p], step, D, true, !WARP);
#pragma unroll
    for (int e = 0; e < 8; e += 2) {
      const float2 h = r[p].pair(e), q = g.pair(e);
      r[p].set(e, h.x * inv2 * (q.x + a.goff), h.y * inv2 * (q.y + a.goff));
    }
    r[p].store((T*)a.out + m * a.ldo, i0[p], step, D);
  }
}

// One CTA a row.  MAXT: the most threads of a launch; below 1024 the registers are
// held to what 1536 threads (1280 with fp32 y) a streaming multiprocessor leave.
template <typename Y, typename T, Mode MODE, int P, int MAXT>
__global__ void __launch_bounds__(MAXT, MAXT < 1024 ? (sizeof(Y) == 4 && MAXT < 768 ? 1280 : 1536) / MAXT : 1)
    norm_kernel(NormArgs a) {
  __shared__ float red[2][32];
  pdl_begin();
  norm_row<Y, T, MODE, P, false>(a, blockIdx.x, threadIdx.x, blockDim.x, [&](float v, int i) { return block_sum(v, red[i]); });
}

// One warp a row, eight rows a CTA: short rows, many of them.
constexpr int ROWS_A_CTA = 8;
template <typename Y, typename T, Mode MODE, int P>
__global__ void __launch_bounds__(32 * ROWS_A_CTA) norm_warp_kernel(NormArgs a) {
  const int64_t m = (int64_t)blockIdx.x * ROWS_A_CTA + (threadIdx.x >> 5);
  pdl_begin();
  if (m >= a.M) return;
  norm_row<Y, T, MODE, P, true>(a, m, threadIdx.x & 31, 32, [](float v, int) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(~0u, v, o);
    return v;
  });
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

// Few rows: more threads, for the latency of one.  Many rows: twice the elements a
// thread, since the sums' steps are shared by them, and more rows at once (4096 rows
// of 4096 in bf16 with a gate: 33.0 us at eight elements a thread, 30.5 us at sixteen,
// 28.8 us with six rows a streaming multiprocessor); short ones a warp each (160000 rows
// of 64 to 99: 162 us at a CTA a row, 53 aligned and 93 shifted at a warp).  Rows that
// begin unaligned, all alike, still go by eights (in bf16, 3000 x 5381: 58 us at APART,
// 40 with ends in the first and last eight, 36 with an element a thread, 29 for 5376
// aligned; 1333 x 12001: 81, 43, 38 and 31).  A launch's registers follow its threads:
// fp32 y, 3000 x 5376, 36.6 us bound for 512, 30.5 for 384.
template <typename Y, typename T, Mode MODE>
cudaError_t run_mode(const NormArgs& a, cudaStream_t s) {
  const int need = MODE == SHIFTED ? std::max(a.D / 8, 1) : (a.D + 7) / 8;      // threads at eight elements each
  const dim3 grid(a.M), warps((a.M - 1) / ROWS_A_CTA + 1);
  const bool many = a.M >= 2 * dev_info().sms;
  if (many && need <= 32) return launch_step(norm_warp_kernel<Y, T, MODE, 1>, warps, 32 * ROWS_A_CTA, 0, s, 1, a);
  if (many && need <= 64) return launch_step(norm_warp_kernel<Y, T, MODE, 2>, warps, 32 * ROWS_A_CTA, 0, s, 1, a);
  if (many && need <= 128) return launch_step(norm_warp_kernel<Y, T, MODE, 4>, warps, 32 * ROWS_A_CTA, 0, s, 1, a);
  const int one = (need + 31) / 32 * 32, two = ((need + 1) / 2 + 31) / 32 * 32;
  if constexpr (MODE != APART) {
    if (many && two <= 256) return launch_step(norm_kernel<Y, T, MODE, 2, 256>, grid, two, 0, s, 1, a);
    if (many && two <= 384) return launch_step(norm_kernel<Y, T, MODE, 2, 384>, grid, two, 0, s, 1, a);
    if (many && two <= 512) return launch_step(norm_kernel<Y, T, MODE, 2, 512>, grid, two, 0, s, 1, a);
    if (many && two <= 768) return launch_step(norm_kernel<Y, T, MODE, 2, 768>, grid, two, 0, s, 1, a);
  }
  if (one <= 1024) return launch_step(norm_kernel<Y, T, MODE, 1, 1024>, grid, one, 0, s, 1, a);
  if constexpr (MODE != APART) {
    if (two <= 1024) return launch_step(norm_kernel<Y, T, MODE, 2, 1024>, grid, two, 0, s, 1, a);
  }
  static thread_local KernCache c;
  const size_t smem = (size_t)a.D * sizeof(T);
  const cudaError_t e = prep_kernel(norm_long_kernel<Y, T>, c, 1024, smem, nullptr);
  if (e != cudaSuccess) return e;
  return launch_step(norm_long_kernel<Y, T>, grid, 1024, smem, s, 1, a);
}

template <typename Y, typename T>
cudaError_t run(const NormArgs& a, cudaStream_t s) {
  // every row of y, residual, gate, h and out begins at the same element of an aligned
  // eight; ALIGNED where that is its first
  const auto shift = [](const void* p, size_t size) { return (uintptr_t)p % (8 * size) / size; };
  const auto like = [&](const void* p, int ld, size_t size) {
    return !p || (shift(p, size) == shift(a.r, 2) && (a.M == 1 || ld % 8 == a.ldr % 8));
  };
  // fp32 rows need 16 of their 32 bytes aligned only, so a shift of four is none
  const bool y_like = like(a.y, a.ldy, sizeof(Y)) ||
                      (sizeof(Y) == 4 && shift(a.r, 2) == 0 && (uintptr_t)a.y % 16 == 0 && (a.M == 1 || a.ldy % 8 == a.ldr % 8));
  const bool gate_like = a.ldg == 0 || like(a.gate, a.ldg, 2);      // one row [D] is read like a vector
  const bool alike = y_like && gate_like && like(a.h, a.ldh, 2) && like(a.out, a.ldo, 2);
  if (!alike) return run_mode<Y, T, APART>(a, s);
  const bool vectors = (uintptr_t)a.gamma_post % 16 == 0 && (uintptr_t)a.gamma_pre % 16 == 0 &&
                       (a.ldg != 0 || (uintptr_t)a.gate % 16 == 0);
  if (a.D % 8 == 0 && shift(a.r, 2) == 0 && (a.M == 1 || a.ldr % 8 == 0) && vectors) return run_mode<Y, T, ALIGNED>(a, s);
  return run_mode<Y, T, SHIFTED>(a, s);
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
