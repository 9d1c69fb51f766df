// qmv_experts.cu -- products of 4-bit expert weights with the tokens routed to them
// (qmv_w4_experts), on the packed layout of qmv_w4.cu.
#include "qmv_pipe.cuh"
#include "qmv_token.cuh"

namespace qmv {

static __device__ int g_experts_error = 0;

int read_experts_error(int clear, int* out) {
  cudaError_t e = cudaMemcpyFromSymbol(out, g_experts_error, sizeof(int));
  if (e == cudaSuccess && clear && *out) {
    const int z = 0;
    e = cudaMemcpyToSymbol(g_experts_error, &z, sizeof(int));
  }
  return (int)e;
}

namespace {

using namespace w4;

__device__ __forceinline__ float f16_of(uint32_t bits16, int bf16) {
  return bf16 ? __uint_as_float(bits16 << 16) : __half2float(__ushort_as_half((unsigned short)bits16));
}

// act(gate) * up, rounded to x's type.
__device__ __forceinline__ float gated(float g, float u, int act, int bf16) {
  float v;
  if (act == QMV_ACT_SILU) {
    v = g / (1.0f + expf(-g)) * u;
  } else {
    const float t = 0.7978845608028654f * (g + 0.044715f * g * g * g);
    v = 0.5f * g * (1.0f + tanhf(t)) * u;
  }
  return bf16 ? __bfloat162float(__float2bfloat16_rn(v)) : __half2float(__float2half_rn(v));
}

// One thread a result row.
__global__ void __launch_bounds__(128) experts_kernel(ExpertsArgs a) {
  pdl_begin();
  const int r = blockIdx.x * 128 + threadIdx.x;
  if (r >= a.R) return;
  const int KB = cdiv(a.K, BK), bb = block_bytes(a.group, a.zeros != 0), gpb = BK / a.group;
  for (int out = blockIdx.y; out < (a.weights ? a.M : a.M * a.T); out += gridDim.y) {
    float y = 0.0f;
    const int first = a.weights ? out * a.T : out, last = a.weights ? first + a.T : out + 1;
    for (int p = first; p < last; ++p) {
      const int e = a.ids[p];
      if ((unsigned)e >= (unsigned)a.E) {
        if (e != -1) atomicCAS(&g_experts_error, 0, pipe::ERR_BAD_EXPERT);
        continue;
      }
      const uint16_t* x = (const uint16_t*)a.x + (int64_t)(a.per_pair ? p : p / a.T) * a.ldx;
      const int n = e * a.R + r, row = n & 31, half = row >> 4, hi = (row >> 3) & 1;
      float v = 0.0f, sum = 0.0f, s = 0.0f;
      int z = 8;
      for (int k = 0; k < a.K; ++k) {
        const uint8_t* b = a.packed + ((int64_t)(n >> 5) * KB + (k >> 7)) * bb;
        if (k % a.group == 0) {
          v += sum * s;
          sum = 0.0f;
          const uint8_t* meta = b + CODE_BYTES;
          const int at = (k & 127) / a.group * ROWS + meta_slot(row);
          s = f16_of(reinterpret_cast<const uint16_t*>(meta)[at], a.scale_bf16);
          if (a.zeros) z = meta[2 * gpb * ROWS + at];
        }
        const int j = (k >> 6) & 1, h = (k >> 5) & 1, lane = (row & 7) * 4 + ((k >> 3) & 3);
        const uint32_t w = reinterpret_cast<const uint32_t*>(b)[((half * 2 + j) * 32 + lane) * 4 + hi * 2 + h];
        const int shift = shift_of(k & 7), code = (int)(__funnelshift_r(w, w, shift) & 15u);
        float xv = f16_of(x[k], a.x_bf16);
        if (a.act != QMV_ACT_NONE) xv = gated(xv, f16_of(x[a.K + k], a.x_bf16), a.act, a.x_bf16);
        sum = fmaf(xv, (float)(code - z), sum);
      }
      v += sum * s;
      y += a.weights ? a.weights[p] * v : v;
    }
    const int64_t at = (int64_t)out * a.ldy + r;
    if (a.y_dtype == QMV_F32)
      ((float*)a.y)[at] = y;
    else if (a.y_dtype == QMV_F16)
      ((__half*)a.y)[at] = __float2half_rn(y);
    else
      ((__nv_bfloat16*)a.y)[at] = __float2bfloat16_rn(y);
  }
}

}  // namespace

size_t experts_workspace(int K, int group, int R, int M, int T, int E) { return 0; }

cudaError_t launch_experts(const ExpertsArgs& a, cudaStream_t s) {
  const int outs = a.weights ? a.M : a.M * a.T;
  return launch_step(experts_kernel, dim3((a.R + 127) / 128, outs < 65535 ? outs : 65535), 128, 0, s, 1, a);
}

}  // namespace qmv
