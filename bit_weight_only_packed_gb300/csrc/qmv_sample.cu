// qmv_sample.cu -- logits to probabilities (qmv_softmax) and drafted tokens
// against the target's probabilities (qmv_verify_draft).
#include <math_constants.h>

#include "qmv_step.cuh"

namespace qmv {
namespace {

constexpr int NT = 512, NW = NT / 32;

// ----------------------------------------------------------------- softmax --

// A temperature as the factor of (x - max): 0 stands for the one-hot form.
// 1/T of a subnormal T is infinite; the largest finite factor keeps 0 * it = 0.
__device__ __forceinline__ float inv_temperature(const SoftmaxArgs& a, int row) {
  const float t = a.t ? a.t[row] : a.t0;
  return t > 0.0f ? fminf(1.0f / t, 3.402823466e38f) : 0.0f;
}

template <typename X>
__global__ void __launch_bounds__(NT) softmax_kernel(SoftmaxArgs a) {
  __shared__ float rm[NW], rs[NW];
  __shared__ int ri[NW], rbad[NW];
  const int row = blockIdx.x, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const X* x = (const X*)a.x + (int64_t)row * a.ldx;
  float* out = a.out + (int64_t)row * a.ldo;
  const float t = a.t ? a.t[row] : a.t0, it = inv_temperature(a, row);
  const bool hot = !(t > 0.0f);
  float mx = -CUDART_INF_F;
  int bad = 0, at = a.V;              // at: the first place of the maximum
  for (int i = threadIdx.x; i < a.V; i += NT) {
    const float v = to_f<X>(x[i]);
    if (v > mx) mx = v, at = i;
    bad |= !(v < CUDART_INF_F);
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    const float m2 = __shfl_xor_sync(~0u, mx, o);
    const int a2 = __shfl_xor_sync(~0u, at, o);
    bad |= __shfl_xor_sync(~0u, bad, o);
    if (m2 > mx || (m2 == mx && a2 < at)) mx = m2, at = a2;
  }
  if (lane == 0) rm[warp] = mx, ri[warp] = at, rbad[warp] = bad;
  __syncthreads();
  mx = rm[0], at = ri[0], bad = rbad[0];
  for (int w = 1; w < NW; ++w) {
    bad |= rbad[w];
    if (rm[w] > mx || (rm[w] == mx && ri[w] < at)) mx = rm[w], at = ri[w];
  }
  const bool none = mx == -CUDART_INF_F;
  float s = 0.0f;
  if (!bad && !hot && !none)
    for (int i = threadIdx.x; i < a.V; i += NT) {
      const float v = to_f<X>(x[i]);
      s += v == -CUDART_INF_F ? 0.0f : expf((v - mx) * it);
    }
#pragma unroll
  for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(~0u, s, o);
  if (lane == 0) rs[warp] = s;
  __syncthreads();
  s = 0.0f;
  for (int w = 0; w < NW; ++w) s += rs[w];
  for (int i = threadIdx.x; i < a.V; i += NT) {
    const float v = to_f<X>(x[i]);
    float o;
    if (bad)
      o = CUDART_NAN_F;
    else if (none)
      o = 0.0f;
    else if (hot)
      o = i == at ? 1.0f : 0.0f;
    else
      o = v == -CUDART_INF_F ? 0.0f : expf((v - mx) * it) / s;
    out[i] = o;
  }
}

// ------------------------------------------------------------------ verify --

// A weight in whole units of 2^-42, clamped to 0..1; NaN counts as 0.
__device__ __forceinline__ long long units(float w) {
  w = fminf(fmaxf(w, 0.0f), 1.0f);        // fmaxf(NaN, 0) = 0
  return __float2ll_rz(w * 4398046511104.0f);
}

// The row pair that a sequence's new token is drawn from.  hot: the drafter
// was sure of token d (no row q); q == nullptr and !hot: no refusal.
struct Rows {
  const float *p, *q;
  int hot;
};
__device__ __forceinline__ float rest_of(const Rows& w, int v) {
  float x = w.p[v];
  if (w.q) x = x - w.q[v];
  if (v == w.hot) x -= 1.0f;
  return x;
}

__device__ __forceinline__ long long block_sum(long long v, long long* red) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(~0u, v, o);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  v = 0;
  for (int w = 0; w < NW; ++w) v += red[w];
  return v;
}

// One CTA a sequence: the first refused token, the total, then thread ranges
// in id order until the running sum passes the threshold.
__global__ void __launch_bounds__(NT) verify_kernel(VerifyArgs a) {
  __shared__ long long red[NW], range[NT];
  __shared__ int s_acc;
  const int b = blockIdx.x, V = a.V, S = a.S;
  const int* draft = a.draft + (int64_t)b * S;
  int n = a.n_draft ? a.n_draft[b] : S;
  n = max(0, min(n, S));
  const float* p0 = a.p + (int64_t)b * (S + 1) * V;
  const float* q0 = a.q ? a.q + (int64_t)b * S * V : nullptr;
  if (threadIdx.x == 0) s_acc = n;
  __syncthreads();
  for (int i = threadIdx.x; i < n; i += NT) {
    const int d = draft[i];
    bool ok = d >= 0 && d < V;
    if (ok) {
      const double p = p0[(int64_t)i * V + d], q = q0 ? (double)q0[(int64_t)i * V + d] : 1.0;
      ok = (double)a.ua[(int64_t)b * S + i] * q < p;     // 48 bits: exact
    }
    if (!ok) atomicMin(&s_acc, i);
  }
  __syncthreads();
  const int acc = s_acc;
  const bool refused = acc < n;
  Rows w{p0 + (int64_t)acc * V, nullptr, -1};
  if (refused) {
    if (q0) w.q = q0 + (int64_t)acc * V;
    else w.hot = draft[acc];
  }
  // thread ranges of consecutive ids
  const int per = (V + NT - 1) / NT, v0 = min(V, (int)threadIdx.x * per), v1 = min(V, v0 + per);
  long long mine = 0, total = 0;
  for (int pass = 0; pass < 2; ++pass) {
    mine = 0;
    for (int v = v0; v < v1; ++v) mine += units(rest_of(w, v));
    total = block_sum(mine, red);
    if (total > 0 || !refused) break;
    w.q = nullptr, w.hot = -1;          // no mass is left: draw from p
  }
  range[threadIdx.x] = mine;
  __syncthreads();
  if (threadIdx.x == 0) {
    int tok = -1;
    if (total > 0) {
      const float us = a.us[b];
      const unsigned long long U = (unsigned long long)fminf(fmaxf(us, 0.0f) * 2147483648.0f, 2147483520.0f);
      const unsigned long long T = (unsigned long long)total;
      const long long t = (long long)(((U * (T >> 32)) << 1) + ((U * (T & 0xffffffffull)) >> 31));
      long long run = 0;
      int r = 0;
      while (run + range[r] <= t) run += range[r++];
      for (int v = r * per;; ++v) {
        run += units(rest_of(w, v));
        if (run > t) {
          tok = v;
          break;
        }
      }
    }
    int* out = a.tokens + (int64_t)b * (S + 1);
    for (int i = 0; i <= S; ++i) out[i] = i < acc ? draft[i] : i == acc ? tok : -1;
    a.n_acc[b] = acc;
  }
}

}  // namespace

cudaError_t launch_softmax(const SoftmaxArgs& a, cudaStream_t s) {
  switch (a.dtype) {
    case QMV_F32: softmax_kernel<float><<<a.rows, NT, 0, s>>>(a); break;
    case QMV_F16: softmax_kernel<__half><<<a.rows, NT, 0, s>>>(a); break;
    default: softmax_kernel<__nv_bfloat16><<<a.rows, NT, 0, s>>>(a); break;
  }
  return cudaGetLastError();
}

cudaError_t launch_verify(const VerifyArgs& a, cudaStream_t s) {
  verify_kernel<<<a.B, NT, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace qmv
