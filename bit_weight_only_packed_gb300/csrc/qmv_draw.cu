// qmv_draw.cu -- one token a row of logits, from given random numbers (qmv_sample).
#include <math_constants.h>

#include "qmv_token.cuh"

namespace qmv {

int read_draw_error(int clear, int* out) {
  *out = 0;
  return 0;
}

namespace {

typedef unsigned long long u64;
constexpr int NT = 1024;

// fp32 as a whole number of the same order; NaN and -inf, which are never drawn, are 0.
__device__ __forceinline__ uint32_t ordered(float v) {
  if (!(v > -CUDART_INF_F)) return 0u;
  const uint32_t b = __float_as_uint(v + 0.0f);            // -0 counts as 0
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float unordered(uint32_t k) {
  return __uint_as_float(k & 0x80000000u ? k & 0x7fffffffu : ~k);
}

// exp((x - top) / T) in whole units of 2^-42 (qmv.h has the steps).
__device__ __forceinline__ u64 weight(float x, float top, float c) {
  const float z = x == top ? 0.0f : fminf(__fmul_rn(__fsub_rn(top, x), c), 64.0f);
  const float n = rintf(z), f = n - z;
  float p = 0.0013381302123889327f;
  p = fmaf(p, f, 0.00966636836528778f);
  p = fmaf(p, f, 0.055503811687231064f);
  p = fmaf(p, f, 0.2402234971523285f);
  p = fmaf(p, f, 0.6931471824645996f);
  p = fmaf(p, f, 1.0f);
  const uint32_t b = __float_as_uint(p);
  const u64 m = (b & 0x7fffffu) | 0x800000u;               // p = m * 2^(exponent - 150)
  const int s = (int)(b >> 23) - 108 - (int)n;             // w = m * 2^s
  return s >= 0 ? m << s : s > -24 ? m >> -s : 0;
}

// floor(total * u / 2^31)
__device__ __forceinline__ u64 share(u64 total, u64 u) { return ((u * (total >> 32)) << 1) + ((u * (total & 0xffffffffull)) >> 31); }

__device__ __forceinline__ u64 block_sum(u64 v, u64* red, u64* before) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  u64 run = v;
  for (int o = 1; o < 32; o <<= 1) {
    const u64 t = __shfl_up_sync(~0u, run, o);
    if (lane >= o) run += t;
  }
  __syncthreads();
  if (lane == 31) red[w] = run;
  __syncthreads();
  u64 base = 0, all = 0;
  for (int i = 0; i < NT / 32; ++i) {
    if (i < w) base += red[i];
    all += red[i];
  }
  *before = base + run - v;
  return all;
}

// A CTA a row; a thread takes neighbouring ids.
template <typename X>
__global__ void __launch_bounds__(NT) draw_kernel(DrawArgs a) {
  __shared__ u64 red[NT / 32], bins[256];
  __shared__ uint32_t s_top, s_digit;
  __shared__ u64 s_above;
  pdl_begin();
  const int row = blockIdx.x, per = (a.V + NT - 1) / NT, i0 = min(a.V, (int)threadIdx.x * per), i1 = min(a.V, i0 + per);
  const X* x = (const X*)a.x + (int64_t)row * a.ldx;
  float t = a.t ? a.t[row] : a.t0;
  const int k = a.k ? a.k[row] : a.k0;
  const float tp = a.p ? a.p[row] : a.p0, mp = a.m ? a.m[row] : a.m0;
  const bool all_p = !(tp < 1.0f);
  const u64 P = (u64)(fmaxf(tp, 0.0f) * 2147483648.0f), U = (u64)fminf(fmaxf(a.u[row], 0.0f) * 2147483648.0f, 2147483520.0f);
  const u64 least = (u64)((double)fminf(fmaxf(mp, 0.0f), 1.0f) * 4398046511104.0);
  if (threadIdx.x == 0) s_top = 0;
  __syncthreads();
  uint32_t top = 0;
  for (int i = i0; i < i1; ++i) top = max(top, ordered(to_f<X>(x[i])));
  atomicMax(&s_top, top);
  __syncthreads();
  top = s_top;
  const float mx = unordered(top);
  const bool greedy = !(t > 0.0f);
  const float c = 1.4426950408889634f / fmaxf(t, 0x1p-100f);
  // what stays: keys above `cut`, and the first `ties` (by id) of those equal to it
  uint32_t cut = 0;
  u64 ties = ~0ull;
  if (greedy) cut = top, ties = 1;
  for (int pass = 0; pass < 2 && !greedy; ++pass) {
    // pass 0: so that k ids stay; pass 1: so that their sum reaches top_p
    if (pass == 0 ? k <= 0 || k >= a.V : all_p) continue;
    u64 rank = 0, before, need = (u64)k;
    if (pass == 1) {
      for (int i = i0; i < i1; ++i) rank += ordered(to_f<X>(x[i])) == cut;
      block_sum(rank, red, &before);
      u64 sum = 0, n = before;
      for (int i = i0; i < i1; ++i) {
        const uint32_t o = ordered(to_f<X>(x[i]));
        if (o && (o > cut || (o == cut && n++ < ties))) sum += weight(to_f<X>(x[i]), mx, c);
      }
      u64 at;
      need = share(block_sum(sum, red, &at), P);
      if (need == 0) need = 1;
      rank = before;
    }
    uint32_t prefix = 0;
    u64 above = 0;
    for (int shift = 24; shift >= 0; shift -= 8) {
      if (threadIdx.x < 256) bins[threadIdx.x] = 0;
      __syncthreads();
      u64 n = rank;
      for (int i = i0; i < i1; ++i) {
        const uint32_t o = ordered(to_f<X>(x[i]));
        const bool in = pass == 0 || o > cut || (o == cut && n++ < ties);
        if (in && (shift == 24 || o >> (shift + 8) == prefix >> (shift + 8)))
          atomicAdd(&bins[o >> shift & 255], pass == 0 ? 1ull : o ? weight(to_f<X>(x[i]), mx, c) : 0ull);
      }
      __syncthreads();
      if (threadIdx.x == 0) {
        int d = 255;
        for (; d > 0 && above + bins[d] < need; --d) above += bins[d];
        s_digit = d;
        s_above = above;
      }
      __syncthreads();
      prefix |= s_digit << shift;
      above = s_above;
      __syncthreads();
    }
    // equal logits have equal weights
    const u64 w = pass == 0 ? 1 : prefix ? weight(unordered(prefix), mx, c) : 1;
    const u64 more = w ? (need - above + w - 1) / w : 1;
    if (pass == 0 || prefix > cut) cut = prefix, ties = more;
    else ties = min(ties, more);
  }
  u64 before, sum = 0, n = 0;
  for (int i = i0; i < i1; ++i) n += ordered(to_f<X>(x[i])) == cut;
  block_sum(n, red, &before);
  n = before;
  const auto stays = [&](float v, u64& n) -> u64 {
    const uint32_t o = ordered(v);
    if (!o || !(o > cut || (o == cut && n++ < ties))) return 0;
    const u64 w = greedy ? 1 : weight(v, mx, c);
    return greedy || w >= least ? w : 0;
  };
  for (int i = i0; i < i1; ++i) sum += stays(to_f<X>(x[i]), n);
  u64 run;
  const u64 total = block_sum(sum, red, &run), at = share(total, U);
  if (total == 0) {
    if (threadIdx.x == 0) a.tokens[row] = -1;
  } else if (run <= at && at < run + sum) {
    n = before;
    for (int i = i0; i < i1; ++i) {
      run += stays(to_f<X>(x[i]), n);
      if (run > at) {
        a.tokens[row] = i;
        break;
      }
    }
  }
}

}  // namespace

cudaError_t launch_draw(const DrawArgs& a, cudaStream_t s) {
  const dim3 grid((unsigned)a.rows);
  switch (a.dtype) {
    case QMV_F32: return launch_step(draw_kernel<float>, grid, NT, 0, s, 1, a);
    case QMV_F16: return launch_step(draw_kernel<__half>, grid, NT, 0, s, 1, a);
    default: return launch_step(draw_kernel<__nv_bfloat16>, grid, NT, 0, s, 1, a);
  }
}

}  // namespace qmv
