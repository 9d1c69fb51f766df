// qmv_route.cu -- the experts of each token and their weights (qmv_route).
//
// A warp takes a token and its lanes N neighbouring experts each, all in registers.  A group's
// worth comes through shared memory (any number of groups of any size); the T largest
// ranks are taken one after another, each with one maximum over the warp.
//
// Ranks are compared as exact arithmetic has them.  Without a bias they follow the
// logits, which are compared themselves.  Otherwise fp32 ranks decide where neighbours in
// the order are further apart than their errors add up to; a token where they are not is
// ranked again in 64 bits (about one in a thousand of 256 experts).
#include <math_constants.h>

#include "qmv_token.cuh"

namespace qmv {
namespace {

constexpr int WARPS = 4, MAX_E = 1024;

// fp32 as a whole number of the same order (NaN does not occur).
__device__ __forceinline__ uint32_t ordered(float v) {
  const uint32_t b = __float_as_uint(v + 0.0f);            // -0 counts as 0
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float unordered(uint32_t k) {
  return __uint_as_float(k & 0x80000000u ? k & 0x7fffffffu : ~k);
}

__device__ __forceinline__ float warp_max(float v) { return unordered(__reduce_max_sync(~0u, ordered(v))); }
__device__ __forceinline__ double warp_max(double v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v = fmax(v, __shfl_xor_sync(~0u, v, o));
  return v;
}
template <typename F>
__device__ __forceinline__ F warp_total(F v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(~0u, v, o);
  return v;
}

// What a score may be off by in fp32: a sigmoid by an ulp of its exponential (1 at most) and two
// roundings; a softmax, relative to itself, by |x - max| 2^-24 (times p: 2^-25 at most), two
// ulps, the sum of 32 partial sums of up to 32 terms, and two roundings.
template <typename F>
__device__ __forceinline__ F score_error(int score) {
  return sizeof(F) == 8 ? (F)0 : score == QMV_SCORE_SIGMOID ? (F)0x1p-22 : (F)0x1p-19;
}

// Scores of a lane's N experts, exps in F.  x: logits, those that cannot be chosen -inf.
template <typename F, int N>
__device__ __forceinline__ void scores(const float (&x)[N], int score, F (&s)[N]) {
  if (score == QMV_SCORE_SIGMOID) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const F e = exp(-fabs((F)x[i]));
      s[i] = (x[i] >= 0.0f ? (F)1 : e) / ((F)1 + e);
    }
    return;
  }
  float top = -CUDART_INF_F;
#pragma unroll
  for (int i = 0; i < N; ++i) top = fmaxf(top, x[i]);
  top = warp_max(top);
  F sum = 0;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    s[i] = x[i] == -CUDART_INF_F ? (F)0 : x[i] == top ? (F)1 : exp((F)x[i] - (F)top);
    sum += s[i];
  }
  sum = warp_total(sum);
#pragma unroll
  for (int i = 0; i < N; ++i) s[i] = sum > 0 ? s[i] / sum : (F)0;
}

// The choice of one token with scores in F: lane t % 32 receives pick t (place t / 32) with its
// score.  Returns whether F could tell all that it had to; rank: a warp's [E] in shared memory.
template <typename F, int N>
__device__ __forceinline__ bool choose(const RouteArgs& a, const float (&x)[N], const float (&b)[N], int lane, F* rank,
                                       int (&id)[2], float (&w)[2]) {
  const F none = (F)(-CUDART_INF_F);
  const int e0 = lane * N;
  F s[N], r[N];
  scores<F, N>(x, a.score, s);
  const F err = score_error<F>(a.score);
  bool sure = true;
  uint32_t left = ~0u;                               // one bit a group
  if (a.groups > 1) {
    const int per = a.E / a.groups;
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (e0 + i < a.E) rank[e0 + i] = x[i] == -CUDART_INF_F ? none : s[i] + (F)b[i];
    __syncwarp();
    int G = 1, g_log = 0;
    while (G < a.groups) G *= 2, ++g_log;
    const int sub = 32 >> g_log, g = lane >> (5 - g_log);      // `sub` lanes a group
    F one = none, two = none;
    if (g < a.groups)
      for (int i = lane & (sub - 1); i < per; i += sub) {
        const F v = rank[g * per + i];
        two = fmax(two, fmin(one, v));
        one = fmax(one, v);
      }
    for (int o = sub >> 1; o; o >>= 1) {
      const F v = __shfl_xor_sync(~0u, one, o), v2 = __shfl_xor_sync(~0u, two, o);
      two = fmax(fmax(two, v2), fmin(one, v));
      one = fmax(one, v);
    }
    // lane g has group g's
    const F worth = __shfl_sync(~0u, a.group_top == 2 ? one + two : one, (lane * sub) & 31);
    int better = 0;
    for (int j = 0; j < a.groups; ++j) {
      const F v = __shfl_sync(~0u, worth, j);
      better += v > worth || (v == worth && j < lane);
    }
    const bool in = lane < a.groups && better < a.group_k;
    left = __ballot_sync(~0u, in);
    if (sizeof(F) == 4 && a.group_k < a.groups) {
      // the last group that stays and the first that does not
      const F last = __shfl_sync(~0u, worth, __ffs(__ballot_sync(~0u, lane < a.groups && better == a.group_k - 1)) - 1);
      const F next = __shfl_sync(~0u, worth, __ffs(__ballot_sync(~0u, lane < a.groups && better == a.group_k)) - 1);
      sure = last - next > 4 * err + (F)0x1p-21 * (fabs(last) + fabs(next)) || next == none;
    }
#pragma unroll
    for (int i = 0; i < N; ++i)
      r[i] = e0 + i < a.E && !(left >> ((e0 + i) / per) & 1) ? none : x[i] == -CUDART_INF_F ? none : a.bias ? s[i] + (F)b[i] : (F)x[i];
    __syncwarp();
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) r[i] = x[i] == -CUDART_INF_F ? none : a.bias ? s[i] + (F)b[i] : (F)x[i];
  }
  F before = none;
  float x_before = 0.0f, b_before = 0.0f;
  for (int t = 0; t <= a.T; ++t) {                   // one more than is wanted, to tell the last apart
    if (t == a.T && (!a.bias || sizeof(F) == 8)) break;
    F best = r[0];
#pragma unroll
    for (int i = 1; i < N; ++i) best = fmax(best, r[i]);
    const F top = warp_max(best);
    if (top == none) {
      if (lane == (t & 31) && t < a.T) id[t >> 5] = -1, w[t >> 5] = 0.0f;
      continue;
    }
    const int owner = __ffs(__ballot_sync(~0u, best == top)) - 1;
    int at = 0;
    float sv = 0.0f, xv = 0.0f, bv = 0.0f;
    bool found = false;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const bool hit = !found && lane == owner && r[i] == top;
      if (hit) at = e0 + i, sv = (float)s[i], xv = x[i], bv = b[i], r[i] = none;
      found |= hit;
    }
    if (a.bias && sizeof(F) == 4) {
      xv = __shfl_sync(~0u, xv, owner), bv = __shfl_sync(~0u, bv, owner);
      // equal ones of the same logit and bias are truly equal
      if (t > 0 && !(before - top > 2 * err + (F)0x1p-22 * (fabs(before) + fabs(top))) && !(xv == x_before && bv == b_before))
        sure = false;
      before = top, x_before = xv, b_before = bv;
    }
    at = __shfl_sync(~0u, at, owner), sv = __shfl_sync(~0u, sv, owner);
    if (lane == (t & 31) && t < a.T) id[t >> 5] = at, w[t >> 5] = sv;
  }
  return sure;
}

template <int N>
__device__ __noinline__ void choose_wide(const RouteArgs& a, const float* xb, int lane, double* rank, int (&id)[2], float (&w)[2]) {
  float x[N], b[N];
#pragma unroll
  for (int i = 0; i < N; ++i) x[i] = xb[i], b[i] = xb[N + i];
  choose<double, N>(a, x, b, lane, rank, id, w);
}

template <typename X, int N>
__global__ void __launch_bounds__(WARPS * 32) route_kernel(RouteArgs a) {
  __shared__ double ranks[WARPS][N * 32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, e0 = lane * N;
  pdl_begin();
  const int64_t m = (int64_t)blockIdx.x * WARPS + warp;
  if (m >= a.M) return;
  const X* row = (const X*)a.x + m * a.ldx;
  float xb[2 * N];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int e = e0 + i;
    float x = -CUDART_INF_F, b = 0.0f;
    if (e < a.E) {
      x = to_f<X>(row[e]);
      if (a.bias) b = a.bias[e];
    }
    // what cannot be chosen: NaN or -inf in either
    if (isnan(x) || isnan(b) || b == -CUDART_INF_F) x = -CUDART_INF_F, b = 0.0f;
    xb[i] = x, xb[N + i] = b;
  }
  int id[2] = {-1, -1};
  float w[2] = {0.0f, 0.0f};
  {
    float x[N], b[N];
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = xb[i], b[i] = xb[N + i];
    if (!choose<float, N>(a, x, b, lane, reinterpret_cast<float*>(ranks[warp]), id, w))
      choose_wide<N>(a, xb, lane, ranks[warp], id, w);
  }
  float f = a.scale;
  if (a.renorm) {
    const float sum = warp_total(w[0] + w[1]);
    f = sum > 0.0f ? a.scale / sum : 0.0f;
  }
#pragma unroll
  for (int p = 0; p < 2; ++p)
    if (lane + 32 * p < a.T) {
      a.ids[m * a.T + lane + 32 * p] = id[p];
      a.w[m * a.T + lane + 32 * p] = w[p] * f;
    }
}

template <typename X>
cudaError_t typed(const RouteArgs& a, cudaStream_t s) {
  const dim3 grid((unsigned)(((int64_t)a.M + WARPS - 1) / WARPS));
  if (a.E <= 32) return launch_step(route_kernel<X, 1>, grid, WARPS * 32, 0, s, 1, a);
  if (a.E <= 64) return launch_step(route_kernel<X, 2>, grid, WARPS * 32, 0, s, 1, a);
  if (a.E <= 128) return launch_step(route_kernel<X, 4>, grid, WARPS * 32, 0, s, 1, a);
  if (a.E <= 256) return launch_step(route_kernel<X, 8>, grid, WARPS * 32, 0, s, 1, a);
  if (a.E <= 512) return launch_step(route_kernel<X, 16>, grid, WARPS * 32, 0, s, 1, a);
  return launch_step(route_kernel<X, 32>, grid, WARPS * 32, 0, s, 1, a);
}

}  // namespace

cudaError_t launch_route(const RouteArgs& a, cudaStream_t s) {
  switch (a.dtype) {
    case QMV_F32: return typed<float>(a, s);
    case QMV_F16: return typed<__half>(a, s);
    default: return typed<__nv_bfloat16>(a, s);
  }
}

}  // namespace qmv
