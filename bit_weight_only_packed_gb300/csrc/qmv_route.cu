// qmv_route.cu -- the experts of each token and their weights (qmv_route).
//
// A warp takes a token and its lanes N neighbouring experts each, all in registers.  A group's worth comes by
// exchanges within the warp where its experts are whole lanes', otherwise through shared memory.  The lanes'
// largest ranks, sorted, give a bound that T + 1 experts reach; the few that reach it, one a lane, are sorted
// into the answer.  Where T is 32 or more, or ties leave no bound that 32 reach, experts are taken one after another, each
// with a maximum over the warp.
//
// Ranks are compared as exact arithmetic has them.  Without a bias they follow the logits, which are compared
// themselves.  Otherwise fp32 ranks decide where neighbours in the order, and the last pick and all behind it, are
// further apart than their errors add up to, or truly equal.  Where they are not (about one token in a thousand of
// 256 experts) the choice of groups, or the order of the few, is formed again in 64 bits, or all of it where a
// softmax needs that.
//
// Bound by instructions where tokens are many, 1235 a token: 16384 tokens of 256 experts in 8 groups
// took 62 us with a maximum over the warp an expert and loads under conditions, 36 with unconditional loads and
// the sort, 27 since only ranks that are near each other are formed in 64 bits (exchanges and compares; HBM
// would take 2.6).  One token is bound by latency: 2.8 us.
#include <math_constants.h>

#include "qmv_token.cuh"

namespace qmv {
namespace {

typedef unsigned long long u64;
constexpr int WARPS = 4, MAX_E = 1024;
constexpr int MAX_SORTED = 31;     // picks by sorting: one more than T have to fit in 32

// One of the experts that may be chosen.
struct alignas(16) Few {
  float rank, x, b;
  int e;
};

// fp32 as a whole number of the same order (NaN does not occur).
__device__ __forceinline__ uint32_t ordered(float v) {
  const uint32_t b = __float_as_uint(v + 0.0f);            // -0 counts as 0
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float unordered(uint32_t k) {
  return __uint_as_float(k & 0x80000000u ? k & 0x7fffffffu : ~k);
}

// Keys of a warp's first n lanes in falling order, equal ones by `who`; the others' come last.
template <typename K>
__device__ __forceinline__ void sort_lanes(K& key, uint32_t& who, int n, int lane) {
#pragma unroll
  for (int size = 2; size <= 32; size *= 2) {
    if (size == 32 && n <= 16) break;                                    // the others are behind those anyway
#pragma unroll
    for (int step = size / 2; step; step /= 2) {
      const K k = __shfl_xor_sync(~0u, key, step);
      const uint32_t w = __shfl_xor_sync(~0u, who, step);
      const bool theirs = k > key || (k == key && w < who);              // comes first
      if ((((lane & size) == 0) == ((lane & step) == 0)) == theirs) key = k, who = w;
    }
  }
}
// The lanes' values in falling order.
__device__ __forceinline__ float sort_lanes(float v, int lane) {
#pragma unroll
  for (int size = 2; size <= 32; size *= 2)
#pragma unroll
    for (int step = size / 2; step; step /= 2) {
      const float o = __shfl_xor_sync(~0u, v, step);
      v = ((lane & size) == 0) == ((lane & step) == 0) ? fmaxf(v, o) : fminf(v, o);
    }
  return v;
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

// e^v, v <= 88, and a / b for b from 1 on; in fp32 by the exponential and reciprocal instructions: off
// by |v| 2^-23 + 2^-22 and 2^-22 of themselves.  (The weights of those that are chosen are formed from
// their logits again, with expf.)
__device__ __forceinline__ double exp_of(double v) { return exp(v); }
__device__ __forceinline__ double over(double a, double b) { return a / b; }
__device__ __forceinline__ float exp_of(float v) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v * 1.4426950408889634f));
  return r;
}
__device__ __forceinline__ float over(float a, float b) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(b));
  return a * r;
}

// What a score may be off by in fp32.  A sigmoid 1 / (1 + e): e's error counts s (1 - s) times, and
// x s (1 - s) is below 1/4, so 2^-25 + 2^-24; the sum 2^-24, the reciprocal 2^-23, the product 2^-24.  A
// softmax p = largest e^-d, d = max - x, relative to itself: d 2^-24 for its argument, expf's 2^-23, the sum of
// 32 sums of up to 32 terms 37 2^-24, over() 2^-22: (43 + d) 2^-24.  As a number it is greatest for d = 0:
// below 2^-18 of `largest`, what a score is at most.
template <typename F>
__device__ __forceinline__ F score_error(int score, F largest) {
  return sizeof(F) == 8 ? (F)0 : score == QMV_SCORE_SIGMOID ? (F)0x1p-21 : (F)0x1p-18 * largest;
}

__device__ __forceinline__ float sigmoid(float x) { return over(1.0f, 1.0f + exp_of(-x)); }
// (e^-x is infinite below -709, where the score is still a number)
__device__ __forceinline__ double sigmoid(double x) {
  const double e = exp_of(-fabs(x));
  return (x < 0.0 ? e : 1.0) / (1.0 + e);
}

// Scores of a lane's N experts.  x: logits, those that cannot be chosen -inf.  Returns the largest logit,
// and in *whole the sum of exp(x - that) (softmax).
template <typename F, int N>
__device__ __forceinline__ float scores(const float (&x)[N], int score, F (&s)[N], F* whole) {
  if (score == QMV_SCORE_SIGMOID) {
#pragma unroll
    for (int i = 0; i < N; ++i) s[i] = sigmoid((F)x[i]);
    return 0.0f;
  }
  float top = -CUDART_INF_F;
#pragma unroll
  for (int i = 0; i < N; ++i) top = fmaxf(top, x[i]);
  top = warp_max(top);
  F sum = 0;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    // expf in the sum, whose error is all weights'
    s[i] = x[i] == -CUDART_INF_F ? (F)0 : x[i] == top ? (F)1 : exp((F)x[i] - (F)top);
    sum += s[i];
  }
  *whole = sum = warp_total(sum);
#pragma unroll
  for (int i = 0; i < N; ++i) s[i] = sum > 0 ? over(s[i], sum) : (F)0;
  return top;
}

__device__ __forceinline__ int group_of(const RouteArgs& a, int e) {
  return a.per == 1 ? e : (int)__umulhi((uint32_t)e, a.per_inv);
}

// What choose_groups() knows of lane g's group g, and between which worths fp32 cannot tell.
template <typename F>
struct Groups {
  F worth, reach, low, high;
  bool sure;
};

// The groups that remain, a bit each.  r: ranks, or logits without a bias; top: as scores() gives it;
// rank: a warp's [E] in shared memory.
template <typename F, int N>
__device__ __forceinline__ uint32_t choose_groups(const RouteArgs& a, const F (&r)[N], float top, F largest, int lane, F* rank, Groups<F>* known) {
  const F none = (F)(-CUDART_INF_F);
  const int per = a.per, lanes = per / N, e0 = lane * N;
  F one = none, two = none;                          // lane g: the largest of group g
  if (per % N == 0 && (lanes & (lanes - 1)) == 0) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      two = fmax(two, fmin(one, r[i]));
      one = fmax(one, r[i]);
    }
    for (int o = 1; o < lanes; o <<= 1) {
      const F v = __shfl_xor_sync(~0u, one, o), v2 = __shfl_xor_sync(~0u, two, o);
      two = fmax(fmax(two, v2), fmin(one, v));
      one = fmax(one, v);
    }
    one = __shfl_sync(~0u, one, (lane * lanes) & 31), two = __shfl_sync(~0u, two, (lane * lanes) & 31);
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (e0 + i < a.E) rank[e0 + i] = r[i];
    __syncwarp();
    int G = 1, g_log = 0;
    while (G < a.groups) G *= 2, ++g_log;
    const int sub = 32 >> g_log, g = lane >> (5 - g_log);      // `sub` lanes a group
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
    one = __shfl_sync(~0u, one, (lane * sub) & 31), two = __shfl_sync(~0u, two, (lane * sub) & 31);
    __syncwarp();
  }
  F worth = one;
  if (a.group_top == 2) {
    // logits: their scores, up to a softmax's sum
    const auto score_of = [&](F v) {
      return v == none ? none : a.score == QMV_SCORE_SIGMOID ? sigmoid(v) : v == (F)top ? (F)1 : exp_of(v - (F)top);
    };
    worth = two == none ? none : a.bias ? one + two : score_of(one) + score_of(two);
  }
  int better = 0;
  for (int j = 0; j < a.groups; ++j) {
    const F v = __shfl_sync(~0u, worth, j);
    better += v > worth || (v == worth && j < lane);
  }
  if (sizeof(F) == 4 && a.group_k < a.groups && (a.bias || a.group_top == 2)) {
    // the last group that stays and the first that does not: apart, or all that are near them truly equal
    const int l = __ffs(__ballot_sync(~0u, lane < a.groups && better == a.group_k - 1)) - 1,
              m = __ffs(__ballot_sync(~0u, lane < a.groups && better == a.group_k)) - 1;
    const F last = __shfl_sync(~0u, worth, l), next = __shfl_sync(~0u, worth, m), one_l = __shfl_sync(~0u, one, l),
            two_l = __shfl_sync(~0u, two, l);
    const bool same = !a.bias && one == one_l && two == two_l;
    const F err = 4 * score_error<F>(a.score, a.bias ? largest : (F)1) + (F)0x1p-22 * (fabs(last) + fabs(next));
    const bool odd = __any_sync(~0u, lane < a.groups && !(worth < next - err) && !(worth > last + err) && !same);
    // (a sum of two large biases may be infinite in fp32: that is no proof either)
    const bool none_out = !__any_sync(~0u, lane < a.groups && better >= a.group_k && (a.group_top == 2 ? two : one) != none);
    known->sure = last - next > err || none_out || !odd;
    // a group's best two in exact arithmetic are among those that reach the second less their errors
    known->worth = worth, known->reach = (a.group_top == 2 ? two : one) - err, known->low = next - err, known->high = last + err;
  }
  return __ballot_sync(~0u, lane < a.groups && better < a.group_k);
}

// Ranks of the groups that do not remain become -inf.
template <typename F, int N>
__device__ __forceinline__ void leave_groups(const RouteArgs& a, F (&r)[N], uint32_t left, int lane) {
  // a lane's experts lie in groups that follow each other
  const int e0 = lane * N, per = a.per;
  int g = group_of(a, e0), next = (g + 1) * per;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    if (e0 + i == next) ++g, next += per;
    if (!(left >> (g & 31) & 1)) r[i] = (F)(-CUDART_INF_F);
  }
}

// The choice of groups in 64 bits.
template <int N>
__device__ __noinline__ uint32_t groups_wide(const RouteArgs& a, const float* xb, int lane, double* rank) {
  float x[N];
  double r[N];
#pragma unroll
  for (int i = 0; i < N; ++i) x[i] = xb[i];
  double whole;
  const float top = scores<double, N>(x, a.score, r, &whole);
#pragma unroll
  for (int i = 0; i < N; ++i) r[i] = x[i] == -CUDART_INF_F ? (double)x[i] : a.bias ? r[i] + (double)xb[N + i] : (double)x[i];
  Groups<double> known;
  return choose_groups<double, N>(a, r, top, 1.0, lane, rank, &known);
}

// The same where a few groups are near each other: only their best experts' ranks are formed in 64 bits,
// one a lane (sigmoid scores and a bias).  Returns 0 where these are more than 32, or what is near infinite.
template <int N>
__device__ __noinline__ uint32_t groups_near(const RouteArgs& a, const float* xb, const float* rb, const Groups<float>& known, int lane, Few* few) {
  if (!(known.high - known.low < CUDART_INF_F)) return 0;
  const uint32_t near = __ballot_sync(~0u, lane < a.groups && known.worth >= known.low && known.worth <= known.high);
  uint32_t in = __ballot_sync(~0u, lane < a.groups && known.worth > known.high);
  int n = 0;
  for (int i = 0; i < N; ++i) {
    const int e = lane * N + i, g = group_of(a, e) & 31;
    const bool one = __shfl_sync(~0u, known.reach, g) <= rb[i] && e < a.E && (near >> g & 1) && rb[i] > -CUDART_INF_F;
    const uint32_t all = __ballot_sync(~0u, one);
    const int at = n + __popc(all & ((1u << lane) - 1));
    if (one && at < 32) few[at] = Few{0.0f, xb[i], xb[N + i], g};
    n += __popc(all);
  }
  __syncwarp();
  if (n > 32) return 0;
  double rank = -CUDART_INF, one = -CUDART_INF, two = -CUDART_INF;
  if (lane < n) rank = sigmoid((double)few[lane].x) + (double)few[lane].b;
  for (int j = 0; j < n; ++j) {
    const double v = __shfl_sync(~0u, rank, j);
    if (few[j].e == lane) two = fmax(two, fmin(one, v)), one = fmax(one, v);
  }
  const double worth = a.group_top == 1 ? one : two == -CUDART_INF ? two : one + two;
  const bool mine = lane < a.groups && (near >> lane & 1);
  int better = 0;
  for (int j = 0; j < a.groups; ++j) {
    const double v = __shfl_sync(~0u, worth, j);
    better += (near >> j & 1) && (v > worth || (v == worth && j < lane));
  }
  const int room = a.group_k - __popc(in);
  in |= __ballot_sync(~0u, mine && better < room);
  __syncwarp();                            // few is written again
  return in;
}

// Experts one after another, of the groups `left`, with ranks in F: lane t % 32 receives pick t (place
// t / 32) with its logit.  Returns whether F could tell.
template <typename F, int N>
__device__ __noinline__ bool choose_each(const RouteArgs& a, const float* xb, uint32_t left, int lane, int (&id)[2], float (&of)[2]) {
  const F none = (F)(-CUDART_INF_F);
  const int e0 = lane * N;
  float x[N], b[N];
  F s[N], r[N];
#pragma unroll
  for (int i = 0; i < N; ++i) x[i] = xb[i], b[i] = xb[N + i];
  F whole = 1;
  scores<F, N>(x, a.score, s, &whole);
  const F err = score_error<F>(a.score, 1 / whole);
#pragma unroll
  for (int i = 0; i < N; ++i) r[i] = x[i] == -CUDART_INF_F ? none : a.bias ? s[i] + (F)b[i] : (F)x[i];
  leave_groups<F, N>(a, r, left, lane);
  bool sure = true;
  F before = none;
  float x_before = 0.0f, b_before = 0.0f;
  for (int t = 0; t < a.T; ++t) {
    F best = r[0];
#pragma unroll
    for (int i = 1; i < N; ++i) best = fmax(best, r[i]);
    const F top = warp_max(best);
    if (top == none) {
      if (lane == (t & 31)) id[t >> 5] = -1;
      before = none;
      continue;
    }
    const int owner = __ffs(__ballot_sync(~0u, best == top)) - 1;
    int at = 0;
    float xv = 0.0f, bv = 0.0f;
    bool found = false;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const bool hit = !found && lane == owner && r[i] == top;
      if (hit) at = e0 + i, xv = x[i], bv = b[i], r[i] = none;
      found |= hit;
    }
    at = __shfl_sync(~0u, at, owner), xv = __shfl_sync(~0u, xv, owner);
    if (a.bias && sizeof(F) == 4) {
      bv = __shfl_sync(~0u, bv, owner);
      // equal ones of the same logit and bias are truly equal
      if (t > 0 && !(before - top > 2 * err + (F)0x1p-22 * (fabs(before) + fabs(top))) && !(xv == x_before && bv == b_before))
        sure = false;
      before = top, x_before = xv, b_before = bv;
    }
    if (lane == (t & 31)) id[t >> 5] = at, of[t >> 5] = xv;
  }
  if (a.bias && sizeof(F) == 4 && before > none) {
    // the last one and the largest of those left that are not truly equal to it
    F best = none;
#pragma unroll
    for (int i = 0; i < N; ++i) best = x[i] == x_before && b[i] == b_before ? best : fmax(best, r[i]);
    const F top = warp_max(best);
    if (top > none && !(before - top > 2 * err + (F)0x1p-22 * (fabs(before) + fabs(top)))) sure = false;
  }
  return sure;
}

// The order of the few in 64 bits (sigmoid scores): lane t has pick t.
__device__ __noinline__ void order_wide(const RouteArgs& a, const Few* few, int n, int lane, int* id, float* of) {
  const Few f = few[lane];
  double rank = -CUDART_INF;
  if (lane < n) rank = sigmoid((double)f.x) + (double)f.b;
  uint32_t who = (lane < n ? f.e : MAX_E) << 5 | lane;
  sort_lanes(rank, who, n, lane);
  const bool in = lane < a.T && rank > -CUDART_INF;
  *id = in ? (int)(who >> 5) : -1;
  *of = few[who & 31].x;
}

// exp(v - top), v <= top, within 2^-21 of itself: what the difference is rounded by, up to 2^-18 of a distance
// of 64, is put right behind it.
__device__ __forceinline__ float exp_below(float v, float top) {
  const float d = v - top, back = d + top;                 // d = v - top + (what follows)
  const float off = (v - back) - (top - (back - d));
  const float e = expf(d);
  return e > 0.0f ? fmaf(e, off, e) : 0.0f;
}

// Weights over their sum where that is small: each relative to the largest of them, so that scores below
// the smallest fp32 number keep their shares (an exponential, a quotient and their sum below 2^-126 are
// off by 2^-148 in all, which is 2^-128 of a sum of 2^-20).  v: logits of a lane's two picks, -inf where there is none.
__device__ __noinline__ float2 small_shares(const RouteArgs& a, float v0, float v1, float top, bool sigmoids) {
  const float m = warp_max(fmaxf(v0, v1));
  const auto share_of = [&](float v) { return v == -CUDART_INF_F ? 0.0f : exp_below(v, m) / (sigmoids ? 1.0f + expf(v) : 1.0f); };
  const float w0 = share_of(v0), w1 = share_of(v1), sum = warp_total(w0 + w1);
  // the sum is 0 where it is so in 64 bits
  const float f = exp((double)m - (sigmoids ? 0.0 : (double)top)) > 0.0 ? a.scale / sum : 0.0f;
  return make_float2(w0 * f, w1 * f);
}

template <typename X, int N, bool VEC>
__global__ void __launch_bounds__(WARPS * 32, N <= 8 ? 10 : 4) route_kernel(RouteArgs a) {
  __shared__ double ranks[WARPS][N * 32];
  __shared__ Few all_few[WARPS][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, e0 = lane * N;
  pdl_begin();
  const int64_t m = (int64_t)blockIdx.x * WARPS + warp;
  if (m >= a.M) return;
  const X* row = (const X*)a.x + m * a.ldx;
  float x[N], b[N];
  // loads without conditions, so that none waits for another
  X raw[N];
  constexpr int EACH = 16 / sizeof(X);
  if constexpr (VEC) {                               // rows and E are whole 16-byte words
    const int last = a.E - EACH;
#pragma unroll
    for (int i = 0; i < N; i += EACH) {
      const uint4 v = *reinterpret_cast<const uint4*>(row + min(e0 + i, last));
      memcpy(raw + i, &v, 16);
    }
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) raw[i] = row[min(e0 + i, a.E - 1)];
  }
#pragma unroll
  for (int i = 0; i < N; ++i) b[i] = 0.0f;
  if (a.bias) {
#pragma unroll
    for (int i = 0; i < N; ++i) b[i] = a.bias[min(e0 + i, a.E - 1)];
  }
  // what cannot be chosen: NaN or -inf in either
#pragma unroll
  for (int i = 0; i < N; ++i) x[i] = to_f<X>(raw[i]) > -CUDART_INF_F ? to_f<X>(raw[i]) : -CUDART_INF_F;
  if (a.bias) {
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (!(b[i] > -CUDART_INF_F)) x[i] = -CUDART_INF_F;
  }
  if (a.E < 32 * N) {
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (e0 + i >= a.E) x[i] = -CUDART_INF_F;
  }
  float s[N], r[N];
  float whole = 1.0f;
  const float top = scores<float, N>(x, a.score, s, &whole), none = -CUDART_INF_F;
  const float largest = a.score == QMV_SCORE_SIGMOID ? 1.0f : whole > 0.0f ? 1.0f / whole : 0.0f;
#pragma unroll
  for (int i = 0; i < N; ++i) r[i] = a.bias && x[i] != none ? s[i] + b[i] : x[i];
  const auto spill = [&](float (&xb)[2 * N]) {
#pragma unroll
    for (int i = 0; i < N; ++i) xb[i] = x[i], xb[N + i] = b[i];
  };
  uint32_t left = ~0u;
  if (a.groups > 1) {
    Groups<float> known;
    known.sure = true;
    left = choose_groups<float, N>(a, r, top, largest, lane, reinterpret_cast<float*>(ranks[warp]), &known);
    if (!known.sure) {
      float xb[2 * N], rb[N];
      spill(xb);
#pragma unroll
      for (int i = 0; i < N; ++i) rb[i] = r[i];
      left = a.bias && a.score == QMV_SCORE_SIGMOID ? groups_near<N>(a, xb, rb, known, lane, all_few[warp]) : 0;
      if (left == 0) left = groups_wide<N>(a, xb, lane, ranks[warp]);
    }
    leave_groups<float, N>(a, r, left, lane);
  }

  int id[2] = {-1, -1};
  float of[2] = {0.0f, 0.0f};                        // their logits
  const float err2 = 2 * score_error<float>(a.score, largest);
  int n = 33;
  Few* few = all_few[warp];
  if (a.T <= MAX_SORTED) {
    // T + 1 experts reach the (T + 1)-th of the lanes' largest ranks.  Where more than 32 do, or experts are left
    // in few lanes, halves of what lies between that and the largest rank of all lead to another bound.
    float best = r[0];
#pragma unroll
    for (int i = 1; i < N; ++i) best = fmaxf(best, r[i]);
    best = sort_lanes(best, lane);
    const auto reach = [&](float v) {
      int c = 0;
#pragma unroll
      for (int i = 0; i < N; ++i) c += r[i] >= v;
      return c;
    };
    // and those that may do so but for their errors (-inf, or inf - inf: all that may be chosen)
    const auto less = [&](float v) { return fmaxf(a.bias ? v - (err2 + 0x1p-21f * fabsf(v)) : v, -3.402823466e38f); };
    float bound = less(__shfl_sync(~0u, best, a.T));
    int mine = reach(bound);
    n = __reduce_add_sync(~0u, mine);
    if (n > 32) {
      uint32_t low = ordered(__shfl_sync(~0u, best, a.T)), high = ordered(__shfl_sync(~0u, best, 0)) + 1;
      while (high - low > 1) {             // T + 1 reach low, and not high
        const uint32_t mid = low + (high - low) / 2;
        const float v = unordered(mid);
        if (__reduce_add_sync(~0u, reach(v)) <= a.T) {
          high = mid;
          continue;
        }
        low = mid;
        bound = less(v);
        mine = reach(bound);
        n = __reduce_add_sync(~0u, mine);
        if (n <= 32) break;
      }
    }
    int at = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(~0u, at, o);
      if (lane >= o) at += v;
    }
    at -= mine;
    if (n <= 32) {
#pragma unroll
      for (int i = 0; i < N; ++i)
        if (r[i] >= bound) few[at++] = Few{r[i], x[i], b[i], e0 + i};
    }
    __syncwarp();
  }
  if (n <= 32) {
    // by rank, then by number: a lane each
    float key = lane < n ? few[lane].rank : none;
    uint32_t who = (lane < n ? few[lane].e : MAX_E) << 5 | lane;
    sort_lanes(key, who, n, lane);
    const bool in = lane < a.T && key > none;
    const Few f = few[who & 31];
    id[0] = in ? (int)(who >> 5) : -1;
    of[0] = f.x;
    if (a.bias) {
      // each pick and the next, and the last pick and each of those behind it
      const int with = lane < a.T - 1 ? lane + 1 : a.T - 1;
      const float key2 = __shfl_sync(~0u, key, with);
      float err = err2;
      if (a.score != QMV_SCORE_SIGMOID) {            // by their own d, and what p itself is off by here
        const float d = top - f.x, own = exp_of(-d) * largest * (48.0f + d) * 0x1p-24f + 0x1p-120f;
        err = own + __shfl_sync(~0u, own, with);
      }
      const bool near = lane != a.T - 1 && key > none && key2 > none &&
                        !(fabsf(key - key2) > err + 0x1p-23f * (fabsf(key) + fabsf(key2)));
      if (__any_sync(~0u, near)) {
        // equal ones of the same logit and bias are truly equal
        const float x2 = __shfl_sync(~0u, f.x, with), b2 = __shfl_sync(~0u, f.b, with);
        if (__any_sync(~0u, near && !(f.x == x2 && f.b == b2))) {
          if (a.score == QMV_SCORE_SIGMOID)
            order_wide(a, few, n, lane, &id[0], &of[0]);
          else
            n = 34;
        }
      }
    }
  }
  if (n > 32) {
    float xb[2 * N];
    spill(xb);
    int id2[2] = {-1, -1};
    float of2[2] = {0.0f, 0.0f};
    if (n == 34 || !choose_each<float, N>(a, xb, left, lane, id2, of2)) choose_each<double, N>(a, xb, left, lane, id2, of2);
#pragma unroll
    for (int p = 0; p < 2; ++p) id[p] = id2[p], of[p] = of2[p];
  }
  float w[2];
#pragma unroll
  for (int p = 0; p < 2; ++p) {
    w[p] = 0.0f;
    if (lane + 32 * p < a.T && id[p] >= 0) {
      const float v = of[p], e = a.score == QMV_SCORE_SIGMOID ? expf(-fabsf(v)) : v == top ? 1.0f : exp_below(v, top);
      w[p] = a.score == QMV_SCORE_SIGMOID ? (v >= 0.0f ? 1.0f : e) / (1.0f + e) : e / whole;
    }
  }
  float f = a.scale;
  if (a.renorm) {
    const float sum = warp_total(w[0] + w[1]);
    if (sum >= 0x1p-20f) {
      f = a.scale / sum;
    } else {
      const float2 v = small_shares(a, id[0] >= 0 ? of[0] : none, id[1] >= 0 ? of[1] : none, top, a.score == QMV_SCORE_SIGMOID);
      w[0] = v.x, w[1] = v.y, f = 1.0f;
    }
  }
#pragma unroll
  for (int p = 0; p < 2; ++p)
    if (lane + 32 * p < a.T) {
      a.ids[m * a.T + lane + 32 * p] = id[p];
      a.w[m * a.T + lane + 32 * p] = w[p] * f;
    }
}

template <typename X, int N>
cudaError_t run(const RouteArgs& a, cudaStream_t s) {
  const dim3 grid((unsigned)(((int64_t)a.M + WARPS - 1) / WARPS));
  constexpr int EACH = 16 / sizeof(X);
  if constexpr (N % EACH == 0) {
    if (a.E % EACH == 0 && (uintptr_t)a.x % 16 == 0 && (a.M == 1 || a.ldx % EACH == 0))
      return launch_step(route_kernel<X, N, true>, grid, WARPS * 32, 0, s, 1, a);
  }
  return launch_step(route_kernel<X, N, false>, grid, WARPS * 32, 0, s, 1, a);
}

template <typename X>
cudaError_t typed(const RouteArgs& a, cudaStream_t s) {
  if (a.E <= 32) return run<X, 1>(a, s);
  if (a.E <= 64) return run<X, 2>(a, s);
  if (a.E <= 128) return run<X, 4>(a, s);
  if (a.E <= 256) return run<X, 8>(a, s);
  if (a.E <= 512) return run<X, 16>(a, s);
  return run<X, 32>(a, s);
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
