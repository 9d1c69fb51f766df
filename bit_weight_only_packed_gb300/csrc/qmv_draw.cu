// qmv_draw.cu -- one token a row of logits, from given random numbers (qmv_sample).
//
// A cluster of CTAs takes a row and keeps it in registers, so that HBM is read once; its CTAs
// tell each other what they know of their parts through their shared memories.  Weights
// are whole numbers, so neither the split nor the order of sums shows in the result.  What
// stays is always the first so many ids of an order (logit, the largest first, then id), so
// every cut is one place of it, a 64-bit number made of both (`Place`).
//   few    (a small top-k, or a row that is short anyway): the k largest come out of a few more
//          candidates, those that reach a bound which k logits reach for certain; one CTA sorts them
//          and finishes the row.  No weight of the other ids is formed.
//   many   (top-p alone, or a large k): the ids are counted by weight in bins of 2^(1/256), which
//          bound the sum above any bin to 0.3 %; in the bins that may hold the cut, about a thousand ids of
//          262144, one CTA sorts for the place.  Where ties make them more, a search by halves over
//          their logits finds it.
//   none   (no cut, or after it): every CTA sums what stays, and the one whose part the
//          threshold falls into finds the id.
#include <math_constants.h>

#include "qmv_token.cuh"

namespace qmv {
namespace {

typedef unsigned long long u64;
typedef u64 Place;               // ordered(logit) << 32 | ~id: larger comes first

constexpr int NT = 512, NW = NT / 32, MAX_C = 16;
constexpr int SUB_LOG = 8, SH = 23 - SUB_LOG, BINS = 43 << SUB_LOG;      // bins of weights from 2^-42 to 1
constexpr uint32_t E_MIN = (127u - 42u) << 23;                           // 2^-42, a weight of 1
constexpr int MAX_CAND = 2048, MAX_FEW = 1024;
constexpr int PER_BIN = (BINS + NT - 1) / NT;

// fp32 as a whole number of the same order; -inf (and NaN), which is never drawn, is 0.
__device__ __forceinline__ uint32_t ordered(float v) {
  if (!(v > -CUDART_INF_F)) return 0u;
  const uint32_t b = __float_as_uint(v + 0.0f);            // -0 counts as 0
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float unordered(uint32_t k) {
  return __uint_as_float(k & 0x80000000u ? k & 0x7fffffffu : ~k);
}
__device__ __forceinline__ Place place_of(float x, int id) { return (u64)ordered(x) << 32 | (uint32_t)~id; }

// 2^-z of qmv.h, its weight being floor(2^42 e).
__device__ __forceinline__ float exp_of(float x, float top, float c) {
  const float z = x == top ? 0.0f : fminf(__fmul_rn(__fsub_rn(top, x), c), 64.0f);
  const float t = z + 12582912.0f, f = (t - 12582912.0f) - z;            // n = z rounded, in t's last bits
  float p = 0.0013381302123889327f;
  p = fmaf(p, f, 0.00966636836528778f);
  p = fmaf(p, f, 0.055503811687231064f);
  p = fmaf(p, f, 0.2402234971523285f);
  p = fmaf(p, f, 0.6931471824645996f);
  p = fmaf(p, f, 1.0f);
  return __uint_as_float(__float_as_uint(p) - (__float_as_uint(t) << 23));
}
// floor(2^42 e) = hi 2^21 + lo, each cut off by the rounding of a sum with 2^23.
__device__ __forceinline__ void add_weight(float e, uint32_t& hi, uint32_t& lo) {
  const float t = __fmaf_rz(e, 2097152.0f, 8388608.0f), r = fmaf(e, 2097152.0f, 8388608.0f - t);
  hi += __float_as_uint(t) & 0x7fffffu;
  lo += __float_as_uint(__fmaf_rz(r, 2097152.0f, 8388608.0f)) & 0x7fffffu;
}
__device__ __forceinline__ u64 weight(float e) {
  uint32_t hi = 0, lo = 0;
  add_weight(e, hi, lo);
  return ((u64)hi << 21) + lo;
}

// floor(total * u / 2^31)
__device__ __forceinline__ u64 share(u64 total, u64 u) { return ((u * (total >> 32)) << 1) + ((u * (total & 0xffffffffull)) >> 31); }

__device__ __forceinline__ u64 warp_sum(u64 v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(~0u, v, o);
  return v;
}
// The sum of the lanes before this one.
__device__ __forceinline__ u64 warp_before(u64 v) {
  const int lane = threadIdx.x & 31;
  u64 run = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const u64 t = __shfl_up_sync(~0u, run, o);
    if (lane >= o) run += t;
  }
  return run - v;
}

__device__ __forceinline__ void st_cluster64(uint32_t a, u64 v) {
  asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(a), "l"(v) : "memory");
}
__device__ __forceinline__ u64 ld_cluster64(uint32_t a) {
  u64 v;
  asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ uint4 ld_cluster128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared::cluster.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
  return v;
}

struct Shared {
  u64 red[2][NW];                // sums of warps
  u64 told[2][MAX_C][3];         // what the CTAs of the cluster tell each other
  u64 cut;
  uint32_t sub[256];
  uint32_t top, bound, n;
  int i0, i1, last;
};

// A CTA's sum of v, in all threads, and what the threads before this one have of it.
__device__ __forceinline__ u64 block_sum(Shared& S, u64 v, u64* before) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const u64 mine = warp_before(v);
  __syncthreads();
  if (lane == 31) S.red[0][w] = mine + v;
  __syncthreads();
  const u64 p = lane < NW ? S.red[0][lane] : 0, b = warp_before(p);
  *before = __shfl_sync(~0u, b, w) + mine;
  return __shfl_sync(~0u, b + p, NW - 1);
}

// The first n of `list` (up to MAX_CAND) in falling order; n2, a power of two from n on, is filled up with 0.
__device__ void sort_down(u64* list, int n, int n2) {
  for (int i = n + threadIdx.x; i < n2; i += NT) list[i] = 0;
  for (int size = 2; size <= n2; size *= 2)
    for (int step = size / 2; step; step /= 2) {
      __syncthreads();
      for (int i = threadIdx.x; i < n2 / 2; i += NT) {
        const int a = 2 * i - (i & (step - 1)), b = a + step;
        const u64 u = list[a], v = list[b];
        if ((u < v) == ((a & size) == 0)) list[a] = v, list[b] = u;
      }
    }
  __syncthreads();
}

// The edges of bin b in whole weights: those in it are at least edge(b) and at most edge(b + 1).
__device__ __forceinline__ u64 edge(int b) {
  const int o = b >> SUB_LOG;
  const u64 v = (u64)((1 << SUB_LOG) + (b & ((1 << SUB_LOG) - 1))) << (42 - SUB_LOG);
  return o <= 42 ? v >> (42 - o) : v << (o - 42);
}

// EPT > 0: a thread's part of the row stays in registers, EPT elements in fours that are
// aligned in memory wherever the row begins; EPT == 0: rows of any length, `fours` a thread, read
// again for each pass.  In either form a warp has neighbouring ids, 128 at a time.
template <typename X, int EPT>
__global__ void __launch_bounds__(NT, 2) draw_kernel(DrawArgs a, int C, int fours) {
  extern __shared__ __align__(16) uint32_t dyn[];
  uint32_t *hist = dyn, *all_hist = dyn + BINS;
  u64 *list = reinterpret_cast<u64*>(hist), *cand = list + MAX_CAND;     // once hist has been added up
  __shared__ Shared S;
  constexpr int R = EPT ? EPT / 4 : 1;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = blockIdx.x % C, row = blockIdx.x / C, V = a.V;
  if (tid == 0) S.n = 0, S.top = 0;
  __syncthreads();
  if (C > 1) cluster_arrive();
  const X* x = (const X*)a.x + (int64_t)row * a.ldx;
  const int shift = (int)((uintptr_t)x / sizeof(X) % 4), rows4 = EPT ? R : fours;
  const int first = ((rank * NW + warp) * rows4) * 128 + lane * 4 - shift;   // the first four's first id
  pdl_begin();
  // four ids, -inf where there are none
  const auto fetch = [&](int j, float (&v)[4]) {
    const int id = first + j * 128;
    if (id >= 0 && id + 4 <= V) {
      X h[4];
      if (sizeof(X) == 4) {
        const float4 w = *reinterpret_cast<const float4*>(x + id);
        memcpy(h, &w, sizeof(h));
      } else {
        const uint2 w = *reinterpret_cast<const uint2*>(x + id);
        memcpy(h, &w, sizeof(h));
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) v[k] = to_f<X>(h[k]);
    } else {
#pragma unroll
      for (int k = 0; k < 4; ++k) v[k] = (unsigned)(id + k) < (unsigned)V ? to_f<X>(x[id + k]) : -CUDART_INF_F;
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) v[k] = isnan(v[k]) ? -CUDART_INF_F : v[k];
  };
  float v[R][4];                 // logits, later 2^-z
  if (EPT) {
#pragma unroll
    for (int j = 0; j < R; ++j) fetch(j, v[j]);
  }
  // f(j, the four logits), f(j, the four of v): the same while v holds logits
  const auto each_logit = [&](auto f) {
    if (EPT) {
#pragma unroll
      for (int j = 0; j < R; ++j) f(j, v[j]);
    } else {
      for (int j = 0; j < fours; ++j) {
        float w[4];
        fetch(j, w);
        f(j, w);
      }
    }
  };
  const float t = a.t ? a.t[row] : a.t0, tp = a.p ? a.p[row] : a.p0, mp = a.m ? a.m[row] : a.m0;
  const int k = a.k ? a.k[row] : a.k0;
  const bool greedy = !(t > 0.0f), k_on = k > 0 && k < V, p_on = tp < 1.0f;
  const u64 P = (u64)(fmaxf(p_on ? tp : 0.0f, 0.0f) * 2147483648.0f);
  const u64 U = (u64)fminf(fmaxf(a.u[row], 0.0f) * 2147483648.0f, 2147483520.0f);
  const u64 least = (u64)((double)fminf(fmaxf(mp, 0.0f), 1.0f) * 4398046511104.0);
  const float c = 1.4426950408889634f / fmaxf(t, 0x1p-100f);

  // Every CTA's three numbers to all of the cluster.
  int turn = 0;
  const auto meet = [&]() {
    __syncwarp();
    if (C > 1) {
      cluster_arrive();
      cluster_wait();
    } else {
      __syncthreads();
    }
  };
  const auto tell = [&](u64 n0, u64 n1, u64 n2) -> const u64(*)[3] {
    turn ^= 1;
    if (tid < C) {
      const uint32_t to = cluster_addr(&S.told[turn][rank][0], tid);
      st_cluster64(to, n0), st_cluster64(to + 8, n1), st_cluster64(to + 16, n2);
    }
    meet();
    return S.told[turn];
  };

  // The largest logit; and where few will stay, a bound that k of them reach: each CTA's is reached
  // by its share of k, the least of them by all.
  const int per = (k + C - 1) / C;
  const bool short_row = C == 1 && V <= MAX_CAND;
  bool few = !greedy && (short_row || (k_on && k <= MAX_FEW && per <= 128));
  float most = -CUDART_INF_F;
  each_logit([&](int, const float(&w)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) most = fmaxf(most, w[i]);
  });
  const uint32_t key = ordered(most), warp_top = __reduce_max_sync(~0u, key);
  if (lane == 0) atomicMax(&S.top, warp_top);
  uint32_t bound = 0;
  if (few && !short_row) {
    // the largest of every warp, eight lanes or two: twice as many as are wanted, or more
    const int lanes = per <= 8 ? 32 : per <= 32 ? 8 : 2, n = NT / lanes;
    uint32_t m = key;
    for (int o = 1; o < lanes; o <<= 1) m = max(m, __shfl_xor_sync(~0u, m, o));
    if (lane % lanes == 0) S.sub[tid / lanes] = m;
    __syncthreads();
    if (tid < n) {
      const uint32_t own = S.sub[tid];
      int above = 0;
      for (int i = 0; i < n; ++i) above += S.sub[i] > own || (S.sub[i] == own && i < tid);
      if (above == per - 1) S.bound = own;
    }
    __syncthreads();
    bound = S.bound;
  } else {
    __syncthreads();
  }
  if (C > 1) cluster_wait();               // all have begun
  uint32_t top = 0;
  {
    const auto told = tell(S.top, bound, 0);
    uint32_t b = lane < C ? (uint32_t)told[lane][1] : ~0u;
    top = __reduce_max_sync(~0u, lane < C ? (uint32_t)told[lane][0] : 0u);
    bound = __reduce_min_sync(~0u, b);
  }
  if (top == 0) {                          // nothing can be drawn
    if (rank == 0 && tid == 0) a.tokens[row] = -1;
    return;
  }
  const float largest = unordered(top);
  if (greedy) {
    int at = V;
    each_logit([&](int j, const float(&w)[4]) {
#pragma unroll
      for (int i = 3; i >= 0; --i)
        if (w[i] == largest) at = min(at, first + j * 128 + i);
    });
    at = __reduce_min_sync(~0u, at);
    if (lane == 0) S.red[0][warp] = at;
    __syncthreads();
    u64 b = V;
    for (int i = 0; i < NW; ++i) b = min(b, S.red[0][i]);
    const auto told = tell(b, 0, 0);
    for (int i = 0; i < C; ++i) b = min(b, told[i][0]);
    if (rank == 0 && tid == 0) a.tokens[row] = (int)b;
    return;
  }

  // The CTAs' lists, one after another, to the first CTA's `cand`; they hold n in all.
  const auto gather = [&](const u64(*told)[3]) {
    int at = 0;
    for (int r = 0; r < C; ++r) {
      const int m = (int)told[r][2];
      const uint32_t from = cluster_addr(list, r);
      for (int i = tid; i < m; i += NT) cand[at + i] = ld_cluster64(from + i * 8);
      at += m;
    }
    return at;
  };
  const auto listed = [&](const u64(*told)[3], bool* fits) {
    int n = 0;
    bool ok = true;
    for (int r = 0; r < C; ++r) ok = ok && told[r][2] <= MAX_CAND, n += (int)min(told[r][2], (u64)MAX_CAND);
    *fits = ok && n <= MAX_CAND;
    return n;
  };
  const auto note = [&](Place p) {
    const uint32_t at = atomicAdd(&S.n, 1u);
    if (at < MAX_CAND) list[at] = p;
  };

  if (few) {
    each_logit([&](int j, const float(&w)[4]) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t o = ordered(w[i]);
        if (o && o >= bound) note((u64)o << 32 | (uint32_t)~(first + j * 128 + i));
      }
    });
    __syncthreads();
    const auto told = tell(0, 0, S.n);
    bool fits;
    const int n = listed(told, &fits);
    if (fits) {
      if (rank == 0) {
        gather(told);
        int n2 = 32;
        while (n2 < n) n2 *= 2;
        __syncthreads();
        sort_down(cand, n, n2);
        // a thread takes four neighbours of the order
        u64 w[4], sum = 0, before;
        const int k1 = k_on ? min(k, n) : n;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int at = tid * 4 + i;
          w[i] = at < k1 ? weight(exp_of(unordered((uint32_t)(cand[at] >> 32)), largest, c)) : 0;
          sum += w[i];
        }
        const u64 need = p_on ? share(block_sum(S, sum, &before), P) : ~0ull;
        if (!p_on) before = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int at = tid * 4 + i;
          const u64 p = at < n2 ? cand[at] : 0;
          if (at < n2)                     // in the order of ids, with what is needed for the weight
            cand[at] = at < k1 && (before < need || at == 0) && w[i] >= least ? (p << 32 | p >> 32) : 0;
          before += w[i];
        }
        __syncthreads();
        sort_down(cand, n2, n2);           // ~id falls as the id rises
        sum = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int at = tid * 4 + i;
          const u64 p = at < n2 ? cand[at] : 0;
          w[i] = p ? weight(exp_of(unordered((uint32_t)p), largest, c)) : 0;
          sum += w[i];
        }
        const u64 total = block_sum(S, sum, &before), at = share(total, U);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if (before <= at && at < before + w[i]) a.tokens[row] = (int)~(uint32_t)(cand[tid * 4 + i] >> 32);
          before += w[i];
        }
      }
      if (C > 1) meet();                   // the others' lists have been read
      return;
    }
    meet();
    if (tid == 0) S.n = 0;
  }

  // Weights in place of logits.
  const bool cutting = k_on || p_on;
  if (EPT) {
#pragma unroll
    for (int j = 0; j < R; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) v[j][i] = exp_of(v[j][i], largest, c);
  }
  const auto each = [&](auto f) {
    if (EPT) {
#pragma unroll
      for (int j = 0; j < R; ++j) f(j, v[j]);
    } else {
      for (int j = 0; j < fours; ++j) {
        float w[4];
        fetch(j, w);
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = exp_of(w[i], largest, c);
        f(j, w);
      }
    }
  };
  const auto logit = [&](int id) { return to_f<X>(x[id]); };

  // What stays so far: weights from `sure` on, and those from `maybe` on whose place is `cut` or before.
  uint32_t sure = 0, maybe = 0;
  Place cut = 0;
  const auto stays = [&](float e, int id) {
    const uint32_t b = __float_as_uint(e);
    return b >= sure || (b >= maybe && place_of(logit(id), id) >= cut);
  };
  const auto sum_of = [&](u64 least) {
    u64 sum = 0;
    each([&](int j, const float(&e)[4]) {
      uint32_t hi = 0, lo = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (stays(e[i], first + j * 128 + i)) {
          if (least == 0) {
            add_weight(e[i], hi, lo);
          } else {
            const u64 w = weight(e[i]);
            sum += w >= least ? w : 0;
          }
        }
      sum += ((u64)hi << 21) + lo;
    });
    return sum;
  };

  if (cutting) {
    sure = maybe = E_MIN;                  // the others weigh nothing
    for (int i = tid; i < BINS / 4; i += NT) reinterpret_cast<uint4*>(hist)[i] = make_uint4(0, 0, 0, 0);
    __syncthreads();
    u64 sum = 0, before;
    each([&](int, const float(&e)[4]) {
      uint32_t hi = 0, lo = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t b = __float_as_uint(e[i]);
        if (b >= E_MIN) {
          atomicAdd(&hist[(b - E_MIN) >> SH], 1u);
          add_weight(e[i], hi, lo);
        }
      }
      sum += ((u64)hi << 21) + lo;
    });
    sum = block_sum(S, sum, &before);
    u64 whole = 0;
    {
      const auto told = tell(sum, 0, 0);   // and hist is complete in all CTAs
      for (int r = 0; r < C; ++r) whole += told[r][0];
    }
    // each CTA adds up its share of the bins and tells the others
    const int q = BINS / 4 / C;            // fours of bins
    static_assert(BINS / 4 % MAX_C == 0, "shares are whole");
    for (int i = tid; i < q; i += NT) {
      uint4 s = make_uint4(0, 0, 0, 0);
      for (int r = 0; r < C; ++r) {
        const uint4 o = ld_cluster128(cluster_addr(reinterpret_cast<uint4*>(hist) + rank * q + i, (rank + r) % C));
        s.x += o.x, s.y += o.y, s.z += o.z, s.w += o.w;
      }
      for (int r = 0; r < C; ++r) {
        const uint32_t to = cluster_addr(reinterpret_cast<uint4*>(all_hist) + rank * q + i, (rank + r) % C);
        asm volatile("st.shared::cluster.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(to), "r"(s.x), "r"(s.y), "r"(s.z), "r"(s.w) : "memory");
      }
    }
    meet();
    int k0 = 0, k1 = BINS - 1;             // bins, from the largest weights on, in which top-k's cut may lie
    for (int stage = 0; stage < 2; ++stage) {
      // stage 0 counts ids up to k, stage 1 weights up to top_p of what is left
      if (stage == 0 ? !k_on : !p_on) continue;
      u64 need = (u64)k;
      if (stage == 1) {
        if (cut) {
          u64 b;
          const u64 s = block_sum(S, sum_of(0), &b);
          const auto told = tell(s, 0, 0);
          whole = 0;
          for (int r = 0; r < C; ++r) whole += told[r][0];
        }
        need = max(share(whole, P), (u64)1);
      }
      // the bins that may hold the cut: the sum up to each lies between `low` and `high`
      u64 low = 0, high = 0;
      const auto bin = [&](int i, u64* lo, u64* hi) {
        const int b = BINS - 1 - i;
        const u64 n = i < BINS && (!cut || i <= k1) ? all_hist[b] : 0;
        *hi = stage == 0 ? n : n * (b == 42 << SUB_LOG ? edge(b) : edge(b + 1));
        *lo = cut && i >= k0 ? 0 : stage == 0 ? n : n * edge(b);
      };
#pragma unroll 1
      for (int i = tid * PER_BIN; i < (tid + 1) * PER_BIN; ++i) {
        u64 lo, hi;
        bin(i, &lo, &hi);
        low += lo, high += hi;
      }
      if (tid == 0) S.i0 = BINS - 1, S.i1 = 0, S.n = 0;
      block_sum(S, low, &low);
      const u64 most_of_all = block_sum(S, high, &high);
      if (stage == 0 && most_of_all <= need) continue;       // what weighs anything all stays
#pragma unroll 1
      for (int i = tid * PER_BIN; i < min(BINS, (tid + 1) * PER_BIN); ++i) {
        u64 lo, hi;
        bin(i, &lo, &hi);
        high += hi;
        if (high >= need && high - hi < need) atomicMin(&S.i0, i);
        if (low < need && hi) atomicMax(&S.i1, i);
        low += lo;
      }
      __syncthreads();
      // one more on either side, since the order within 2^-20 of a weight is that of logits alone
      int i0 = max(0, S.i0 - 1), i1 = min(BINS - 1, S.i1 + 1);
      if (cut) i0 = min(i0, k0), i1 = min(i1, k1);
      const uint32_t was_maybe = maybe;
      const Place was_cut = cut;
      const uint32_t above = E_MIN + ((uint32_t)(BINS - i0) << SH), from = E_MIN + ((uint32_t)(BINS - 1 - i1) << SH);
      // what lies above them, exactly, and their ids
      const auto in_band = [&](uint32_t b) { return b < above && b >= from; };
      u64 over = 0;
      uint32_t count = 0;
      each([&](int j, const float(&e)[4]) {
        uint32_t hi = 0, lo = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t b = __float_as_uint(e[i]);
          if (b >= above) {
            ++count;
            add_weight(e[i], hi, lo);
          } else if (b >= from && b >= was_maybe) {
            const int id = first + j * 128 + i;
            const Place p = place_of(logit(id), id);
            if (p >= was_cut) note(p);
          }
        }
        over += ((u64)hi << 21) + lo;
      });
      over = block_sum(S, stage == 0 ? (u64)count : over, &before);
      const auto told = tell(over, 0, S.n);
      over = 0;
      for (int r = 0; r < C; ++r) over += told[r][0];
      bool fits;
      const int n = listed(told, &fits);
      if (fits) {
        if (rank == 0) {
          gather(told);
          int n2 = 32;
          while (n2 < n) n2 *= 2;
          if (tid == 0) S.last = 0;
          __syncthreads();
          sort_down(cand, n, n2);
          u64 w[4], s = 0, run;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int at = tid * 4 + i;
            w[i] = at >= n ? 0 : stage == 0 ? 1 : weight(exp_of(unordered((uint32_t)(cand[at] >> 32)), largest, c));
            s += w[i];
          }
          block_sum(S, s, &run);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int at = tid * 4 + i;
            if (at < n && over + run < need) atomicMax(&S.last, at);
            run += w[i];
          }
          __syncthreads();
          if (tid < C) st_cluster64(cluster_addr(&S.cut, tid), cand[S.last]);
        }
        meet();
      } else {
        // more than fit, as ties make them: halves of their logits, each time between the
        // smallest and the largest that are left
        uint32_t k_lo = ~0u, k_hi = 0;
        const auto band = [&](auto f) {
          each([&](int j, const float(&e)[4]) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const uint32_t b = __float_as_uint(e[i]);
              if (!in_band(b) || b < was_maybe) continue;
              const int id = first + j * 128 + i;
              const Place p = place_of(logit(id), id);
              if (p >= was_cut) f((uint32_t)(p >> 32), e[i], j, i);
            }
          });
        };
        const auto least_of = [&](uint32_t v) {
          v = __reduce_min_sync(~0u, v);
          __syncthreads();
          if (lane == 0) S.sub[warp] = v;
          __syncthreads();
          return __reduce_min_sync(~0u, S.sub[lane % NW]);
        };
        const auto agree = [&](u64 sum, uint32_t lo, uint32_t hi, u64* all, uint32_t* all_lo, uint32_t* all_hi) {
          u64 b;
          sum = block_sum(S, sum, &b);
          lo = least_of(lo);
          hi = ~least_of(~hi);
          const auto told = tell(sum, lo, hi);
          *all = 0;
          *all_lo = ~0u, *all_hi = 0;
          for (int r = 0; r < C; ++r) {
            *all += told[r][0];
            *all_lo = min(*all_lo, (uint32_t)told[r][1]);
            *all_hi = max(*all_hi, (uint32_t)told[r][2]);
          }
        };
        u64 s;
        band([&](uint32_t o, float, int, int) { k_lo = min(k_lo, o), k_hi = max(k_hi, o); });
        agree(0, k_lo, k_hi, &s, &k_lo, &k_hi);
        while (k_lo < k_hi) {
          const uint32_t mid = k_lo + (k_hi - k_lo) / 2;
          u64 up = 0;
          uint32_t up_lo = ~0u, down_hi = 0;
          band([&](uint32_t o, float e, int, int) {
            if (o > mid && o <= k_hi) up += stage == 0 ? 1 : weight(e), up_lo = min(up_lo, o);
            if (o <= mid && o >= k_lo) down_hi = max(down_hi, o);
          });
          agree(up, up_lo, down_hi, &s, &up_lo, &down_hi);
          if (over + s >= need)
            k_lo = up_lo;
          else
            over += s, k_hi = down_hi;
        }
        // equal logits: the first so many by id
        const u64 one = stage == 0 ? 1 : weight(exp_of(unordered(k_lo), largest, c));
        u64 wanted = (need - over + one - 1) / one, mine = 0;
        band([&](uint32_t o, float, int, int) { mine += o == k_lo; });
        const u64 warp_ties = warp_sum(mine);
        __syncthreads();
        if (lane == 0) S.red[1][warp] = warp_ties;
        const u64 ties = block_sum(S, mine, &before);
        const auto told = tell(ties, 0, 0);
        u64 run = 0;
        for (int r = 0; r < rank; ++r) run += told[r][0];
        for (int w = 0; w < warp; ++w) run += S.red[1][w];
        if (run < wanted && wanted <= run + warp_ties) {
          // the warp with the last of them, 128 ids at a time
          each([&](int j, const float(&e)[4]) {
            u64 n = 0;
            bool tie[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const uint32_t b = __float_as_uint(e[i]);
              const int id = first + j * 128 + i;
              tie[i] = in_band(b) && b >= was_maybe && ordered(logit(id)) == k_lo && place_of(logit(id), id) >= was_cut;
              n += tie[i];
            }
            u64 at = run + warp_before(n);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              at += tie[i];
              if (tie[i] && at == wanted)
                for (int r = 0; r < C; ++r) st_cluster64(cluster_addr(&S.cut, r), (u64)k_lo << 32 | (uint32_t)~(first + j * 128 + i));
            }
            run += warp_sum(n);
          });
        }
        meet();
      }
      cut = S.cut;
      sure = above, maybe = from;
      k0 = i0, k1 = i1;
      meet();                              // before anything here is written again
    }
  }

  // What stays, all of it; then the id at the threshold.
  const u64 own = sum_of(least), warp_own = warp_sum(own);
  u64 before;
  __syncthreads();
  if (lane == 0) S.red[1][warp] = warp_own;
  const u64 cta = block_sum(S, own, &before);
  u64 total = 0, run = 0;
  {
    const auto told = tell(cta, 0, 0);
    for (int r = 0; r < C; ++r) {
      if (r < rank) run += told[r][0];
      total += told[r][0];
    }
  }
  const u64 at = share(total, U);
  for (int w = 0; w < warp; ++w) run += S.red[1][w];
  if (run > at || at >= run + warp_own) return;
  bool found = false;
  each([&](int j, const float(&e)[4]) {
    if (found) return;
    u64 w[4], n = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      w[i] = stays(e[i], first + j * 128 + i) ? weight(e[i]) : 0;
      w[i] = w[i] >= least ? w[i] : 0;
      n += w[i];
    }
    const u64 all = warp_sum(n);
    if (run + all > at) {
      u64 here = run + warp_before(n);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (here <= at && at < here + w[i]) a.tokens[row] = first + j * 128 + i;
        here += w[i];
      }
      found = true;
    }
    run += all;
  });
}

template <typename X, int EPT>
cudaError_t run(const DrawArgs& a, int C, int fours, cudaStream_t s) {
  static thread_local KernCache cache;
  static thread_local int allowed = -1;
  constexpr int SMEM = 2 * BINS * 4;
  cudaError_t e = prep_kernel(draw_kernel<X, EPT>, cache, NT, SMEM, nullptr);
  if (e == cudaSuccess && C > 8 && allowed != cache.dev) {  // clusters of 16 are opt-in, a function and device
    e = cudaFuncSetAttribute(draw_kernel<X, EPT>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    allowed = cache.dev;
  }
  if (e != cudaSuccess) return e;
  return launch_step(draw_kernel<X, EPT>, dim3((unsigned)a.rows * C), NT, SMEM, s, C, a, C, fours);
}

// CTAs a row: as few as hold it, or more where rows are few.
template <typename X>
cudaError_t typed(const DrawArgs& a, cudaStream_t s) {
  const int64_t elements = (int64_t)a.V + 3;               // wherever the row begins
  const int slots = 2 * dev_info().sms;
  int C = 1;
  while (C < MAX_C && (int64_t)C * NT * 32 < elements) C *= 2;
  if ((int64_t)C * NT * 32 < elements) return run<X, 0>(a, C, (int)((elements + (int64_t)C * NT * 4 - 1) / ((int64_t)C * NT * 4)), s);
  int C8 = C;
  while (C8 < MAX_C && (int64_t)C8 * NT * 8 < elements) C8 *= 2;
  if ((int64_t)C8 * NT * 8 >= elements && (int64_t)C8 * a.rows <= slots) return run<X, 8>(a, C8, 2, s);
  return run<X, 32>(a, C, 8, s);
}

}  // namespace

cudaError_t launch_draw(const DrawArgs& a, cudaStream_t s) {
  switch (a.dtype) {
    case QMV_F32: return typed<float>(a, s);
    case QMV_F16: return typed<__half>(a, s);
    default: return typed<__nv_bfloat16>(a, s);
  }
}

}  // namespace qmv
