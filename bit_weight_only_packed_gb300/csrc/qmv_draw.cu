// qmv_draw.cu -- one token a row of logits, from given random numbers (qmv_sample).
//
// A cluster of CTAs takes a row; they tell each other what they know of their parts through their shared
// memories.  Weights are whole numbers, so neither the split nor the order of sums shows in the result.  What
// stays is always the first so many ids of an order (logit, the largest first, then id), so every cut is one
// place of it, a 64-bit number made of both (`Place`).
//   few    (a small top-k, or a row that is short anyway): the k largest come out of a few more candidates,
//          those that reach a bound which k logits reach for certain; one CTA sorts them and finishes the
//          row.  No weight of the other ids is formed.
//   many   (top-p alone, or a large k): the ids are counted by weight in bins, 256 even steps an octave, whose edges
//          differ by 1/256 to 1/512 of a weight and so bound the sum above any bin (weights below 2^8 units, whose
//          bins are narrower than a unit, only from above); in the bins that may hold the cut, about a thousand ids of
//          262144, one CTA sorts for the place.  Where ties make them more, a search by halves over their logits finds it.
//   none   (no cut, or after it): every CTA sums what stays, and the one whose part the threshold falls into
//          finds the id.
//
// A row of 262144 with top-k 64 and top-p 0.95 takes 13 us, a latency: the row is read twice, the cluster meets
// three times, 1.5 us are the sorts.  128 rows of them with top-p 0.9 alone take 189 us (134 MB, 20 us from HBM):
// 28 the largest logits, 50 each of the two passes that form the weights, by their instructions (some 40 a weight
// and its bin), the rest the meetings and sorts of CTAs that run two to a multiprocessor.
#include <math_constants.h>

#include <type_traits>

#include "qmv_token.cuh"

namespace qmv {
namespace {

typedef unsigned long long u64;
typedef u64 Place;               // ordered(logit) << 32 | ~id: larger comes first

constexpr int NT = 512, NW = NT / 32, MAX_C = 16;
constexpr int SUB_LOG = 8, SH = 23 - SUB_LOG, BINS = 43 << SUB_LOG;      // bins of weights from 2^-42 to 1
constexpr uint32_t E_MIN = (127u - 42u) << 23;                           // 2^-42, a weight of 1
constexpr int MAX_CAND = 2048, MAX_FEW = 1024;
constexpr int OCTAVES = 43;

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

// z of qmv.h, and e = 2^-z, the weight being floor(2^42 e).  top is finite; NaN and -inf have z = 64,
// whatever c is, and weigh nothing.
__device__ __forceinline__ float z_of(float x, float top, float c) { return fminf(__fmul_rn(__fsub_rn(top, x), c), 64.0f); }
__device__ __forceinline__ float exp_of(float x, float top, float c) {
  const float z = z_of(x, top, c);
  const float t = z + 12582912.0f, f = (t - 12582912.0f) - z;            // n = z rounded, in t's last bits
  float p = 0.0013381302123889327f;
  p = fmaf(p, f, 0.00966636836528778f);
  p = fmaf(p, f, 0.055503811687231064f);
  p = fmaf(p, f, 0.2402234971523285f);
  p = fmaf(p, f, 0.6931471824645996f);
  p = fmaf(p, f, 1.0f);
  return __uint_as_float(__float_as_uint(p) - (__float_as_uint(t) << 23));
}
// Sums of weights: floor(2^42 e) = hi 2^21 + lo, each cut off by the rounding of a sum with 2^23, whose
// other bits come off at the end.
struct Weights {
  uint32_t hi = 0, lo = 0;
  __device__ __forceinline__ void add(float e) {
    const float t = __fmaf_rz(e, 2097152.0f, 8388608.0f), r = fmaf(e, 2097152.0f, 8388608.0f - t);
    hi += __float_as_uint(t);
    lo += __float_as_uint(__fmaf_rz(r, 2097152.0f, 8388608.0f));
  }
  // of so many, at most 1024
  __device__ __forceinline__ u64 sum(int n) const {
    return ((u64)(hi - n * 0x4B000000u) << 21) + (lo - n * 0x4B000000u);
  }
};
__device__ __forceinline__ u64 weight(float e) {
  Weights w;
  w.add(e);
  return w.sum(1);
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
__device__ __forceinline__ void st_cluster32(uint32_t a, uint32_t v) {
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(a), "r"(v) : "memory");
}
__device__ __forceinline__ u64 ld_cluster64(uint32_t a) {
  u64 v;
  asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(a) : "memory");
  return v;
}
struct Shared {
  u64 red[2][NW];                // sums of warps
  u64 told[2][MAX_C][3];         // what the CTAs of the cluster tell each other
  u64 octaves[MAX_C][OCTAVES];   // and of the octaves of weights: ids, and sums of their bins
  uint32_t ends[2 << SUB_LOG];   // the bins of the two octaves that hold a range's ends
  uint32_t start[NT];            // where buckets begin; the threads' largest logits
  u64 cut;
  uint32_t sub[NW];
  uint32_t top, bound, n;
  int o[2], i[2];                // the octaves, and the bins that end the range
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

// The least of a CTA's values, in all threads.
__device__ __forceinline__ uint32_t block_min(Shared& S, uint32_t v) {
  v = __reduce_min_sync(~0u, v);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) S.sub[threadIdx.x >> 5] = v;
  __syncthreads();
  return __reduce_min_sync(~0u, S.sub[threadIdx.x % NW]);
}

// n keys that all differ, up to four a thread, in falling order to `sorted`: into NT buckets by a
// number that falls as the key rises, within one by comparing all of its keys.  (2048
// keys: 1.5 us, against 18 us for a sorting network.)
__device__ __noinline__ void sort_down(Shared& S, const u64 (&key)[4], const float (&number)[4], int n, u64* spread, u64* sorted) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  uint32_t least = 0x7f800000u, most = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (tid + i * NT < n) least = min(least, __float_as_uint(number[i])), most = max(most, __float_as_uint(number[i]));
  S.start[tid] = 0;
  const float from = __uint_as_float(block_min(S, least)), range = __uint_as_float(~block_min(S, ~most)) - from;
  const float scale = range > 0.0f ? fminf((NT - 1) / range, 1e30f) : 0.0f;
  int bucket[4], slot[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (tid + i * NT < n) {
      bucket[i] = min(NT - 1, (int)((number[i] - from) * scale));
      slot[i] = atomicAdd(&S.start[bucket[i]], 1u);
    }
  __syncthreads();
  const int count = S.start[tid];
  int run = count;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int t = __shfl_up_sync(~0u, run, o);
    if (lane >= o) run += t;
  }
  if (lane == 31) S.sub[warp] = run;
  __syncthreads();
  const int w = lane < warp ? S.sub[lane] : 0;             // at most 16 warps
  S.start[tid] = run - count + __reduce_add_sync(~0u, w);
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (tid + i * NT < n) spread[S.start[bucket[i]] + slot[i]] = key[i];
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (tid + i * NT < n) {
      const int at = S.start[bucket[i]], end = bucket[i] + 1 < NT ? S.start[bucket[i] + 1] : n;
      int to = at;
      for (int j = at; j < end; ++j) to += spread[j] > key[i];
      sorted[to] = key[i];
    }
  __syncthreads();
}

// C CTAs a row, each with an even share: a warp has neighbouring ids, 128 * fours, a thread fours of
// them, aligned in memory wherever the row begins.  Every pass reads them again, from L2.  (Kept on the
// streaming multiprocessor, in shared memory or in registers, 128 rows of 262144 need clusters of
// sixteen with 64 KB a CTA, so that eight rows are worked on at once, and each takes its 14 meetings:
// 557 us.)
template <typename X>
__global__ void __launch_bounds__(NT, 2) draw_kernel(DrawArgs a, int C, int fours) {
  extern __shared__ __align__(16) uint32_t dyn[];
  uint32_t* hist = dyn;
  u64 *list = reinterpret_cast<u64*>(dyn), *cand = list + MAX_CAND;      // once hist has been read
  static_assert(2 * MAX_CAND * 8 <= BINS * 4, "they fit there");
  __shared__ Shared S;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = blockIdx.x % C, row = blockIdx.x / C, V = a.V;
  if (tid == 0) S.n = 0, S.top = 0;
  __syncthreads();
  if (C > 1) cluster_arrive();
  const X* x = (const X*)a.x + (int64_t)row * a.ldx;
  const int shift = (int)((uintptr_t)x / sizeof(X) % 4);
  const int first = ((rank * NW + warp) * fours) * 128 + lane * 4 - shift;   // the first four's first id
  pdl_begin();
  bool infinite = false;         // +inf is among them: from where that is known, 0 in its place and -inf in all others'
  typedef typename std::conditional<sizeof(X) == 4, uint4, uint2>::type Raw;
  // the first and the last four that lie whole in the row, if any
  const int low = (4 - shift) & 3, high = V - 4 >= low ? low + (V - 4 - low) / 4 * 4 : -1;
  // f(j, four logits, -inf where there are none) for all of a thread's fours; AHEAD of them are on their
  // way, as they are stored, while one is worked on.  Each load is made, from a place inside the row: one
  // under a condition waits for those before it (the largest logits of 128 rows of 262144, a CTA
  // each: 65 us so, whatever AHEAD is, against 28).  Fours that stick out of the row are read
  // an element at a time when their turn comes.
  const auto each = [&](auto ahead, auto f) {
    constexpr int AHEAD = decltype(ahead)::value;
    const auto load = [&](int j) { return *reinterpret_cast<const Raw*>(x + min(max(first + j * 128, low), high)); };
    Raw raw[AHEAD];
    if (high >= 0) {
#pragma unroll
      for (int q = 0; q < AHEAD; ++q) raw[q] = load(q);
    }
#pragma unroll 1
    for (int j = 0; j < fours; j += AHEAD) {
#pragma unroll
      for (int q = 0; q < AHEAD; ++q) {
        const int id = first + (j + q) * 128;
        float v[4];
        X h[4];
        memcpy(h, &raw[q], sizeof(Raw));
        if (high >= 0) raw[q] = load(j + q + AHEAD);
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = to_f<X>(h[i]);
        if (id < low || id > high) {
#pragma unroll
          for (int i = 0; i < 4; ++i) v[i] = (unsigned)(id + i) < (unsigned)V ? to_f<X>(x[id + i]) : -CUDART_INF_F;
        }
        if (infinite) {
#pragma unroll
          for (int i = 0; i < 4; ++i) v[i] = v[i] == CUDART_INF_F ? 0.0f : -CUDART_INF_F;
        }
        if (j + q < fours) f(j + q, v);
      }
    }
  };
  constexpr std::integral_constant<int, 4> ahead;          // where little is done with them
  constexpr std::integral_constant<int, 2> two_ahead;
  constexpr std::integral_constant<int, 1> one_by_one;
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
  // by its share of k, as it has of the row, the least of them by all.
  const bool short_row = C == 1 && V <= MAX_CAND;
  const int part = NW * fours * 128, here = max(0, min(part, V + shift - rank * part));
  const int most_per = (int)(((int64_t)k * min(part, V) + V - 1) / V);   // the same for all CTAs
  const bool few = !greedy && (short_row || (k_on && k <= MAX_FEW && most_per <= NT / 2));
  const int per = few ? (int)(((int64_t)k * min(here, V) + V - 1) / V) : 0;
  float most = -CUDART_INF_F;
  each(ahead, [&](int, const float(&w)[4]) { most = fmaxf(fmaxf(most, fmaxf(w[0], w[1])), fmaxf(w[2], w[3])); });
  const uint32_t key = ordered(most), warp_top = __reduce_max_sync(~0u, key);
  if (lane == 0) atomicMax(&S.top, warp_top);
  uint32_t bound = 0;
  if (few && !short_row) {
    if (most_per > 32) {
      // the largest of every thread, of which twice as many as are wanted: the bits of the last wanted one
#pragma unroll 1
      for (uint32_t bit = 1u << 31; bit; bit >>= 1)
        if (__syncthreads_count(key >= (bound | bit)) >= per) bound |= bit;
    } else {
      // the largest of every warp or eight lanes
      const int lanes = most_per <= 8 ? 32 : 8, n = NT / lanes;
      if (tid == 0) S.bound = ~0u;         // of a CTA that has no share
      uint32_t m = key;
      for (int o = 1; o < lanes; o <<= 1) m = max(m, __shfl_xor_sync(~0u, m, o));
      if (lane % lanes == 0) S.start[tid / lanes] = m;
      __syncthreads();
      if (tid < n) {
        const uint32_t own = S.start[tid];
        int above = 0;
        for (int i = 0; i < n; ++i) above += S.start[i] > own || (S.start[i] == own && i < tid);
        if (above == per - 1) S.bound = own;
      }
      __syncthreads();
      bound = S.bound;
    }
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
  float largest = unordered(top);
  if (greedy) {
    int at = V;
    each(ahead, [&](int j, const float(&w)[4]) {
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

  if (largest == CUDART_INF_F) infinite = true, largest = 0.0f;

  // The CTAs' lists, one after another, to the first CTA's `cand`: a warp a list.
  const auto gather = [&](const u64(*told)[3]) {
    const int mine = lane < C ? (int)told[lane][2] : 0;
    const int at = __reduce_add_sync(~0u, lane < warp ? mine : 0), m = __shfl_sync(~0u, mine, warp);
    if (warp < C) {
      const uint32_t from = cluster_addr(list, warp);
      for (int i = lane; i < m; i += 32) cand[at + i] = ld_cluster64(from + i * 8);
    }
    __syncthreads();
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

  // The candidates that the first CTA has gathered, in falling order: those neighbouring
  // places 4 * tid .. are in p afterwards, 0 behind the last.
  Place p[4];
  float z[4];
  const auto in_order = [&](int n) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (tid + i * NT < n) p[i] = cand[tid + i * NT], z[i] = z_of(unordered((uint32_t)(p[i] >> 32)), largest, c);
    sort_down(S, p, z, n, list, cand);
#pragma unroll
    for (int i = 0; i < 4; ++i) p[i] = 4 * tid + i < n ? cand[4 * tid + i] : 0;
  };
  const auto weight_of = [&](Place p) { return weight(exp_of(unordered((uint32_t)(p >> 32)), largest, c)); };

  if (few) {
    const float reach = infinite ? 0.0f : bound ? unordered(bound) : -CUDART_INF_F;
    each(ahead, [&](int j, const float(&w)[4]) {
#pragma unroll
      for (int i = 0; i < 4; ++i)          // from 2^-43 on nothing weighs anything
        if (w[i] >= reach && z_of(w[i], largest, c) < 43.0f) note(place_of(w[i], first + j * 128 + i));
    });
    __syncthreads();
    const auto told = tell(0, 0, S.n);
    bool fits;
    int n = listed(told, &fits);
    if (fits) {
      if (rank == 0) {
        gather(told);
        in_order(n);
        u64 w[4], sum = 0, before;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          w[i] = 4 * tid + i < (k_on ? min(k, n) : n) ? weight_of(p[i]) : 0;
          sum += w[i];
        }
        sum = block_sum(S, sum, &before);
        const u64 need = p_on ? max(share(sum, P), (u64)1) : ~0ull;
        if (tid == 0) S.n = 0;
        __syncthreads();
        // what stays, by id
        sum = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const bool in = before < need && w[i] >= max(least, (u64)1);
          before += w[i];
          if (in) cand[atomicAdd(&S.n, 1u)] = p[i] << 32 | p[i] >> 32, sum += w[i];
        }
        sum = block_sum(S, sum, &before);
        n = S.n;
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (tid + i * NT < n) p[i] = cand[tid + i * NT], z[i] = (float)~(uint32_t)(p[i] >> 32);
        sort_down(S, p, z, n, list, cand);
        u64 own = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          p[i] = 4 * tid + i < n ? cand[4 * tid + i] : 0;
          w[i] = p[i] ? weight_of(p[i] << 32) : 0;
          own += w[i];
        }
        block_sum(S, own, &before);
        const u64 at = share(sum, U);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if (before <= at && at < before + w[i]) a.tokens[row] = (int)~(uint32_t)(p[i] >> 32);
          before += w[i];
        }
      }
      if (C > 1) meet();                   // the others' lists have been read
      return;
    }
    meet();
  }

  // What stays so far: weights from `sure` on, and of those from `maybe` on the ones whose place is
  // `cut` or before.
  uint32_t sure = 0, maybe = 0;
  Place cut = 0;
  const auto e_of = [&](float x) { return exp_of(x, largest, c); };
  // e of four neighbours, 0 for those that do not stay
  const auto left_of = [&](const float(&x)[4], int j, float(&e)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) e[i] = e_of(x[i]);
    if (sure > E_MIN) {                    // else those weigh nothing
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t b = __float_as_uint(e[i]);
        const int id = first + j * 128 + i;
        if (b < sure && !(b >= maybe && place_of(x[i], id) >= cut)) e[i] = 0.0f;
      }
    }
  };
  if (k_on || p_on) sure = maybe = E_MIN;  // the others weigh nothing, and may lie outside the row
  bool summed = false;                     // the sums of the warps are known already
  for (int stage = 0; stage < 2; ++stage) {
    // stage 0 counts ids up to k, stage 1 weights up to top_p of what is left
    if (stage == 0 ? !k_on : !p_on) continue;
    for (int i = tid; i < BINS / 4; i += NT) reinterpret_cast<uint4*>(hist)[i] = make_uint4(0, 0, 0, 0);
    if (tid == 0) S.n = 0;
    __syncthreads();
    u64 whole = 0, before;
    each(two_ahead, [&](int j, const float(&x)[4]) {
      float e[4];
      left_of(x, j, e);
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (__float_as_uint(e[i]) >= E_MIN) atomicAdd(&hist[(__float_as_uint(e[i]) - E_MIN) >> SH], 1u);
      Weights w;
#pragma unroll
      for (int i = 0; i < 4; ++i) w.add(e[i]);
      whole += w.sum(4);
    });
    whole = block_sum(S, whole, &before);
    // each octave's ids, and the sum of their bins' lower edges (256 .. 511), to all CTAs
    for (int o = warp; o < OCTAVES; o += NW) {
      const uint4* h = reinterpret_cast<const uint4*>(hist + (o << SUB_LOG)) + lane * 2;
      const uint4 u = h[0], w = h[1];
      const uint32_t ids = u.x + u.y + u.z + u.w + w.x + w.y + w.z + w.w, e = (1 << SUB_LOG) + lane * 8;
      const uint32_t all = __reduce_add_sync(~0u, ids);
      const uint32_t edges = __reduce_add_sync(~0u, ids * e + u.y + 2 * u.z + 3 * u.w + 4 * w.x + 5 * w.y + 6 * w.z + 7 * w.w);
      if (lane < C) st_cluster64(cluster_addr(&S.octaves[rank][o], lane), (u64)all << 32 | edges);
    }
    const auto told_whole = tell(whole, 0, 0);
    whole = 0;
    for (int r = 0; r < C; ++r) whole += told_whole[r][0];
    u64 need = stage == 0 ? (u64)k : max(share(whole, P), (u64)1);
    // The bins that may hold the cut.  The sum down to a bin lies between those of the bins' edges, from
    // the top as from the bottom, the whole sum being known.  Warp 0 looks for the first bin
    // down to which it may reach `need`, warp 1 for the last one above which it may not have yet:
    // for their octaves first.
    struct Bounds {
      u64 most, least;
    };
    const auto bounds = [&](u64 ids, u64 edges, int o) {
      if (stage == 0) return Bounds{ids, ids};
      if (o == OCTAVES - 1) return Bounds{ids << 42, ids << 42};         // the largest logits alone
      if (o < SUB_LOG) return Bounds{ids << (o + 1), 0};
      return Bounds{(edges + ids) << (o - SUB_LOG), edges << (o - SUB_LOG)};
    };
    const bool far = warp == 1;
    u64 most_all = 0, least_all = 0, most0 = 0, least0 = 0, sum = 0;
    const auto there = [&](u64 m, u64 l, u64 m1, u64 l1) {               // sums above and down to here
      return far ? max(l, sum + m > most_all ? sum + m - most_all : 0) < need : min(m1, sum - least_all + l1) >= need;
    };
    if (warp < 2) {
      Bounds v[2];                         // two octaves a lane, the largest weights first
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int o = OCTAVES - 1 - (2 * lane + i);
        u64 ids = 0, edges = 0;
        if (o >= 0)
          for (int r = 0; r < C; ++r) ids += S.octaves[r][o] >> 32, edges += (uint32_t)S.octaves[r][o];
        v[i] = bounds(ids, edges, max(o, 0));
      }
      u64 most = warp_before(v[0].most + v[1].most), least = warp_before(v[0].least + v[1].least);
      most_all = __shfl_sync(~0u, most + v[0].most + v[1].most, 31);
      least_all = __shfl_sync(~0u, least + v[0].least + v[1].least, 31);
      sum = stage == 0 ? most_all : whole;
      int mine = -1;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const u64 m1 = most + v[i].most, l1 = least + v[i].least;
        if (2 * lane + i < OCTAVES && (far || mine < 0) && there(most, least, m1, l1)) mine = 2 * lane + i, most0 = most, least0 = least;
        most = m1, least = l1;
      }
      const uint32_t who = __ballot_sync(~0u, mine >= 0);
      const int from = (far ? 31 - __clz(who) : __ffs(who) - 1) & 31;
      mine = __shfl_sync(~0u, mine, from);
      most0 = __shfl_sync(~0u, most0, from), least0 = __shfl_sync(~0u, least0, from);
      // stage 0: where no more than k weigh anything, all of those stay
      if (lane == 0) S.o[warp] = stage == 0 && sum <= need ? -1 : OCTAVES - 1 - max(mine, 0);
    }
    __syncthreads();
    const int o0 = S.o[0], o1 = S.o[1];
    if (o0 < 0) {
      meet();                              // S.octaves has been read
      continue;
    }
    {
      // the bins of those two octaves: C threads a bin add it up, and tell one CTA each
      const int b = rank * (NT / C) + tid / C, r = tid & (C - 1);
      static_assert(NT == 2 << SUB_LOG, "a bin a thread of each CTA");
      const uint32_t* h = hist + ((b >> SUB_LOG ? o1 : o0) << SUB_LOG) + (b & ((1 << SUB_LOG) - 1));
      uint32_t n = ld_cluster32(cluster_addr(h, r));
      for (int o = C >> 1; o; o >>= 1) n += __shfl_xor_sync(~0u, n, o);
      st_cluster32(cluster_addr(&S.ends[b], r), n);
      meet();
    }
    if (warp < 2) {
      Bounds v[8];                         // eight bins a lane, the largest weights first
      const int o = far ? o1 : o0, b = (31 - lane) * 8;
      u64 m8 = 0, l8 = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const u64 n = S.ends[(warp << SUB_LOG) + b + i];
        v[i] = bounds(n, n * ((1 << SUB_LOG) + b + i), o);
        m8 += v[i].most, l8 += v[i].least;
      }
      u64 most = most0 + warp_before(m8), least = least0 + warp_before(l8);
      int bin = -1;
#pragma unroll
      for (int i = 7; i >= 0; --i) {
        const u64 m1 = most + v[i].most, l1 = least + v[i].least;
        if ((far || bin < 0) && there(most, least, m1, l1)) bin = b + i;
        most = m1, least = l1;
      }
      const uint32_t hit = __ballot_sync(~0u, bin >= 0);
      bin = __shfl_sync(~0u, bin, (far ? 31 - __clz(hit) : __ffs(hit) - 1) & 31);
      if (lane == 0) S.i[warp] = (o << SUB_LOG) + bin;
    }
    __syncthreads();
    // one more on either side, since the order within 2^-20 of a weight is that of logits alone
    const int b_hi = min(BINS - 1, S.i[0] + 1), b_lo = max(0, S.i[1] - 1);
    const uint32_t above = E_MIN + ((uint32_t)(b_hi + 1) << SH), from = E_MIN + ((uint32_t)b_lo << SH);
    // what lies above them, exactly; those among them go to the list
    uint32_t count = 0;
    u64 over = 0;
    each(two_ahead, [&](int j, const float(&x)[4]) {
      float e[4];
      left_of(x, j, e);
      Weights w;
      uint32_t among = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t b = __float_as_uint(e[i]);
        w.add(b >= above ? e[i] : 0.0f);
        if (stage == 0) count += b >= above;
        if (b - from < above - from) among |= 1u << i;
      }
      over += w.sum(4);
      if (among) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (among >> i & 1) note(place_of(x[i], first + j * 128 + i));
      }
    });
    // f(place) for each of those among them
    const auto band = [&](auto f) {
      each(one_by_one, [&](int j, const float(&x)[4]) {
        float e[4];
        left_of(x, j, e);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t b = __float_as_uint(e[i]);
          if (b >= from && b < above) f(place_of(x[i], first + j * 128 + i));
        }
      });
    };
    const u64 warp_over = warp_sum(over);
    over = block_sum(S, stage == 0 ? (u64)count : over, &before);
    const auto told = tell(over, 0, S.n);
    over = 0;
    for (int r = 0; r < C; ++r) over += told[r][0];
    bool fits;
    const int n = listed(told, &fits);
    if (fits) {
      if (rank == 0) {
        gather(told);
        in_order(n);
        u64 w[4], own = 0, run;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          w[i] = !p[i] ? 0 : stage == 0 ? 1 : weight_of(p[i]);
          own += w[i];
        }
        block_sum(S, own, &run);
        run += over;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if (run < need && need <= run + w[i])
            for (int r = 0; r < C; ++r) st_cluster64(cluster_addr(&S.cut, r), p[i]);
          run += w[i];
        }
      }
      meet();
    } else {
      // More than fit, as ties make them: halves of their logits, each time between the smallest and
      // the largest that are left.
      uint32_t k_lo = ~0u, k_hi = 0;
      const auto size_of = [&](Place p) { return stage == 0 ? (u64)1 : weight_of(p); };
      const auto agree = [&](u64 v, uint32_t lo, uint32_t hi, u64* all, uint32_t* all_lo, uint32_t* all_hi) {
        u64 b;
        v = block_sum(S, v, &b);
        lo = block_min(S, lo);
        hi = ~block_min(S, ~hi);
        const auto told = tell(v, lo, hi);
        *all = 0;
        *all_lo = ~0u, *all_hi = 0;
        for (int r = 0; r < C; ++r) {
          *all += told[r][0];
          *all_lo = min(*all_lo, (uint32_t)told[r][1]);
          *all_hi = max(*all_hi, (uint32_t)told[r][2]);
        }
      };
      u64 v;
      band([&](Place p) { k_lo = min(k_lo, (uint32_t)(p >> 32)), k_hi = max(k_hi, (uint32_t)(p >> 32)); });
      agree(0, k_lo, k_hi, &v, &k_lo, &k_hi);
      while (k_lo < k_hi) {
        const uint32_t mid = k_lo + (k_hi - k_lo) / 2;
        u64 up = 0;
        uint32_t up_lo = ~0u, down_hi = 0;
        band([&](Place p) {
          const uint32_t o = (uint32_t)(p >> 32);
          if (o > mid && o <= k_hi) up += size_of(p), up_lo = min(up_lo, o);
          if (o <= mid && o >= k_lo) down_hi = max(down_hi, o);
        });
        agree(up, up_lo, down_hi, &v, &up_lo, &down_hi);
        if (over + v >= need)
          k_lo = up_lo;
        else
          over += v, k_hi = down_hi;
      }
      // equal logits: the first so many by id
      const u64 one = size_of((Place)k_lo << 32), wanted = (need - over + one - 1) / one;
      u64 mine = 0;
      band([&](Place p) { mine += p >> 32 == k_lo; });
      const u64 warp_ties = warp_sum(mine);
      __syncthreads();
      if (lane == 0) S.red[1][warp] = warp_ties;
      const u64 cta = block_sum(S, mine, &before);
      const auto told = tell(cta, 0, 0);
      u64 run = 0;
      for (int r = 0; r < rank; ++r) run += told[r][0];
      for (int w = 0; w < warp; ++w) run += S.red[1][w];
      if (run < wanted && wanted <= run + warp_ties) {
        // the warp with the last of them, 128 ids at a time
        each(one_by_one, [&](int j, const float(&x)[4]) {
          float e[4];
          left_of(x, j, e);
          u64 n = 0;
          bool tie[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            tie[i] = ordered(x[i]) == k_lo && __float_as_uint(e[i]) >= E_MIN;
            n += tie[i];
          }
          u64 at = run + warp_before(n);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            at += tie[i];
            if (tie[i] && at == wanted)
              for (int r = 0; r < C; ++r) st_cluster64(cluster_addr(&S.cut, r), place_of(unordered(k_lo), first + j * 128 + i));
          }
          run += warp_sum(n);
        });
      }
      meet();
    }
    cut = S.cut;
    // Sums of warps: what lies above, known already, and what of the list stays; unless min-p takes off more.
    summed = stage == 1 && fits && least <= weight(__uint_as_float(from));
    if (summed) {
      __syncthreads();
      if (lane == 0) S.red[1][warp] = warp_over;
      __syncthreads();
      // the first CTA's own list has been sorted away: it looks through all
      const u64* of = rank == 0 ? cand : list;
      const int m = rank == 0 ? n : (int)told[rank][2], id0 = rank * NW * fours * 128 - shift;
      for (int i = tid; i < m; i += NT) {
        const int w = ((int)~(uint32_t)of[i] - id0) / (fours * 128);
        if (of[i] >= cut && w < NW) atomicAdd(&S.red[1][w], weight_of(of[i]));
      }
      __syncthreads();
    }
    sure = max(sure, above), maybe = from;                 // what top-k has cut off stays so
    meet();                                // before anything here is written again
  }

  // What stays, all of it; then the id at the threshold.
  // (w >= least where 2^42 e is)
  const float e_least = __double2float_ru((double)least * 0x1p-42);
  if (!summed) {
    u64 own = 0;
    each(two_ahead, [&](int j, const float(&x)[4]) {
      float e[4];
      left_of(x, j, e);
      Weights w;
#pragma unroll
      for (int i = 0; i < 4; ++i) w.add(e[i] >= e_least ? e[i] : 0.0f);
      own += w.sum(4);
    });
    own = warp_sum(own);
    __syncthreads();
    if (lane == 0) S.red[1][warp] = own;
    __syncthreads();
  }
  const u64 warp_own = S.red[1][warp];
  u64 cta = warp_sum(lane < NW ? S.red[1][lane] : 0);
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
  each(one_by_one, [&](int j, const float(&x)[4]) {
    if (found) return;
    float e[4];
    left_of(x, j, e);
    u64 w[4], n = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      w[i] = e[i] >= e_least ? weight(e[i]) : 0;
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

template <typename X>
cudaError_t run(const DrawArgs& a, int C, int fours, cudaStream_t s) {
  static thread_local KernCache cache;
  static thread_local int allowed = -1;
  constexpr int SMEM = BINS * 4;
  cudaError_t e = prep_kernel(draw_kernel<X>, cache, NT, SMEM, nullptr);
  if (e == cudaSuccess && C > 8 && allowed != cache.dev) {  // clusters of 16 are opt-in, a function and device
    e = cudaFuncSetAttribute(draw_kernel<X>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    allowed = cache.dev;
  }
  if (e != cudaSuccess) return e;
  return launch_step(draw_kernel<X>, dim3((unsigned)a.rows * C), NT, SMEM, s, C, a, C, fours);
}

// CTAs a row: so many that each thread has two fours, but no more than run at once, or twice as many
// while a thread has more than 16 (128 rows of 262144: 205 us with two CTAs a row, 186 with four, 210 with
// eight; 32 rows: 75, 60 and 103 with four, eight and sixteen; 512 rows of 32000: 101 and 134 with one and two).
// One CTA is enough where a thread has four fours at most, since its barriers cost less than a
// cluster's (a row of 6000 with top-k 50: 11.3 us, 12.6 with two).  A cluster of 16 keeps one of the eight parts of the
// GPU to itself, so more rows than these have them only for long rows (9 rows of 50257, top-k 50: 14.7 us with sixteen
// CTAs and 12.0 with eight; one row 11.2 and 11.5).
template <typename X>
cudaError_t typed(const DrawArgs& a, cudaStream_t s) {
  const bool even = (a.rows == 1 || a.ldx % 4 == 0) && (uintptr_t)a.x % (4 * sizeof(X)) == 0;
  const int elements = a.V + (even ? 0 : 3);               // wherever the row begins
  const auto fours = [&](int C) { return (elements + C * NT * 4 - 1) / (C * NT * 4); };
  int C = 1;
  const int64_t at_once = 2 * dev_info().sms;
  if (fours(1) > 4)
    while (C < MAX_C && (fours(C) > 2 && C * 2 * (int64_t)a.rows <= at_once || fours(C) > 16 && C * (int64_t)a.rows <= at_once) &&
           !(C == 8 && a.rows > 8 && fours(C) <= 4))
      C *= 2;
  return run<X>(a, C, fours(C), s);
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
