// qmv_rope.cu -- norms of query and key heads and their position rotation (qmv_qk_norm_rope):
//   u = x / sqrt(mean x^2 + eps) * gamma;  (a, b) -> amplitude * (a cos t - b sin t, b cos t + a sin t).
//
// A lane owns whole pairs: W neighbouring elements of the first half of what is turned and the W that they
// pair with (or 2 W neighbours, where pairs lie side by side or nothing is turned), so a head costs no
// exchange but the sum of its squares.  Its cosines and sines belong to the token, whose heads a warp takes one
// after another, so they are formed once for all of them.  The angle is position * turns modulo 2^64, exact at
// any position; its upper 32 bits go to sincospi.  The gammas go into the cosines and sines, so that an element
// of a head costs three operations, its square and its conversions.
//
// Bound by HBM where tokens are many, which takes more heads on their way than registers hold: with the next
// head in registers (loads without conditions, since one under a condition waits for those before it) 8192
// tokens of 32 + 8 heads of 256 took 91 us, with the next two 76; with three in shared memory, copied by each
// thread for itself so that nobody waits for another, 55 (6.1 TB/s; a copy of the same bytes takes 51), and
// 1024 tokens of 32 + 8 heads of 128 8.3 us against 10.4.  Runs of other sizes than 16 bytes gain nothing by that
// (3000 tokens of 68 heads of 64 in fp32: 20.0 us and 18.1; of 15 heads of 72: 10.3 both) and keep to registers.
// Heads whose size, place or stride leaves no runs (odd ones, and all above 512) go an element at a time: 4096 tokens of
// 10 heads of 100 in 12.8 us, of 9 heads of 528 in 66.8, where 9 heads of 512 in runs of 8 take 17.1.
// A few tokens are bound by latency: 2.1 us.
#include "qmv_token.cuh"

namespace qmv {
namespace {

// W neighbouring elements, aligned to themselves, as they are stored.
template <typename T, int W>
struct alignas(W * sizeof(T) < 16 ? W * sizeof(T) : 16) Run {
  T v[W];
};

// Two neighbours rounded by one instruction.
__device__ __forceinline__ void pair_of(float a, float b, __half* to) { *reinterpret_cast<__half2*>(to) = __floats2half2_rn(a, b); }
__device__ __forceinline__ void pair_of(float a, float b, __nv_bfloat16* to) {
  *reinterpret_cast<__nv_bfloat162*>(to) = __floats2bfloat162_rn(a, b);
}

// 16 bytes from global to shared memory, on their way.
__device__ __forceinline__ void copy_ahead(void* to, const void* from) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"((uint32_t)__cvta_generic_to_shared(to)), "l"(from) : "memory");
}

constexpr int STAGES = 4;

// Heads on their way in shared memory: where a run is one copy of 16 bytes.
template <typename X, int W>
constexpr bool RINGED = W * sizeof(X) == 16;

template <typename X, typename T, int W, int U, bool SIDE>
__global__ void __launch_bounds__(128, RINGED<X, W> ? 5 : U <= 1 ? 4 : 1) rope_kernel(RopeArgs a, int lanes_log, int units, int splits, int per) {
  const int lane = threadIdx.x & 31, L = 1 << lanes_log, l = lane & (L - 1), hpw = 32 >> lanes_log;
  const int64_t item = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
  const int m = (int)(item / splits), part = (int)(item - (int64_t)m * splits), H = a.nq + a.nk;
  pdl_begin();
  if (m >= a.M) return;
  // this lane's units: where their two halves begin (the head's first elements, where it has none)
  const int turned = a.rot / (2 * W);
  int ea[U], eb[U];
  bool on[U], both[U];
#pragma unroll
  for (int j = 0; j < U; ++j) {
    const int u = l + j * L;
    const bool half = !SIDE && u < turned;
    on[j] = u < units;
    ea[j] = half ? u * W : 2 * u * W;
    eb[j] = half ? a.rot / 2 + u * W : (2 * u + 1) * W;
    both[j] = on[j] && (W > 1 || eb[j] < a.D);
    if (!on[j]) ea[j] = 0;
    if (!both[j]) eb[j] = 0;
  }
  const X* x = (const X*)a.x + (int64_t)m * a.ld;
  const int first = part * per * hpw, h_end = min(H, first + per * hpw), own = lane >> lanes_log;
  Run<X, W> xa[U], xb[U];
  const auto load = [&](int h0) {
    const X* head = x + (int64_t)min(h0 + own, H - 1) * a.D;
#pragma unroll
    for (int j = 0; j < U; ++j) {
      xa[j] = *reinterpret_cast<const Run<X, W>*>(head + ea[j]);
      xb[j] = *reinterpret_cast<const Run<X, W>*>(head + eb[j]);
    }
  };
  constexpr bool RING = RINGED<X, W>;
  __shared__ uint4 ring[RING ? STAGES : 1][2][RING ? 128 : 1];           // a thread's two runs
  const auto copy = [&](int h0, int stage) {
    if (h0 < h_end) {
      const X* head = x + (int64_t)min(h0 + own, H - 1) * a.D;
      copy_ahead(&ring[stage][0][threadIdx.x], head + ea[0]);
      copy_ahead(&ring[stage][1][threadIdx.x], head + eb[0]);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  if constexpr (RING) {
    for (int i = 0; i < STAGES - 1; ++i) copy(first + i * hpw, i);
  } else {
    load(first);
  }
  // and their cosines and sines
  float c[U][W], s[U][W];
#pragma unroll
  for (int j = 0; j < U; ++j)
#pragma unroll
    for (int i = 0; i < W; ++i) c[j][i] = 1.0f, s[j][i] = 0.0f;
  if (turned) {
    const uint64_t pos = (uint64_t)(int64_t)a.positions[m];
#pragma unroll
    for (int j = 0; j < U; ++j) {
      const int u = l + j * L;
      uint64_t turns[W];
#pragma unroll
      for (int i = 0; i < W; ++i) turns[i] = (uint64_t)a.turns[min(u, turned - 1) * W + i];
      if (u < turned) {
#pragma unroll
        for (int i = 0; i < W; ++i) {
          const int t = (int)((pos * turns[i]) >> 32);           // turns, in 2^-32
          sincospif((float)t * 0x1p-31f, &s[j][i], &c[j][i]);
          s[j][i] *= a.amplitude;
          c[j][i] *= a.amplitude;
        }
      }
    }
  }
  const float inv_d = 1.0f / (float)a.D;
  // pair i of a unit: element first_of(i) and its second, of the W in a and the W in b
  constexpr bool BESIDE = SIDE && W > 1;
  const auto first_of = [](int i) { return BESIDE ? 2 * i : i; };
  const auto second_of = [](int i) { return BESIDE ? 2 * i + 1 : W + i; };
  float p1[U][W], p2[U][W], q1[U][W], q2[U][W];
  int of = -1;                   // whose they are: 1 queries', 0 keys'
  const auto coefficients = [&](bool is_q) {
    const T* gamma = (const T*)(is_q ? a.gamma_q : a.gamma_k);
#pragma unroll
    for (int j = 0; j < U; ++j) {
      float g[2 * W];
#pragma unroll
      for (int i = 0; i < 2 * W; ++i) g[i] = 1.0f;
      if (gamma) {
        const Run<T, W> ga = *reinterpret_cast<const Run<T, W>*>(gamma + ea[j]), gb = *reinterpret_cast<const Run<T, W>*>(gamma + eb[j]);
#pragma unroll
        for (int i = 0; i < W; ++i) g[i] = to_f<T>(ga.v[i]) + a.goff, g[W + i] = to_f<T>(gb.v[i]) + a.goff;
      }
#pragma unroll
      for (int i = 0; i < W; ++i) {
        const float gp = g[first_of(i)], gq = g[second_of(i)];
        p1[j][i] = gp * c[j][i], p2[j][i] = gq * s[j][i], q1[j][i] = gq * c[j][i], q2[j][i] = gp * s[j][i];
      }
    }
    of = is_q;
  };
  int stage = 0;
  for (int h0 = first; h0 < h_end; h0 += hpw) {
    // (in place, the heads ahead lie outside what this one writes)
    Run<X, W> ya[U], yb[U];
    if constexpr (RING) {
      copy(h0 + (STAGES - 1) * hpw, stage ? stage - 1 : STAGES - 1);
      asm volatile("cp.async.wait_group %0;" ::"n"(STAGES - 1) : "memory");
      memcpy(ya[0].v, &ring[stage][0][threadIdx.x], 16);
      memcpy(yb[0].v, &ring[stage][1][threadIdx.x], 16);
      stage = stage + 1 < STAGES ? stage + 1 : 0;
    } else {
#pragma unroll
      for (int j = 0; j < U; ++j) ya[j] = xa[j], yb[j] = xb[j];
      if (h0 + hpw < h_end) load(h0 + hpw);
    }
    const int h = h0 + own;
    const bool is_q = h < a.nq;
    if (of != (int)is_q) coefficients(is_q);
    float v[U][2 * W], ss = 0.0f;
#pragma unroll
    for (int j = 0; j < U; ++j)
#pragma unroll
      for (int i = 0; i < W; ++i) {
        v[j][i] = to_f<X>(ya[j].v[i]);
        v[j][W + i] = to_f<X>(yb[j].v[i]);
        ss = on[j] ? fmaf(v[j][i], v[j][i], ss) : ss;
        ss = both[j] ? fmaf(v[j][W + i], v[j][W + i], ss) : ss;
      }
    for (int o = L >> 1; o; o >>= 1) ss += __shfl_xor_sync(~0u, ss, o);
    const float r = (is_q ? a.gamma_q : a.gamma_k) ? rsqrtf(fmaf(ss, inv_d, a.eps)) : 1.0f;
    T* out = is_q ? (T*)a.q + (int64_t)m * a.ldq + (int64_t)h * a.D : (T*)a.k + (int64_t)m * a.ldk + (int64_t)(h - a.nq) * a.D;
#pragma unroll
    for (int j = 0; j < U; ++j) {
      float y[2 * W];
#pragma unroll
      for (int i = 0; i < W; ++i) {
        const float p = v[j][first_of(i)], q = v[j][second_of(i)];
        float y1 = p * p1[j][i], y2 = q * q1[j][i];
        // (not 0 times the other one, which may be infinite)
        if (l + j * L < turned) y1 = fmaf(-q, p2[j][i], y1), y2 = fmaf(p, q2[j][i], y2);
        y[first_of(i)] = y1 * r;
        y[second_of(i)] = y2 * r;
      }
      Run<T, W> oa, ob;
      if constexpr (W > 1) {
#pragma unroll
        for (int i = 0; i < W; i += 2) pair_of(y[i], y[i + 1], oa.v + i), pair_of(y[W + i], y[W + i + 1], ob.v + i);
      } else {
        oa.v[0] = from_f<T>(y[0]), ob.v[0] = from_f<T>(y[1]);
      }
      if (h < h_end && on[j]) *reinterpret_cast<Run<T, W>*>(out + ea[j]) = oa;
      if (h < h_end && both[j]) *reinterpret_cast<Run<T, W>*>(out + eb[j]) = ob;
    }
  }
}

template <typename X, typename T, int W, int U, bool SIDE>
cudaError_t run(const RopeArgs& a, cudaStream_t s) {
  const int units = W > 1 ? a.D / (2 * W) : a.rot / 2 + (a.D - a.rot + 1) / 2;
  int lanes_log = 0;
  while (lanes_log < 5 && (U << lanes_log) < units) ++lanes_log;
  // a warp for all heads of a token where tokens are many, for fewer heads otherwise
  const int heads = 32 >> lanes_log, batches = (a.nq + a.nk + heads - 1) / heads;
  const int64_t want = (int64_t)dev_info().sms * 16;
  int splits = (int)((want + a.M - 1) / a.M);
  splits = splits < batches ? splits : batches;
  const int per = (batches + splits - 1) / splits;
  splits = (batches + per - 1) / per;
  return launch_step(rope_kernel<X, T, W, U, SIDE>, dim3((unsigned)(((int64_t)a.M * splits + 3) / 4)), 128, 0, s, 1, a,
                     lanes_log, units, splits, per);
}

template <typename X, typename T>
cudaError_t typed(const RopeArgs& a, cudaStream_t s) {
  const bool side = a.layout == QMV_ROPE_INTERLEAVED;
  const auto whole = [&](int w) {             // runs of w elements are whole and aligned everywhere
    const auto at = [&](const void* p, int64_t ld, size_t size) {
      const size_t al = w * size < 16 ? w * size : 16;
      return (uintptr_t)p % al == 0 && (a.M == 1 || ld * size % al == 0);
    };
    return a.D % (2 * w) == 0 && a.rot % (2 * w) == 0 && at(a.x, a.ld, sizeof(X)) && at(a.q, a.ldq, 2) && at(a.k, a.ldk, 2) &&
           at(a.gamma_q, 0, 2) && at(a.gamma_k, 0, 2);
  };
  if (a.D <= 512 && whole(8)) return side ? run<X, T, 8, 1, true>(a, s) : run<X, T, 8, 1, false>(a, s);
  if (a.D <= 256 && whole(4)) return side ? run<X, T, 4, 1, true>(a, s) : run<X, T, 4, 1, false>(a, s);
  // single elements: the layouts differ in places only
  if (a.D <= 64) return side ? run<X, T, 1, 1, true>(a, s) : run<X, T, 1, 1, false>(a, s);
  if (a.D <= 256) return side ? run<X, T, 1, 4, true>(a, s) : run<X, T, 1, 4, false>(a, s);
  return side ? run<X, T, 1, 16, true>(a, s) : run<X, T, 1, 16, false>(a, s);
}

}  // namespace

cudaError_t launch_rope(const RopeArgs& a, cudaStream_t s) {
  if (a.bf16) {
    switch (a.x_dtype) {
      case QMV_F32: return typed<float, __nv_bfloat16>(a, s);
      case QMV_F16: return typed<__half, __nv_bfloat16>(a, s);
      default: return typed<__nv_bfloat16, __nv_bfloat16>(a, s);
    }
  }
  switch (a.x_dtype) {
    case QMV_F32: return typed<float, __half>(a, s);
    case QMV_F16: return typed<__half, __half>(a, s);
    default: return typed<__nv_bfloat16, __half>(a, s);
  }
}

}  // namespace qmv
