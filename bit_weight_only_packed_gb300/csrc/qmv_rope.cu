// qmv_rope.cu -- norms of query and key heads and their position rotation (qmv_qk_norm_rope):
//   u = x / sqrt(mean x^2 + eps) * gamma;  (a, b) -> amplitude * (a cos t - b sin t, b cos t + a sin t).
//
// A lane owns whole pairs: W neighbouring elements of the first half of what is turned and the
// W that they pair with (or 2 W neighbours, where pairs lie side by side or nothing is
// turned), so a head costs no exchange but the sum of its squares.  Its cosines and
// sines belong to the token, and a warp takes B heads at a time of one token, so they are formed
// once for all its heads.  The angle is position * turns modulo 2^64, exact at any
// position; its upper 32 bits go to sincospi.
#include "qmv_token.cuh"

namespace qmv {
namespace {

// W neighbouring elements, aligned to themselves, as they are stored.
template <typename T, int W>
struct alignas(W * sizeof(T) < 16 ? W * sizeof(T) : 16) Run {
  T v[W];
};

template <typename X, typename T, int W, int U, int B, bool SIDE>
__global__ void __launch_bounds__(128) rope_kernel(RopeArgs a, int lanes_log, int units, int splits, int per) {
  const int lane = threadIdx.x & 31, L = 1 << lanes_log, l = lane & (L - 1), hpw = 32 >> lanes_log;
  const int64_t item = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
  const int m = (int)(item / splits), part = (int)(item - (int64_t)m * splits), H = a.nq + a.nk;
  pdl_begin();
  if (m >= a.M) return;
  // this lane's units: where their two halves begin, and their cosines and sines
  const int turned = a.rot / (2 * W);
  int ea[U], eb[U];
  float c[U][W], s[U][W];
  bool on[U], both[U];
#pragma unroll
  for (int j = 0; j < U; ++j) {
    const int u = l + j * L;
    const bool half = !SIDE && u < turned;
    on[j] = u < units;
    ea[j] = half ? u * W : 2 * u * W;
    eb[j] = half ? a.rot / 2 + u * W : (2 * u + 1) * W;
    both[j] = on[j] && (W > 1 || eb[j] < a.D);
#pragma unroll
    for (int i = 0; i < W; ++i) c[j][i] = 1.0f, s[j][i] = 0.0f;
    if (u < turned) {
      const uint64_t pos = (uint64_t)(int64_t)a.positions[m];
#pragma unroll
      for (int i = 0; i < W; ++i) {
        const int t = (int)((pos * (uint64_t)a.turns[u * W + i]) >> 32);       // turns, in 2^-32
        sincospif((float)t * 0x1p-31f, &s[j][i], &c[j][i]);
        s[j][i] *= a.amplitude;
        c[j][i] *= a.amplitude;
      }
    }
  }
  const X* x = (const X*)a.x + (int64_t)m * a.ld;
  const float inv_d = 1.0f / (float)a.D;
  const int h_end = min(H, (part + 1) * per * hpw * B);
  for (int h0 = part * per * hpw * B + (lane >> lanes_log); h0 < h_end + (lane >> lanes_log); h0 += hpw * B) {
    Run<X, W> xa[B][U], xb[B][U];
#pragma unroll
    for (int b = 0; b < B; ++b) {
      const int h = h0 + b * hpw;
#pragma unroll
      for (int j = 0; j < U; ++j) {
#pragma unroll
        for (int i = 0; i < W; ++i) xa[b][j].v[i] = xb[b][j].v[i] = from_f<X>(0.0f);
        if (h < h_end && on[j]) xa[b][j] = *reinterpret_cast<const Run<X, W>*>(x + (int64_t)h * a.D + ea[j]);
        if (h < h_end && both[j]) xb[b][j] = *reinterpret_cast<const Run<X, W>*>(x + (int64_t)h * a.D + eb[j]);
      }
    }
#pragma unroll
    for (int b = 0; b < B; ++b) {
      const int h = h0 + b * hpw;
      const bool is_q = h < a.nq;
      const T* gamma = (const T*)(is_q ? a.gamma_q : a.gamma_k);
      float va[U][W], vb[U][W], ss = 0.0f;
#pragma unroll
      for (int j = 0; j < U; ++j)
#pragma unroll
        for (int i = 0; i < W; ++i) {
          va[j][i] = to_f<X>(xa[b][j].v[i]);
          vb[j][i] = to_f<X>(xb[b][j].v[i]);
          ss = fmaf(va[j][i], va[j][i], ss);
          ss = fmaf(vb[j][i], vb[j][i], ss);
        }
      for (int o = L >> 1; o; o >>= 1) ss += __shfl_xor_sync(~0u, ss, o);
      if (h >= h_end) continue;
      if (gamma) {
        const float r = 1.0f / sqrtf(fmaf(ss, inv_d, a.eps));
#pragma unroll
        for (int j = 0; j < U; ++j) {
          Run<T, W> ga, gb;
#pragma unroll
          for (int i = 0; i < W; ++i) ga.v[i] = gb.v[i] = from_f<T>(0.0f);
          if (on[j]) ga = *reinterpret_cast<const Run<T, W>*>(gamma + ea[j]);
          if (both[j]) gb = *reinterpret_cast<const Run<T, W>*>(gamma + eb[j]);
#pragma unroll
          for (int i = 0; i < W; ++i) {
            va[j][i] = va[j][i] * r * (to_f<T>(ga.v[i]) + a.goff);
            vb[j][i] = vb[j][i] * r * (to_f<T>(gb.v[i]) + a.goff);
          }
        }
      }
      T* out = is_q ? (T*)a.q + (int64_t)m * a.ldq + (int64_t)h * a.D : (T*)a.k + (int64_t)m * a.ldk + (int64_t)(h - a.nq) * a.D;
#pragma unroll
      for (int j = 0; j < U; ++j) {
        Run<T, W> oa, ob;
        if (SIDE && W > 1) {
#pragma unroll
          for (int i = 0; i < W; ++i) {
            // pair i: the first W / 2 lie in a, the others in b
            float(&v)[W] = i < W / 2 ? va[j] : vb[j];
            Run<T, W>& o = i < W / 2 ? oa : ob;
            const int k = 2 * (i % (W / 2));
            o.v[k] = from_f<T>(v[k] * c[j][i] - v[(k + 1) % W] * s[j][i]);
            o.v[(k + 1) % W] = from_f<T>(v[(k + 1) % W] * c[j][i] + v[k] * s[j][i]);
          }
        } else {
#pragma unroll
          for (int i = 0; i < W; ++i) {
            oa.v[i] = from_f<T>(va[j][i] * c[j][i] - vb[j][i] * s[j][i]);
            ob.v[i] = from_f<T>(vb[j][i] * c[j][i] + va[j][i] * s[j][i]);
          }
        }
        if (on[j]) *reinterpret_cast<Run<T, W>*>(out + ea[j]) = oa;
        if (both[j]) *reinterpret_cast<Run<T, W>*>(out + eb[j]) = ob;
      }
    }
  }
}

template <typename X, typename T, int W, int U, int B, bool SIDE>
cudaError_t run(const RopeArgs& a, cudaStream_t s) {
  const int units = W > 1 ? a.D / (2 * W) : a.rot / 2 + (a.D - a.rot + 1) / 2;
  int lanes_log = 0;
  while (lanes_log < 5 && (U << lanes_log) < units) ++lanes_log;
  // a warp for all heads of a token where tokens are many, for fewer heads otherwise
  const int heads = (32 >> lanes_log) * B, batches = (a.nq + a.nk + heads - 1) / heads;
  const int64_t want = (int64_t)dev_info().sms * 16;
  int splits = (int)((want + a.M - 1) / a.M);
  splits = splits < batches ? splits : batches;
  const int per = (batches + splits - 1) / splits;
  splits = (batches + per - 1) / per;
  return launch_step(rope_kernel<X, T, W, U, B, SIDE>, dim3((unsigned)(((int64_t)a.M * splits + 3) / 4)), 128, 0, s, 1, a,
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
  constexpr int B = sizeof(X) == 4 ? 2 : 4;
  if (a.D <= 512 && whole(8)) return side ? run<X, T, 8, 1, B, true>(a, s) : run<X, T, 8, 1, B, false>(a, s);
  if (a.D <= 256 && whole(4)) return side ? run<X, T, 4, 1, B, true>(a, s) : run<X, T, 4, 1, B, false>(a, s);
  // single elements: the layouts differ in places only
  if (a.D <= 64) return side ? run<X, T, 1, 1, 4, true>(a, s) : run<X, T, 1, 1, 4, false>(a, s);
  if (a.D <= 256) return side ? run<X, T, 1, 4, 2, true>(a, s) : run<X, T, 1, 4, 2, false>(a, s);
  return side ? run<X, T, 1, 16, 1, true>(a, s) : run<X, T, 1, 16, 1, false>(a, s);
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
