// qmv_sample.cu -- logits to probabilities (qmv_softmax) and drafted tokens
// against the target's probabilities (qmv_verify_draft).
#include <math_constants.h>

#include "qmv_step.cuh"

namespace qmv {
namespace {

constexpr int MAX_NT = 512, MAX_C = 16;

// ----------------------------------------------------------------- softmax --

// What a CTA knows of its part of a row, and two parts joined.
struct Part {
  float m, s;      // maximum; sum of exp((x - m) / T)
  int at, bad;     // first place of the maximum; NaN or +inf seen
};

__device__ __forceinline__ void join_max(Part& a, const Part& b) {
  if (b.m > a.m || (b.m == a.m && b.at < a.at)) a.m = b.m, a.at = b.at;
  a.bad |= b.bad;
}

// Maximum (and sum, once every part is relative to one maximum) over a CTA.
__device__ __forceinline__ Part block_max(Part p, Part* red) {
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    Part q;
    q.m = __shfl_xor_sync(~0u, p.m, o);
    q.at = __shfl_xor_sync(~0u, p.at, o);
    q.bad = __shfl_xor_sync(~0u, p.bad, o);
    join_max(p, q);
  }
  const int lane = threadIdx.x & 31, nw = blockDim.x >> 5;
  if (lane == 0) red[threadIdx.x >> 5] = p;
  __syncthreads();
  p = red[lane < nw ? lane : 0];
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    Part q;
    q.m = __shfl_xor_sync(~0u, p.m, o);
    q.at = __shfl_xor_sync(~0u, p.at, o);
    q.bad = __shfl_xor_sync(~0u, p.bad, o);
    join_max(p, q);
  }
  return p;
}

__device__ __forceinline__ float block_sum(float v, float* red) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(~0u, v, o);
  const int lane = threadIdx.x & 31, nw = blockDim.x >> 5;
  if (lane == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  v = lane < nw ? red[lane] : 0.0f;
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(~0u, v, o);
  return v;
}

// A cluster of C CTAs a row (C = 1: no cluster).  EPT > 0: a CTA's part of the
// row stays in registers, EPT elements a thread, so that the row is read once;
// EPT == 0: a part of any length, read a second and third time (from L2).
template <typename X, int EPT>
__global__ void __launch_bounds__(MAX_NT) softmax_kernel(SoftmaxArgs a, int C, int len) {
  __shared__ Part red[MAX_NT / 32], mine;
  __shared__ float reds[MAX_NT / 32];
  const int row = blockIdx.x / C, rank = blockIdx.x - row * C, NT = blockDim.x, tid = threadIdx.x;
  const int v0 = min(a.V, rank * len), n = min(a.V - v0, len);     // this CTA's part
  const X* x = (const X*)a.x + (int64_t)row * a.ldx + v0;
  float* out = a.out + (int64_t)row * a.ldo + v0;
  pdl_begin();
  const float t = a.t ? a.t[row] : a.t0;
  const bool hot = !(t > 0.0f);
  // 1/T of a subnormal T is infinite; the largest finite factor keeps 0 * it = 0
  const float it = hot ? 0.0f : fminf(1.0f / t, 3.402823466e38f);
  constexpr int R = EPT ? EPT : 1;
  float e[R];
  Part p{-CUDART_INF_F, 0.0f, a.V, 0};
  if (EPT) {
#pragma unroll
    for (int j = 0; j < R; ++j) e[j] = j * NT + tid < n ? to_f<X>(x[j * NT + tid]) : -CUDART_INF_F;
#pragma unroll
    for (int j = 0; j < R; ++j) {
      if (e[j] > p.m) p.m = e[j], p.at = v0 + j * NT + tid;
      p.bad |= !(e[j] < CUDART_INF_F);
    }
  } else {
    for (int i = tid; i < n; i += NT) {
      const float v = to_f<X>(x[i]);
      if (v > p.m) p.m = v, p.at = v0 + i;
      p.bad |= !(v < CUDART_INF_F);
    }
  }
  p = block_max(p, red);
  // nothing but -inf so far: any finite maximum will do, every term is 0
  const float m = p.m == -CUDART_INF_F ? 0.0f : p.m;
  float s = 0.0f;
  if (EPT) {
#pragma unroll
    for (int j = 0; j < R; ++j) {
      e[j] = e[j] == -CUDART_INF_F ? 0.0f : expf((e[j] - m) * it);
      s += e[j];
    }
  } else {
    for (int i = tid; i < n; i += NT) {
      const float v = to_f<X>(x[i]);
      s += v == -CUDART_INF_F ? 0.0f : expf((v - m) * it);
    }
  }
  p.s = block_sum(s, reds);
  Part all = p;
  if (C > 1) {
    if (tid == 0) mine = p;
    cluster_arrive();
    cluster_wait();
    const uint32_t at = cluster_addr(&mine, (tid & 31) < C ? (tid & 31) : 0);
    Part q;
    q.m = __uint_as_float(ld_cluster32(at));
    q.s = (tid & 31) < C ? __uint_as_float(ld_cluster32(at + 4)) : 0.0f;
    q.at = (int)ld_cluster32(at + 8);
    q.bad = (int)ld_cluster32(at + 12);
    cluster_arrive();                        // waited for at the end: the others still read `mine`
    all = q;
#pragma unroll
    for (int o = 16; o; o >>= 1) {
      Part w;
      w.m = __shfl_xor_sync(~0u, all.m, o);
      w.at = __shfl_xor_sync(~0u, all.at, o);
      w.bad = __shfl_xor_sync(~0u, all.bad, o);
      join_max(all, w);
    }
    float sum = q.m == -CUDART_INF_F ? 0.0f : q.s * expf((q.m - all.m) * it);
#pragma unroll
    for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(~0u, sum, o);
    all.s = sum;
  }
  // special rows: NaN or +inf anywhere, nothing but -inf, the one-hot form
  if (all.bad || all.m == -CUDART_INF_F || hot) {
    for (int i = tid; i < n; i += NT)
      out[i] = all.bad ? CUDART_NAN_F : hot && v0 + i == all.at ? 1.0f : 0.0f;
  } else {
    const float f = expf((m - all.m) * it) / all.s;   // a part of -inf alone has only zeros
    if (EPT) {
#pragma unroll
      for (int j = 0; j < R; ++j)
        if (j * NT + tid < n) out[j * NT + tid] = p.m == -CUDART_INF_F ? 0.0f : e[j] * f;
    } else {
      for (int i = tid; i < n; i += NT) {
        const float v = to_f<X>(x[i]);
        out[i] = v == -CUDART_INF_F ? 0.0f : expf((v - all.m) * it) / all.s;
      }
    }
  }
  if (C > 1) cluster_wait();
}

template <typename X, int EPT>
cudaError_t run_softmax(const SoftmaxArgs& a, int C, cudaStream_t s) {
  static thread_local int allowed = -1;
  if (C > 8) {                                // clusters of 16 are opt-in, a function and device
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess && allowed != dev) {
      e = cudaFuncSetAttribute(softmax_kernel<X, EPT>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
      allowed = dev;
    }
    if (e != cudaSuccess) return e;
  }
  const int len = (a.V + C - 1) / C;
  int nt = EPT ? (len + EPT - 1) / EPT : MAX_NT;
  nt = (nt + 31) / 32 * 32;
  return launch_step(softmax_kernel<X, EPT>, dim3((unsigned)a.rows * C), nt, 0, s, C, a, C, len);
}

template <typename X>
cudaError_t softmax_x(const SoftmaxArgs& a, cudaStream_t s) {
  if (a.V <= 4096) return run_softmax<X, 8>(a, 1, s);
  int C = 1;
  while (C < MAX_C && (int64_t)C * MAX_NT * 32 < a.V) C *= 2;
  if ((int64_t)C * MAX_NT * 32 >= a.V) return run_softmax<X, 32>(a, C, s);
  return run_softmax<X, 0>(a, MAX_C, s);
}

// ------------------------------------------------------------------ verify --

// A weight in whole units of 2^-42, clamped to 0..1; NaN counts as 0.
__device__ __forceinline__ long long units(float w) {
  w = fminf(fmaxf(w, 0.0f), 1.0f);        // fmaxf(NaN, 0) = 0
  return __float2ll_rz(w * 4398046511104.0f);
}

__device__ __forceinline__ long long warp_sum(long long v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(~0u, v, o);
  return v;
}

// The sum of the entries before this lane's.
__device__ __forceinline__ long long warp_before(long long v) {
  long long s = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long u = __shfl_up_sync(~0u, s, o);
    if ((int)(threadIdx.x & 31) >= o) s += u;
  }
  return s - v;
}

// A chunk: 256 neighbouring ids, eight a lane (chunk + 32 j + lane), as units.
// q: the draft's row, or null; hot: the id whose q is 1 where the drafter was sure.
constexpr int CHUNK = 256;
__device__ __forceinline__ void load_chunk(const float* p, const float* q, int hot, int at, int V, long long (&u)[8]) {
  const int lane = threadIdx.x & 31;
  float x[8], y[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const int v = at + 32 * j + lane;
    x[j] = v < V ? p[v] : 0.0f;
    y[j] = q && v < V ? q[v] : 0.0f;
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const int v = at + 32 * j + lane;
    u[j] = units(x[j] - (v == hot ? 1.0f : y[j]));
  }
}

// A cluster of C CTAs a sequence; warps own `per` consecutive chunks each and
// keep every chunk's sum, so that after the total is known one warp re-reads the
// one chunk in which the running sum passes the threshold.
constexpr int MAX_PER = 32;
static_assert((int64_t)8 * (MAX_NT / 32) * MAX_PER * CHUNK >= 1 << 20, "a chunk sum for every id");
__global__ void __launch_bounds__(MAX_NT) verify_kernel(VerifyArgs a, int C, int per) {
  constexpr int NW = MAX_NT / 32;
  __shared__ long long chunk[NW][MAX_PER], wsum[NW], mine[2];
  __shared__ int s_acc;
  const int b = blockIdx.x / C, rank = blockIdx.x - b * C, V = a.V, S = a.S;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  pdl_begin();
  const int* draft = a.draft + (int64_t)b * S;
  const float us = a.us[b];
  int n = a.n_draft ? a.n_draft[b] : S;
  n = max(0, min(n, S));
  const float* p0 = a.p + (int64_t)b * (S + 1) * V;
  const float* q0 = a.q ? a.q + (int64_t)b * S * V : nullptr;
  // the first drafted token that does not stand
  if (threadIdx.x == 0) s_acc = n;
  __syncthreads();
  for (int i = threadIdx.x; i < n; i += MAX_NT) {
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
  const float* p = p0 + (int64_t)acc * V;
  const float* q = refused && q0 ? q0 + (int64_t)acc * V : nullptr;
  int hot = refused && !q0 ? draft[acc] : -1;
  const int first = (rank * NW + warp) * per;           // this warp's chunks
  long long total = 0, before = 0, own = 0;
  for (int pass = 0; pass < 2; ++pass) {
    long long w = 0;
    for (int i = 0; i < per; ++i) {
      const int at = (first + i) * CHUNK;
      if (at >= V) {
        if (lane == 0) chunk[warp][i] = 0;
        continue;
      }
      long long u[8], s = 0;
      load_chunk(p, q, hot, at, V, u);
#pragma unroll
      for (int j = 0; j < 8; ++j) s += u[j];
      s = warp_sum(s);
      if (lane == 0) chunk[warp][i] = s;
      w += s;
    }
    if (lane == 0) wsum[warp] = w;
    __syncthreads();
    own = warp_sum(lane < NW ? wsum[lane] : 0);
    before = 0;
    total = own;
    if (C > 1) {
      // a slot for each pass: nobody overwrites what another CTA still reads
      if (threadIdx.x == 0) mine[pass] = own;
      cluster_arrive();
      cluster_wait();
      const long long v = lane < C ? ld_cluster64(cluster_addr(&mine[pass], lane)) : 0;
      total = warp_sum(v);
      before = __shfl_sync(~0u, warp_before(v), rank);
    }
    if (total > 0 || !refused) break;
    q = nullptr, hot = -1;              // no mass is left: draw from p
    __syncthreads();                    // wsum is written again
  }
  if (C > 1) cluster_arrive();          // waited for at the end: the others still read `mine`
  int* out = a.tokens + (int64_t)b * (S + 1);
  if (rank == 0) {
    for (int i = threadIdx.x; i <= S; i += MAX_NT)
      if (i != acc || total == 0) out[i] = i < acc ? draft[i] : -1;
    if (threadIdx.x == 0) a.n_acc[b] = acc;
  }
  const unsigned long long U = (unsigned long long)fminf(fmaxf(us, 0.0f) * 2147483648.0f, 2147483520.0f);
  const unsigned long long T = (unsigned long long)total;
  const long long t = (long long)(((U * (T >> 32)) << 1) + ((U * (T & 0xffffffffull)) >> 31));
  if (total > 0 && t >= before && t < before + own) {
    // the warp, the chunk, the row of 32 and the id in which the sum passes t
    const long long wv = lane < NW ? wsum[lane] : 0, wb = before + warp_before(wv);
    const int tw = __ffs(__ballot_sync(~0u, t >= wb && t < wb + wv)) - 1;
    if (warp == tw) {
      long long run = __shfl_sync(~0u, wb, tw);
      int i = 0;
      while (run + chunk[warp][i] <= t) run += chunk[warp][i++];
      const int at = (first + i) * CHUNK;
      long long u[8];
      load_chunk(p, q, hot, at, V, u);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const long long lo = run + warp_before(u[j]);
        if (t >= lo && t < lo + u[j]) out[acc] = at + 32 * j + lane;
        run += warp_sum(u[j]);
      }
    }
  }
  if (C > 1) cluster_wait();
}

}  // namespace

cudaError_t launch_softmax(const SoftmaxArgs& a, cudaStream_t s) {
  switch (a.dtype) {
    case QMV_F32: return softmax_x<float>(a, s);
    case QMV_F16: return softmax_x<__half>(a, s);
    default: return softmax_x<__nv_bfloat16>(a, s);
  }
}

cudaError_t launch_verify(const VerifyArgs& a, cudaStream_t s) {
  constexpr int NW = MAX_NT / 32;
  const int chunks = (a.V + CHUNK - 1) / CHUNK;
  // CTAs a sequence: two chunks a warp, or eight CTAs and more chunks
  int C = 1;
  while (C < 8 && C * NW * 2 < chunks) C *= 2;
  const int per = (chunks + C * NW - 1) / (C * NW);
  return launch_step(verify_kernel, dim3((unsigned)a.B * C), MAX_NT, 0, s, C, a, C, per);
}

}  // namespace qmv
