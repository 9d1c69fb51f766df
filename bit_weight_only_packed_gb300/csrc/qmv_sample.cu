// qmv_sample.cu -- logits to probabilities (qmv_softmax) and drafted tokens
// against the target's probabilities (qmv_verify_draft).
#include <math_constants.h>

#include "qmv_step.cuh"

namespace qmv {
namespace {

constexpr int MAX_NT = 512, MAX_C = 16;

// ----------------------------------------------------------------- softmax --

// The largest value of a CTA, and the first place of it (asked for by `place`).
__device__ __forceinline__ void block_max(float& m, int& at, bool place, float* red, int* redi) {
  const int lane = threadIdx.x & 31, nw = blockDim.x >> 5;
#pragma unroll
  for (int pass = 0; pass < 2; ++pass) {
#pragma unroll
    for (int o = 16; o; o >>= 1) {
      const float m2 = __shfl_xor_sync(~0u, m, o);
      if (place) {
        const int a2 = __shfl_xor_sync(~0u, at, o);
        if (m2 > m || (m2 == m && a2 < at)) at = a2;
      }
      m = fmaxf(m, m2);
    }
    if (pass) break;
    if (lane == 0) red[threadIdx.x >> 5] = m, redi[threadIdx.x >> 5] = at;
    __syncthreads();
    m = red[lane < nw ? lane : 0];
    at = redi[lane < nw ? lane : 0];
  }
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

// 2^v to 2 units in the last place; results below 2^-126 become 0.
__device__ __forceinline__ float ex2(float v) {
  float d;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(d) : "f"(v));
  return d;
}

// What a CTA knows of its part of a row.
struct Part {
  float m, s;      // maximum; sum of exp((x - m) / T), in the one-hot form of 0 * x (NaN marks the row)
  int at;          // first place of the maximum
};

// A cluster of C CTAs a row (C = 1: no cluster).  EPT > 0: a CTA's part of the
// row stays in registers, EPT elements a thread, so that the row is read once;
// EPT == 0: a part of any length, read a second and third time (from L2).
// exp((x - m) / T) is taken as exp2((x - m) * c), c = log2(e) / T.  A row with
// NaN or +inf has the sum NaN, which reaches every place by itself.
template <typename X, int EPT, int NT>
__global__ void __launch_bounds__(NT, 1024 / NT) softmax_kernel(SoftmaxArgs a, int C, int len) {
  __shared__ Part mine;
  __shared__ float redm[NT / 32], reds[NT / 32];
  __shared__ int redi[NT / 32];
  const int row = blockIdx.x / C, rank = blockIdx.x - row * C, tid = threadIdx.x;
  const int v0 = min(a.V, rank * len), n = min(a.V - v0, len);     // this CTA's part
  const X* x = (const X*)a.x + (int64_t)row * a.ldx + v0;
  float* out = a.out + (int64_t)row * a.ldo + v0;
  pdl_begin();
  const float t = a.t ? a.t[row] : a.t0;
  const bool hot = !(t > 0.0f);
  // kept finite and above 0, so that 0 * c = 0 and -inf * c = -inf at any T
  const float c = fminf(fmaxf(1.4426950408889634f / t, 1e-37f), 1e38f);
  constexpr int R = EPT ? EPT : 1;
  float e[R];
  Part p{-CUDART_INF_F, 0.0f, a.V};
  if (EPT) {
#pragma unroll
    for (int j = 0; j < R; ++j) e[j] = j * NT + tid < n ? to_f<X>(x[j * NT + tid]) : -CUDART_INF_F;
#pragma unroll
    for (int j = 0; j < R; ++j) p.m = fmaxf(p.m, e[j]);
    if (hot) {
#pragma unroll
      for (int j = R - 1; j >= 0; --j) {
        if (e[j] == p.m) p.at = v0 + j * NT + tid;
        if (!(e[j] < CUDART_INF_F)) p.s = CUDART_NAN_F;
      }
    }
  } else {
    for (int i = tid; i < n; i += NT) {
      const float v = to_f<X>(x[i]);
      if (v > p.m) p.m = v, p.at = v0 + i;
      if (hot && !(v < CUDART_INF_F)) p.s = CUDART_NAN_F;
    }
  }
  block_max(p.m, p.at, hot, redm, redi);
  // nothing but -inf so far: any finite maximum will do, every term is 0
  const float m = p.m == -CUDART_INF_F ? 0.0f : p.m;
  if (!hot) {
    if (EPT) {
#pragma unroll
      for (int j = 0; j < R; ++j) {
        e[j] = ex2((e[j] - m) * c);
        p.s += e[j];
      }
    } else {
      for (int i = tid; i < n; i += NT) p.s += ex2((to_f<X>(x[i]) - m) * c);
    }
  }
  p.s = block_sum(p.s, reds);
  Part all = p;
  if (C > 1) {
    const int lane = tid & 31;
    if (tid == 0) mine = p;
    if (tid < 32) {
      __syncwarp();
      cluster_arrive();
    } else {
      cluster_arrive_relaxed();
    }
    cluster_wait();
    const uint32_t at = cluster_addr(&mine, lane < C ? lane : 0);
    Part q;
    q.m = __uint_as_float(ld_cluster32(at));
    q.s = __uint_as_float(ld_cluster32(at + 4));
    q.at = (int)ld_cluster32(at + 8);
    all = q;
#pragma unroll
    for (int o = 16; o; o >>= 1) {
      const float m2 = __shfl_xor_sync(~0u, all.m, o);
      const int a2 = __shfl_xor_sync(~0u, all.at, o);
      if (m2 > all.m || (m2 == all.m && a2 < all.at)) all.at = a2;
      all.m = fmaxf(all.m, m2);
    }
    float sum = lane >= C || q.m == -CUDART_INF_F ? 0.0f : hot ? q.s : q.s * ex2((q.m - all.m) * c);
    // a part of NaN alone has the maximum -inf and the sum NaN
    if (lane < C && isnan(q.s)) sum = q.s;
#pragma unroll
    for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(~0u, sum, o);
    all.s = sum;
    cluster_arrive_relaxed();                // waited for at the end: the others still read `mine`
  }
  if (hot || all.m == -CUDART_INF_F) {       // the one-hot form, or nothing but -inf (or NaN)
    const float rest = isnan(all.s) ? all.s : 0.0f, one = all.m == -CUDART_INF_F ? rest : 1.0f + rest;
    for (int i = tid; i < n; i += NT) out[i] = v0 + i == all.at ? one : rest;
  } else {
    // at most 1 over the sum; 0 where this part had only -inf, whose terms are 0
    const float f = ex2((p.m - all.m) * c) / all.s;
    if (EPT) {
#pragma unroll
      for (int j = 0; j < R; ++j)
        if (j * NT + tid < n) out[j * NT + tid] = e[j] * f;
    } else {
      for (int i = tid; i < n; i += NT) out[i] = ex2((to_f<X>(x[i]) - all.m) * c) / all.s;
    }
  }
  if (C > 1) cluster_wait();
}

template <typename X, int EPT, int NT>
cudaError_t run_softmax(const SoftmaxArgs& a, int C, cudaStream_t s) {
  static thread_local int allowed = -1;
  if (C > 8) {                                // clusters of 16 are opt-in, a function and device
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess && allowed != dev) {
      e = cudaFuncSetAttribute(softmax_kernel<X, EPT, NT>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
      allowed = dev;
    }
    if (e != cudaSuccess) return e;
  }
  return launch_step(softmax_kernel<X, EPT, NT>, dim3((unsigned)a.rows * C), NT, 0, s, C, a, C, (a.V + C - 1) / C);
}

template <typename X>
cudaError_t softmax_x(const SoftmaxArgs& a, cudaStream_t s) {
  if (a.V <= 1024) return run_softmax<X, 8, 128>(a, 1, s);
  if (a.V <= 4096) return run_softmax<X, 8, 512>(a, 1, s);
  int C = 1;
  while (C < MAX_C && (int64_t)C * MAX_NT * 32 < a.V) C *= 2;
  if ((int64_t)C * MAX_NT * 32 >= a.V) return run_softmax<X, 32, MAX_NT>(a, C, s);
  return run_softmax<X, 0, MAX_NT>(a, MAX_C, s);
}

// ------------------------------------------------------------------ verify --

// A weight, clamped to 0..1 (NaN counts as 0), in whole units of 2^-42 as hi *
// 2^21 + lo.  Adding 2^23 while rounding towards 0 leaves the whole part of a
// number below 2^23 in the mantissa, so hi and lo come from four operations of
// the floating-point pipe; both are returned on top of the bits of 2^23, which
// the sums take off at the end (modulo 2^32).
constexpr uint32_t BIAS = 0x4B000000u;
__device__ __forceinline__ void units(float w, uint32_t& hi, uint32_t& lo) {
  w = fminf(fmaxf(w, 0.0f), 1.0f);        // fmaxf(NaN, 0) = 0
  const float h = __fmaf_rz(w, 2097152.0f, 8388608.0f);
  const float rem = __fmaf_rn(w, 2097152.0f, -(h - 8388608.0f));   // exact, below 1
  hi = __float_as_uint(h);
  lo = __float_as_uint(__fmaf_rz(rem, 2097152.0f, 8388608.0f));
}
__device__ __forceinline__ long long whole(uint32_t hi, uint32_t lo) { return ((long long)hi << 21) + lo; }

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

// A chunk: 256 neighbouring ids, eight a lane (chunk + 32 j + lane).
constexpr int CHUNK = 256;
struct Chunk {
  float x[8], y[8];
  __device__ __forceinline__ void load(const float* p, const float* q, int at, int V) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int v = at + 32 * j + lane;
      x[j] = v < V ? p[v] : 0.0f;
      y[j] = q && v < V ? q[v] : 0.0f;
    }
  }
  // hot: the id whose q is 1 where the drafter was sure
  __device__ __forceinline__ float weight(int j, int at, int hot) const {
    return x[j] - (at + 32 * j + (int)(threadIdx.x & 31) == hot ? 1.0f : y[j]);
  }
  __device__ __forceinline__ long long sum(int at, int hot) const {
    uint32_t h = 0, l = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      uint32_t hi, lo;
      units(weight(j, at, hot), hi, lo);
      h += hi;
      l += lo;
    }
    // at most 2^21 a weight, 2^29 a chunk
    return whole(__reduce_add_sync(~0u, h - 8 * BIAS), __reduce_add_sync(~0u, l - 8 * BIAS));
  }
};

// A cluster of C CTAs a sequence; warps own `per` consecutive chunks each and
// keep every chunk's sum, so that after the total is known one warp re-reads the
// one chunk in which the running sum passes the threshold.
constexpr int V_NT = 512, V_NW = V_NT / 32, MAX_PER = 32;
static_assert((int64_t)8 * V_NW * MAX_PER * CHUNK >= 1 << 20, "a chunk sum for every id");
__global__ void __launch_bounds__(V_NT, 2) verify_kernel(VerifyArgs a, int C, int per) {
  constexpr int NW = V_NW;
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
  for (int i = threadIdx.x; i < n; i += V_NT) {
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
    const int last = min(per, max(0, (V + CHUNK - 1) / CHUNK - first));
    Chunk c;
    if (last > 0) c.load(p, q, first * CHUNK, V);
    for (int i = 0; i < last; ++i) {
      Chunk next;                         // on its way while this one is summed
      if (i + 1 < last) next.load(p, q, (first + i + 1) * CHUNK, V);
      const long long s = c.sum((first + i) * CHUNK, hot);
      if (lane == 0) chunk[warp][i] = s;
      w += s;
      c = next;
    }
    if (lane == 0) wsum[warp] = w;
    __syncthreads();
    own = warp_sum(lane < NW ? wsum[lane] : 0);
    before = 0;
    total = own;
    if (C > 1) {
      // a slot for each pass: nobody overwrites what another CTA still reads
      if (threadIdx.x == 0) mine[pass] = own;
      if (warp == 0) {
        __syncwarp();
        cluster_arrive();
      } else {
        cluster_arrive_relaxed();
      }
      cluster_wait();
      const long long v = lane < C ? ld_cluster64(cluster_addr(&mine[pass], lane)) : 0;
      total = warp_sum(v);
      before = __shfl_sync(~0u, warp_before(v), rank);
    }
    if (total > 0 || !refused) break;
    q = nullptr, hot = -1;              // no mass is left: draw from p
    __syncthreads();                    // wsum is written again
  }
  if (C > 1) cluster_arrive_relaxed();  // waited for at the end: the others still read `mine`
  int* out = a.tokens + (int64_t)b * (S + 1);
  if (rank == 0) {
    for (int i = threadIdx.x; i <= S; i += V_NT)
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
      Chunk c;
      c.load(p, q, at, V);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        uint32_t hi, lo;
        units(c.weight(j, at, hot), hi, lo);
        const long long u = whole(hi - BIAS, lo - BIAS);
        const long long b0 = run + warp_before(u);
        if (t >= b0 && t < b0 + u) out[acc] = at + 32 * j + lane;
        run += warp_sum(u);
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
  const int chunks = (a.V + CHUNK - 1) / CHUNK;
  // CTAs a sequence: two chunks a warp or eight CTAs and more chunks; sixteen, which
  // are opt-in, where the sequences are too few to fill the device with eight
  int C = 1;
  while (C < 8 && C * V_NW * 2 < chunks) C *= 2;
  if (C == 8 && C * V_NW * 2 < chunks && (int64_t)a.B * 16 <= dev_info().sms) {
    static thread_local int allowed = -1;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess && allowed != dev) {
      e = cudaFuncSetAttribute(verify_kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
      allowed = dev;
    }
    if (e != cudaSuccess) return e;
    C = 16;
  }
  const int per = (chunks + C * V_NW - 1) / (C * V_NW);
  return launch_step(verify_kernel, dim3((unsigned)a.B * C), V_NT, 0, s, C, a, C, per);
}

}  // namespace qmv
