// qmv_sample.cu -- logits to probabilities (qmv_softmax) and drafted tokens
// against the target's probabilities (qmv_verify_draft).
#include <math_constants.h>

#include <type_traits>

#include "qmv_pipe.cuh"
#include "qmv_step.cuh"

namespace qmv {

__device__ int g_sample_error = 0;

int read_sample_error(int clear, int* out) {
  cudaError_t e = cudaMemcpyFromSymbol(out, g_sample_error, sizeof(int));
  if (e == cudaSuccess && clear && *out) {
    const int z = 0;
    e = cudaMemcpyToSymbol(g_sample_error, &z, sizeof(int));
  }
  return (int)e;
}

namespace {

// The CTAs of a cluster tell each other one value: each stores its own into all
// of their shared memories, and each waits, on an mbarrier of its own, until all
// have come.  The one barrier that this needs (no store before the others have set
// theirs up) is arrived at when a kernel begins and waited for only here, so it
// costs nothing; and a CTA may end as soon as it has what it waited for, since
// only then does nobody store to it any more.  One whose wait ran out goes through
// exchange_leave first.  (Five rows of 262144, sixteen CTAs a row: 7.8 us, against
// 9.4 us with a cluster barrier before and after reading the others' shared memory.)
__device__ __forceinline__ void exchange_begin(uint64_t* bar, int bars, uint32_t bytes) {
  if (threadIdx.x == 0) {
    for (int i = 0; i < bars; ++i) {
      pipe::mbar_init(bar + i, 1);
      asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
      pipe::mbar_arrive_tx(bar + i, bytes);
    }
  }
  if (threadIdx.x < 32) {
    __syncwarp();
    cluster_arrive();
  } else {
    cluster_arrive_relaxed();
  }
}

// The end of a warp whose wait ran out: the others may still store to this CTA, so it
// stays until each of them has ended or come here too (each has stored by then, and its
// own wait is bounded), and until what they sent has landed.
__device__ __noinline__ void exchange_leave(uint64_t* bar, int bars) {
  __syncwarp();
  cluster_arrive();
  cluster_wait();
  for (int i = 0; i < bars; ++i) pipe::mbar_drain(bar + i, 0, &g_sample_error);
}

constexpr int MAX_NT = 512, MAX_C = 16;

// ----------------------------------------------------------------- softmax --

// What a warp, a CTA or a cluster knows of its part of a row: 16 bytes, stored whole
// into another CTA's shared memory.
struct alignas(16) Part {
  float m, s;      // maximum; sum of exp((x - m) / T), in the one-hot form of 0 * x (NaN marks the row)
  int at;          // first place of the maximum (in the one-hot form only)
  int unused;
};
static_assert(sizeof(Part) == 16 && alignof(Part) == 16, "one 16-byte store");

// 2^v to 2 units in the last place; results below 2^-126 become 0.
__device__ __forceinline__ float ex2(float v) {
  float d;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(d) : "f"(v));
  return d;
}

// The parts of a warp's first W lanes (a power of two) as one, in each of them;
// parts of nothing but -inf have the sum 0, or NaN where there was one.
__device__ __forceinline__ Part join(Part p, int W, float c, bool hot) {
  Part all = p;
  for (int o = W >> 1; o; o >>= 1) {
    const float m2 = __shfl_xor_sync(~0u, all.m, o);
    if (hot) {
      const int a2 = __shfl_xor_sync(~0u, all.at, o);
      if (m2 > all.m || (m2 == all.m && a2 < all.at)) all.at = a2;
    }
    all.m = fmaxf(all.m, m2);
  }
  all.s = hot || p.m == -CUDART_INF_F ? p.s : p.s * ex2((p.m - all.m) * c);
  for (int o = W >> 1; o; o >>= 1) all.s += __shfl_xor_sync(~0u, all.s, o);
  return all;
}

// Four neighbouring elements, aligned to themselves, as they are stored and as fp32.
template <typename X>
struct Four {
  typename std::conditional<sizeof(X) == 4, float4, uint2>::type w;
  __device__ __forceinline__ void none() {                   // all -inf
    constexpr uint32_t P = std::is_same<X, float>::value ? 0xFF800000u : std::is_same<X, __half>::value ? 0xFC00FC00u : 0xFF80FF80u;
    const uint32_t v[4] = {P, P, P, P};
    memcpy(&w, v, sizeof(w));
  }
  __device__ __forceinline__ void values(float (&v)[4]) const {
    X h[4];
    memcpy(h, &w, sizeof(w));
#pragma unroll
    for (int k = 0; k < 4; ++k) v[k] = to_f<X>(h[k]);
  }
};

// A CTA's part of a row (EPT > 0): `wholes` aligned fours inside the row, the first
// at element e0, and what sticks out of the fours at the row's two ends, elements
// e1 .. e1 + 3 as far as they are in the row: thread 0's and thread 1's extra four.
template <typename X>
struct Place {
  const X* x;
  float* out;
  int e0, wholes, e1;
  bool extra;
  __device__ __forceinline__ Place(const SoftmaxArgs& a, int row, int f0, int len, bool fours) {
    x = (const X*)a.x + (int64_t)row * a.ldx;
    out = a.out + (int64_t)row * a.ldo;
    if (!fours) return;
    const int shift = (int)((uintptr_t)x / sizeof(X) % 4);
    const int n = max(0, min(len, (a.V + shift + 3) / 4 - f0)), skip = f0 == 0 && shift ? 1 : 0;
    wholes = max(0, min(n, (a.V + shift) / 4 - f0) - skip);
    e0 = 4 * (f0 + skip) - shift;
    const bool behind = skip + wholes < n;
    extra = (threadIdx.x == 0 && skip && n > 0) || (threadIdx.x == 1 && behind);
    e1 = threadIdx.x == 0 ? -shift : 4 * (f0 + n - 1) - shift;
  }
};

// A cluster of C CTAs a row (C = 1: no cluster).  EPT > 0: a CTA's
// part of the row stays in registers, EPT elements a thread, so that the row is
// read once.  A row is taken in fours that are aligned in memory, wherever it
// begins (an odd V shifts every row; logits and out are shifted alike), `len` of
// them a CTA; all loads of a thread are on their way before the first value is
// used.
// EPT == 0: rows of any length and alignment, `len` elements a CTA, read a second
// and third time (from L2).
// exp((x - m) / T) is taken as 2^((x - m) * c), c = log2(e) / T.  A row with
// NaN or +inf has the sum NaN, which reaches every place by itself.
template <typename X, int EPT, int NT>
__global__ void __launch_bounds__(NT, 1024 / NT) softmax_kernel(SoftmaxArgs a, int C, int len) {
  constexpr int NW = NT / 32, R = EPT ? EPT / 4 : 1;
  __shared__ Part warps[NW], parts[MAX_C];
  __shared__ uint64_t all_here;
  __shared__ int abort_flag;
  const int rank = blockIdx.x % C, tid = threadIdx.x, lane = tid & 31, V = a.V, f0 = rank * len;
  const int row = blockIdx.x / C;
  const Place<X> at(a, row, f0, len, EPT > 0);
  if (C > 1) {
    if (tid == 0) abort_flag = 0;
    exchange_begin(&all_here, 1, C * sizeof(Part));
  }
  Four<X> w[R];                                // the row as it is stored
  X we[4];
  pdl_begin();
  if (EPT) {
#pragma unroll
    for (int j = 0; j < R; ++j) {
      w[j].none();
      if (j * NT + tid < at.wholes) w[j].w = reinterpret_cast<const decltype(w[j].w)*>(at.x + at.e0)[j * NT + tid];
    }
    if (at.extra) {
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if ((unsigned)(at.e1 + k) < (unsigned)V) we[k] = at.x[at.e1 + k];
    }
  }
  const float t = a.t ? a.t[row] : a.t0;
  const bool hot = !(t > 0.0f);
  // kept finite and above 0, so that 0 * c = 0 and -inf * c = -inf at any T
  const float c = fminf(fmaxf(1.4426950408889634f / t, 1e-37f), 1e38f);
  const int n0 = max(0, min(len, V - f0));                 // EPT == 0: elements
  float e[R][4], ee[4] = {-CUDART_INF_F, -CUDART_INF_F, -CUDART_INF_F, -CUDART_INF_F};
  Part p{-CUDART_INF_F, 0.0f, V, 0};
  if (EPT) {
#pragma unroll
    for (int j = 0; j < R; ++j) {
      w[j].values(e[j]);
      p.m = fmaxf(p.m, fmaxf(fmaxf(e[j][0], e[j][1]), fmaxf(e[j][2], e[j][3])));
    }
    if (at.extra) {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if ((unsigned)(at.e1 + k) < (unsigned)V) ee[k] = to_f<X>(we[k]);
        p.m = fmaxf(p.m, ee[k]);
      }
    }
    if (hot) {
      const auto note = [&](const float (&v)[4], int e0) {
#pragma unroll
        for (int k = 3; k >= 0; --k) {
          if (v[k] == p.m) p.at = min(p.at, e0 + k);
          if (!(v[k] < CUDART_INF_F)) p.s = CUDART_NAN_F;
        }
      };
#pragma unroll
      for (int j = 0; j < R; ++j)
        if (j * NT + tid < at.wholes) note(e[j], at.e0 + 4 * (j * NT + tid));
      if (at.extra) note(ee, at.e1);
    }
  } else {
    for (int i = tid; i < n0; i += NT) {
      const float v = to_f<X>(at.x[f0 + i]);
      if (v > p.m) p.m = v, p.at = f0 + i;
      if (hot && !(v < CUDART_INF_F)) p.s = CUDART_NAN_F;
    }
  }
  // the warp's maximum; its terms are relative to it
  {
    const float own = p.m;
#pragma unroll
    for (int o = 16; o; o >>= 1) p.m = fmaxf(p.m, __shfl_xor_sync(~0u, p.m, o));
    if (hot) {
      if (own != p.m) p.at = V;
#pragma unroll
      for (int o = 16; o; o >>= 1) p.at = min(p.at, __shfl_xor_sync(~0u, p.at, o));
    }
  }
  // nothing but -inf so far: any finite maximum will do, every term is 0
  const float m = p.m == -CUDART_INF_F ? 0.0f : p.m;
  if (!hot) {
    if (EPT) {
#pragma unroll
      for (int j = 0; j < R; ++j)
        if (j * NT < at.wholes) {            // the same for all threads
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            e[j][k] = ex2((e[j][k] - m) * c);
            p.s += e[j][k];
          }
        }
      if (at.extra) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          ee[k] = ex2((ee[k] - m) * c);
          p.s += ee[k];
        }
      }
    } else {
      for (int i = tid; i < n0; i += NT) p.s += ex2((to_f<X>(at.x[f0 + i]) - m) * c);
    }
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) p.s += __shfl_xor_sync(~0u, p.s, o);
  if (lane == 0) warps[tid >> 5] = p;
  __syncthreads();
  Part all;
  if (C == 1) {
    all = join(warps[lane & (NW - 1)], NW, c, hot);
  } else {
    cluster_wait();                          // all have begun
    if (tid < 32) {
      const Part q = join(warps[lane & (NW - 1)], NW, c, hot);
      if (lane < C)
        st_async128(cluster_addr(&parts[rank], lane), cluster_addr(&all_here, lane), __float_as_uint(q.m),
                    __float_as_uint(q.s), (uint32_t)q.at, 0u);
    }
    const bool came = pipe::mbar_wait_fast(&all_here, 0, &abort_flag, pipe::ERR_TIMEOUT_FULL, &g_sample_error);
    if (!__all_sync(~0u, came)) return exchange_leave(&all_here, 1);
    all = join(parts[lane & (C - 1)], C, c, hot);
  }
  // special rows, the one-hot form and rows of nothing but -inf (or NaN), have one
  // value at all.at and another elsewhere; f is at most 1 over the sum, and NaN or
  // finite where this warp had only -inf, whose terms are 0
  const bool special = hot || all.m == -CUDART_INF_F;
  const float rest = isnan(all.s) ? all.s : 0.0f, one = all.m == -CUDART_INF_F ? rest : 1.0f + rest;
  const float f = p.m == -CUDART_INF_F ? rest : ex2((p.m - all.m) * c) / all.s;
  if (EPT) {
    float4* to = reinterpret_cast<float4*>(at.out + at.e0);
    const auto value = [&](int el) { return el == all.at ? one : rest; };
    if (special) {
      for (int i = tid; i < at.wholes; i += NT) {
        const int el = at.e0 + 4 * i;
        to[i] = make_float4(value(el), value(el + 1), value(el + 2), value(el + 3));
      }
    } else {
#pragma unroll
      for (int j = 0; j < R; ++j)
        if (j * NT < at.wholes) {            // the same for all threads
          const float4 q = make_float4(e[j][0] * f, e[j][1] * f, e[j][2] * f, e[j][3] * f);
          if (j * NT + tid < at.wholes) to[j * NT + tid] = q;
        }
    }
    if (at.extra) {
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if ((unsigned)(at.e1 + k) < (unsigned)V) at.out[at.e1 + k] = special ? value(at.e1 + k) : ee[k] * f;
    }
  } else {
    for (int i = tid; i < n0; i += NT)
      at.out[f0 + i] = special ? (f0 + i == all.at ? one : rest) : ex2((to_f<X>(at.x[f0 + i]) - all.m) * c) / all.s;
  }
}

template <typename X, int EPT, int NT>
cudaError_t run_softmax(const SoftmaxArgs& a, int parts, int C, cudaStream_t s) {
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
  return launch_step(softmax_kernel<X, EPT, NT>, dim3((unsigned)a.rows * C), NT, 0, s, C, a, C, (parts - 1) / C + 1);
}

// Many rows that fit twice into a CTA's shared memory: a CTA a streaming multiprocessor
// stays for the whole launch and takes whole rows, the next one on its way while one is
// worked on, so that HBM is read while exponentials are formed and nobody waits for
// another CTA.  A row's 16-byte words come by bulk copies; what sticks out of them at
// its two ends, less than 2 * E elements, lies in registers of the first threads.  Against
// a cluster a row (fp16): 384 rows of 50257 26.3 for 32.7 us, 1000 rows 56.7 for 78.4 (78 % of
// the measured copy rate); fp32, 600 rows of 27001: 26.1 for 28.7.  Each row costs two
// waits of a whole CTA, so rows that one CTA of the other kernel holds stay there (1500
// rows of 16001 in fp16: 29.6 for 41.5).
constexpr int A_NT = 1024;
template <typename X>
__global__ void __launch_bounds__(A_NT, 1) softmax_ahead_kernel(SoftmaxArgs a, int pitch) {
  constexpr int E = 16 / sizeof(X), NW = A_NT / 32;
  extern __shared__ __align__(128) uint8_t rows_smem[];
  __shared__ uint64_t full[2];
  __shared__ Part warps[2][NW];
  __shared__ int abort_flag;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, V = a.V, step = gridDim.x;
  if (tid == 0) {
    abort_flag = 0;
    for (int i = 0; i < 2; ++i) pipe::mbar_init(full + i, 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  __syncthreads();
  pdl_begin();
  const auto row_at = [&](int row) { return (const X*)a.x + (int64_t)row * a.ldx; };
  // the row's elements before its first aligned word
  const auto lead = [&](const X* x) { return (int)((uintptr_t)(-(intptr_t)x) / sizeof(X) % E); };
  // its first word's place in a line of 128 bytes, the same in shared memory
  const auto off_of = [](const X* x) { return (int)((uintptr_t)x / 16 % 8); };
  // by the first warp: a row's words to a buffer, in 32 copies
  const auto fetch = [&](int row, int buf) {
    const X* x = row_at(row);
    const int e0 = lead(x), words = (V - e0) / E, off = off_of(x + e0), share = ((off + words + 31) / 32 + 7) & ~7;
    if (lane == 0) pipe::mbar_arrive_tx(full + buf, words * 16);
    __syncwarp();
    const int w0 = max(0, lane * share - off), n = min((lane + 1) * share - off, words) - w0;
    if (n > 0)
      asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                       pipe::sa(rows_smem + (size_t)buf * pitch + (off + w0) * 16)),
                   "l"(x + e0 + w0 * E), "r"(n * 16), "r"(pipe::sa(full + buf))
                   : "memory");
  };
  // the element at an end that is this thread's, or V
  const auto end_of = [&](const X* x) {
    const int e0 = lead(x), behind = e0 + (V - e0) / E * E;
    return tid < E ? (tid < e0 ? tid : V) : tid < 2 * E ? min(behind + tid - E, V) : V;
  };
  const X none = from_f<X>(-CUDART_INF_F);
  X edge = none;
  int row = blockIdx.x;
  if (warp == 0) {
    fetch(row, 0);
    const int i = end_of(row_at(row));
    if (i < V) edge = row_at(row)[i];
  }
  float t_next = a.t ? a.t[row] : a.t0;
  for (int it = 0; row < a.rows; ++it, row += step) {
    const int buf = it & 1;
    const X* x = row_at(row);
    float* out = a.out + (int64_t)row * a.ldo;
    const int e0 = lead(x), fours = (V - e0) / E * (E / 4), ei = end_of(x);
    const float ev = to_f<X>(edge), t = t_next;
    const bool hot = !(t > 0.0f);
    const float c = fminf(fmaxf(1.4426950408889634f / t, 1e-37f), 1e38f);
    if (it == 0 && warp == 0 && row + step < a.rows) fetch(row + step, 1);
    if (row + step < a.rows) {
      if (a.t) t_next = a.t[row + step];
      if (warp == 0) {
        const int i = end_of(row_at(row + step));
        edge = i < V ? row_at(row + step)[i] : none;
      }
    }
    bool dead = !pipe::mbar_wait_fast(full + buf, (it >> 1) & 1, &abort_flag, pipe::ERR_TIMEOUT_FULL, &g_sample_error);
    const uint8_t* in = rows_smem + (size_t)buf * pitch + off_of(x + e0) * 16;
    const auto take = [&](int i, float (&v)[4]) {
      Four<X> f;
      f.w = reinterpret_cast<const decltype(f.w)*>(in)[i];
      f.values(v);
    };
    Part p{ev, 0.0f, V, 0};
    if (!(ev > -CUDART_INF_F)) p.m = -CUDART_INF_F;          // NaN too
#pragma unroll 4
    for (int i = tid; i < fours; i += A_NT) {
      float v[4];
      take(i, v);
      p.m = fmaxf(p.m, fmaxf(fmaxf(v[0], v[1]), fmaxf(v[2], v[3])));
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) p.m = fmaxf(p.m, __shfl_xor_sync(~0u, p.m, o));
    const float m = p.m == -CUDART_INF_F ? 0.0f : p.m;
    if (hot) {
      const auto note = [&](float v, int el) {
        if (v == p.m) p.at = min(p.at, el);
        if (!(v < CUDART_INF_F)) p.s = CUDART_NAN_F;
      };
      if (ei < V) note(ev, ei);
      for (int i = tid; i < fours; i += A_NT) {
        float v[4];
        take(i, v);
#pragma unroll
        for (int k = 0; k < 4; ++k) note(v[k], e0 + 4 * i + k);
      }
#pragma unroll
      for (int o = 16; o; o >>= 1) p.at = min(p.at, __shfl_xor_sync(~0u, p.at, o));
    } else {
      p.s = ex2((ev - m) * c);
#pragma unroll 4
      for (int i = tid; i < fours; i += A_NT) {
        float v[4];
        take(i, v);
        p.s += (ex2((v[0] - m) * c) + ex2((v[1] - m) * c)) + (ex2((v[2] - m) * c) + ex2((v[3] - m) * c));
      }
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) p.s += __shfl_xor_sync(~0u, p.s, o);
    if (lane == 0) warps[buf][warp] = p;
    // also: every thread is done with the row before, whose buffer is filled again
    if (__syncthreads_or(dead)) {
      // a copy that did not come: nothing more is stored, and what is in flight lands
      if (tid == 0) {
        pipe::mbar_drain(full + buf, (it >> 1) & 1, &g_sample_error);
        if (it == 0 && row + step < a.rows) pipe::mbar_drain(full + 1, 0, &g_sample_error);
      }
      return;
    }
    if (it > 0 && warp == 0 && row + step < a.rows) fetch(row + step, buf ^ 1);
    const Part all = join(warps[buf][lane], NW, c, hot);
    const float rest = isnan(all.s) ? all.s : 0.0f, one = all.m == -CUDART_INF_F ? rest : 1.0f + rest;
    float4* to = reinterpret_cast<float4*>(out + e0);
    if (hot || all.m == -CUDART_INF_F) {
      const auto value = [&](int el) { return el == all.at ? one : rest; };
      for (int i = tid; i < fours; i += A_NT) {
        const int el = e0 + 4 * i;
        to[i] = make_float4(value(el), value(el + 1), value(el + 2), value(el + 3));
      }
      if (ei < V) out[ei] = value(ei);
    } else {
      const float f = 1.0f / all.s;
#pragma unroll 4
      for (int i = tid; i < fours; i += A_NT) {
        float v[4];
        take(i, v);
        to[i] = make_float4(ex2((v[0] - all.m) * c) * f, ex2((v[1] - all.m) * c) * f, ex2((v[2] - all.m) * c) * f,
                            ex2((v[3] - all.m) * c) * f);
      }
      if (ei < V) out[ei] = ex2((ev - all.m) * c) * f;
    }
  }
}

template <typename X>
cudaError_t run_ahead(const SoftmaxArgs& a, int pitch, cudaStream_t s) {
  static thread_local KernCache c;
  const cudaError_t e = prep_kernel(softmax_ahead_kernel<X>, c, A_NT, 2 * (size_t)pitch, nullptr);
  if (e != cudaSuccess) return e;
  const int sms = dev_info().sms;
  return launch_step(softmax_ahead_kernel<X>, dim3(a.rows < sms ? a.rows : sms), A_NT, 2 * (size_t)pitch, s, 1, a, pitch);
}

template <typename X>
cudaError_t softmax_x(const SoftmaxArgs& a, cudaStream_t s) {
  // every row of logits and of out begins at the same place of an aligned four
  const int sx = (int)((uintptr_t)a.x / sizeof(X) % 4), so = (int)((uintptr_t)a.out / 4 % 4);
  const bool alike = (a.rows == 1 || a.ldx % 4 == a.ldo % 4) && sx == so;
  const bool even = (a.rows == 1 || a.ldx % 4 == 0) && sx == 0;
  const int fours = (int)(((int64_t)a.V + (even ? 0 : 3) + 3) / 4);   // of a row, at most
  if (alike) {
    if (fours <= 128 * 2) return run_softmax<X, 8, 128>(a, fours, 1, s);
    if (fours <= MAX_NT * 2) return run_softmax<X, 8, MAX_NT>(a, fours, 1, s);
    // rows of more than one CTA's registers, two or more a streaming multiprocessor; a row
    // begins in shared memory where it does in a line of 128 bytes
    const int64_t pitch = ((int64_t)a.V * sizeof(X) + 255) / 128 * 128;
    if (fours > MAX_NT * 8 && a.rows >= 2 * dev_info().sms && 2 * pitch <= dev_info().max_smem_optin - 4096)
      return run_ahead<X>(a, (int)pitch, s);
    int C = 1;
    while (C < MAX_C && C * MAX_NT * 8 < fours) C *= 2;
    if (C * MAX_NT * 8 >= fours) return run_softmax<X, 32, MAX_NT>(a, fours, C, s);
  }
  int C = 1;                                  // 32 elements a thread, or 16 CTAs and more
  while (C < MAX_C && (int64_t)C * MAX_NT * 32 < a.V) C *= 2;
  return run_softmax<X, 0, MAX_NT>(a, a.V, C, s);
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

// A chunk: 256 neighbouring ids, eight a lane.  VEC (rows that begin aligned to 16
// bytes, V a multiple of 4): two fours, 128 h + 4 lane + k; otherwise 32 j + lane.
constexpr int CHUNK = 256;
template <bool VEC>
struct Chunk {
  float x[8], y[8];
  static __device__ __forceinline__ int id(int j) {
    const int lane = threadIdx.x & 31;
    return VEC ? 128 * (j >> 2) + 4 * lane + (j & 3) : 32 * j + lane;
  }
  __device__ __forceinline__ void load(const float* p, const float* q, int at, int V) {
    if (VEC) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int v = at + id(4 * h);
        float4 a = make_float4(0, 0, 0, 0), b = a;
        if (v < V) {
          a = *reinterpret_cast<const float4*>(p + v);
          if (q) b = *reinterpret_cast<const float4*>(q + v);
        }
        x[4 * h] = a.x, x[4 * h + 1] = a.y, x[4 * h + 2] = a.z, x[4 * h + 3] = a.w;
        y[4 * h] = b.x, y[4 * h + 1] = b.y, y[4 * h + 2] = b.z, y[4 * h + 3] = b.w;
      }
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int v = at + id(j);
        x[j] = v < V ? p[v] : 0.0f;
        y[j] = q && v < V ? q[v] : 0.0f;
      }
    }
  }
  // hot: the id whose q is 1 where the drafter was sure, relative to the chunk
  __device__ __forceinline__ void sure(int hot) {
    if ((unsigned)hot < (unsigned)CHUNK) {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (id(j) == hot) y[j] = 1.0f;
    }
  }
  __device__ __forceinline__ long long sum() const {
    uint32_t h = 0, l = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      uint32_t hi, lo;
      units(x[j] - y[j], hi, lo);
      h += hi;
      l += lo;
    }
    // at most 2^21 a weight, 2^29 a chunk
    return whole(__reduce_add_sync(~0u, h - 8 * BIAS), __reduce_add_sync(~0u, l - 8 * BIAS));
  }
  // The id (relative to the chunk) in which the running sum passes t, from `run`
  // before the chunk, in the one lane that has it; -1 in the others.
  __device__ __forceinline__ int find(long long run, long long t) const {
    int found = -1;
#pragma unroll
    for (int g = 0; g < (VEC ? 2 : 8); ++g) {
      constexpr int N = VEC ? 4 : 1;             // neighbours a lane
      long long u[N], s = 0;
#pragma unroll
      for (int k = 0; k < N; ++k) {
        uint32_t hi, lo;
        units(x[g * N + k] - y[g * N + k], hi, lo);
        u[k] = whole(hi - BIAS, lo - BIAS);
        s += u[k];
      }
      long long b = run + warp_before(s);
#pragma unroll
      for (int k = 0; k < N; ++k) {
        if (t >= b && t < b + u[k]) found = id(g * N + k);
        b += u[k];
      }
      run += warp_sum(s);
    }
    return found;
  }
};

// A cluster of C CTAs a sequence; warps own `per` consecutive chunks each and
// keep every chunk's sum, so that after the total is known one warp re-reads the
// one chunk in which the running sum passes the threshold.  Bound by HBM: one row
// of p and one of q a sequence; small CTAs, so that all sequences run at once, and
// loads well ahead (48 sequences over 262144 ids, 100 MB: 22.3 us with 512 threads
// and one chunk ahead, 19.6 us with 256, 17.1 us with two chunks ahead).
constexpr int V_NT = 256, V_NW = V_NT / 32, MAX_PER = 64;
static_assert((int64_t)8 * V_NW * MAX_PER * CHUNK >= 1 << 20, "a chunk sum for every id");
template <bool VEC>
__global__ void __launch_bounds__(V_NT, 3) verify_kernel(VerifyArgs a, int C, int per) {
  constexpr int NW = V_NW;
  __shared__ long long chunk[NW][MAX_PER], wsum[NW], parts[2][MAX_C];
  __shared__ uint64_t all_here[2];
  __shared__ int s_acc, abort_flag, s_dead;
  const int b = blockIdx.x / C, rank = blockIdx.x - b * C, V = a.V, S = a.S;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) abort_flag = s_dead = 0;
  if (C > 1) exchange_begin(all_here, 2, C * sizeof(long long));
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
  if (hot >= V) hot = -1;
  hot = max(hot, -1);
  const int first = (rank * NW + warp) * per;           // this warp's chunks
  long long total = 0, before = 0, own = 0;
  for (int pass = 0; pass < 2; ++pass) {
    long long w = 0;
    const int last = min(per, max(0, (V + CHUNK - 1) / CHUNK - first));
    Chunk<VEC> c[3];                      // two on their way while one is summed
#pragma unroll
    for (int j = 0; j < 2; ++j)
      if (j < last) c[j].load(p, q, (first + j) * CHUNK, V);
    for (int i0 = 0; i0 < last; i0 += 3) {
#pragma unroll
      for (int j = 0; j < 3; ++j) {
        const int i = i0 + j;
        if (i >= last) break;
        if (i + 2 < last) c[(j + 2) % 3].load(p, q, (first + i + 2) * CHUNK, V);
        c[j].sure(hot - (first + i) * CHUNK);
        const long long s = c[j].sum();
        if (lane == 0) chunk[warp][i] = s;
        w += s;
      }
    }
    if (lane == 0) wsum[warp] = w;
    __syncthreads();
    own = warp_sum(lane < NW ? wsum[lane] : 0);
    before = 0;
    total = own;
    if (C > 1) {
      // a barrier and a place for each pass
      if (pass == 0) cluster_wait();      // all have begun
      if (warp == 0) {
        if (lane < C) st_async64(cluster_addr(&parts[pass][rank], lane), cluster_addr(&all_here[pass], lane), own);
        const bool came = pipe::mbar_wait_fast(&all_here[pass], 0, &abort_flag, pipe::ERR_TIMEOUT_FULL, &g_sample_error);
        if (!came) s_dead = 1;
      }
      __syncthreads();
      if (s_dead) return exchange_leave(all_here, 2);       // the same for all threads
      const long long v = lane < C ? parts[pass][lane] : 0;
      total = warp_sum(v);
      before = __shfl_sync(~0u, warp_before(v), rank);
    }
    if (total > 0 || !refused) break;
    q = nullptr, hot = -1;              // no mass is left: draw from p
    __syncthreads();                    // wsum is written again
  }
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
      Chunk<VEC> c;
      c.load(p, q, at, V);
      c.sure(hot - at);
      const int id = c.find(run, t);
      if (id >= 0) out[acc] = at + id;
    }
  }
}

}  // namespace

cudaError_t launch_softmax(const SoftmaxArgs& a, cudaStream_t s) {
  switch (a.dtype) {
    case QMV_F32: return softmax_x<float>(a, s);
    case QMV_F16: return softmax_x<__half>(a, s);
    default: return softmax_x<__nv_bfloat16>(a, s);
  }
}

template <bool VEC>
static cudaError_t run_verify(const VerifyArgs& a, cudaStream_t s) {
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
      e = cudaFuncSetAttribute(verify_kernel<VEC>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
      allowed = dev;
    }
    if (e != cudaSuccess) return e;
    C = 16;
  }
  const int per = (chunks + C * V_NW - 1) / (C * V_NW);
  return launch_step(verify_kernel<VEC>, dim3((unsigned)a.B * C), V_NT, 0, s, C, a, C, per);
}

cudaError_t launch_verify(const VerifyArgs& a, cudaStream_t s) {
  const bool vec = a.V % 4 == 0 && (uintptr_t)a.p % 16 == 0 && (uintptr_t)a.q % 16 == 0;
  return vec ? run_verify<true>(a, s) : run_verify<false>(a, s);
}

}  // namespace qmv
