// qmv_experts.cu -- around the experts' products (qmv_experts.cuh): the pairs of token and expert in
// the order of experts, x in fp16 with the activation in front of it, and the weighted sum
// behind them.
#include <algorithm>

#include "qmv_experts.cuh"

namespace qmv {
namespace w4 {

extern template cudaError_t run_experts<32>(const ExpertsArgs&, const ExpertsPlan&, cudaStream_t);
extern template cudaError_t run_experts<64>(const ExpertsArgs&, const ExpertsPlan&, cudaStream_t);
extern template cudaError_t run_experts<128>(const ExpertsArgs&, const ExpertsPlan&, cudaStream_t);
extern template cudaError_t read_x_error<32>(int, int*);
extern template cudaError_t read_x_error<64>(int, int*);
extern template cudaError_t read_x_error<128>(int, int*);
// read_x_error<0>: this file's

}  // namespace w4

int read_experts_error(int clear, int* out) {
  cudaError_t (*const read[])(int, int*) = {w4::read_x_error<32>, w4::read_x_error<64>, w4::read_x_error<128>, w4::read_x_error<0>};
  *out = 0;
  for (const auto f : read) {
    int v = 0;
    const cudaError_t e = f(clear, &v);
    if (e != cudaSuccess) return (int)e;
    if (v) *out = v;
  }
  return 0;
}

namespace {

using namespace w4;

// The pairs in the order of their experts, pairs of one expert as they came, and the tasks.  Each of nw
// warps counts a contiguous part of the pairs in counters of its own, [warp][expert], which then become
// the places where it puts them.  EACH: experts a thread.
template <int EACH>
__device__ __forceinline__ void sort_each(const ExpertsArgs& a, int cols, int* head, int* order, Task* tasks, int* counts) {
  __shared__ int sums[X_W], t_sums[X_W];
  const int P = a.M * a.T, E1 = a.E + 1, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int nw = min(X_W, cdiv(P, 32)), per = cdiv(cdiv(P, nw), 32) * 32, p0 = min(P, warp * per), p1 = min(P, p0 + per);
  const auto expert_of = [&](int e) { return (unsigned)e < (unsigned)a.E ? e : a.E; };    // those without one come last
  // the first of a warp's ids, for both of its passes, is on its way meanwhile
  const int first = p0 + lane < p1 ? a.ids[p0 + lane] : -1;
  for (int i = tid; i < nw * E1; i += X_NT) counts[i] = 0;
  __syncthreads();
  for (int p = p0 + lane; p < p1; p += 32) {
    const int e = p < p0 + 32 ? first : a.ids[p];
    if (e < -1 || e >= a.E) atomicCAS(&g_x_error, 0, pipe::ERR_BAD_EXPERT);
    atomicAdd(&counts[warp * E1 + expert_of(e)], 1);
  }
  __syncthreads();
  // running sums over the experts, of pairs and of tasks
  int n[EACH], tn[EACH], all = 0, t_all = 0;
#pragma unroll
  for (int j = 0; j < EACH; ++j) {
    const int e = tid * EACH + j;
    n[j] = 0;
    if (e < E1)
      for (int w = 0; w < nw; ++w) n[j] += counts[w * E1 + e];
    tn[j] = e < a.E ? cdiv(n[j], cols) : 0;
    all += n[j];
    t_all += tn[j];
  }
  int run = all, t_run = t_all;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(~0u, run, o), tv = __shfl_up_sync(~0u, t_run, o);
    if (lane >= o) run += v, t_run += tv;
  }
  if (lane == 31) sums[warp] = run, t_sums[warp] = t_run;
  __syncthreads();
  run += __reduce_add_sync(~0u, lane < warp ? sums[lane] : 0) - all;
  t_run += __reduce_add_sync(~0u, lane < warp ? t_sums[lane] : 0) - t_all;
#pragma unroll
  for (int j = 0; j < EACH; ++j) {
    const int e = tid * EACH + j;
    if (e < a.E)
      for (int i = 0; i < tn[j]; ++i) tasks[t_run + i] = Task(e, run + i * cols, min(cols, n[j] - i * cols));
    if (e == a.E) head[0] = t_run, head[1] = run;
    t_run += tn[j];
    if (e < E1)
      for (int w = 0, at = run; w < nw; ++w) {
        const int c = counts[w * E1 + e];
        counts[w * E1 + e] = at;
        at += c;
      }
    run += n[j];
  }
  __syncthreads();
  for (int b = p0; b < p1; b += 32) {
    const int p = b + lane, e = p < p1 ? expert_of(b == p0 ? first : a.ids[p]) : -1;
    const unsigned same = __match_any_sync(~0u, e);
    const int before = __popc(same & ((1u << lane) - 1));
    int at = 0;
    if (p < p1) {
      at = counts[warp * E1 + e];
      order[at + before] = p;
    }
    __syncwarp();
    if (p < p1 && before == 0) counts[warp * E1 + e] = at + __popc(same);
    __syncwarp();
  }
}

__device__ __forceinline__ void sort_pairs(const ExpertsArgs& a, int cols, int* head, int* order, Task* tasks, int* counts) {
  static_assert(3 * X_NT > EXPERTS_MAX_E, "a thread for every three experts");
  if (a.E < X_NT)
    sort_each<1>(a, cols, head, order, tasks, counts);
  else
    sort_each<3>(a, cols, head, order, tasks, counts);
}

// CTA 0 sorts the pairs where they are many; each of the others makes a row of x: the activation, then fp16, for bf16
// scaled by a power of two that puts the row's largest value at 2^14 (as the 4-bit matvec does).  Bound by latency where rows
// are few; 4096 gated rows of 2048 took 42 us more than plain ones with one load at a time, 22 with four.
__global__ void __launch_bounds__(X_NT) prepare_kernel(ExpertsArgs a, int sort, int cols, int* head, int* order, Task* tasks,
                                                          int* exps, uint16_t* xh, int64_t ldxh) {
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ uint32_t s_top;
  if (threadIdx.x == 0) s_top = 0;
  __syncthreads();
  pdl_begin();
  if (sort && blockIdx.x == 0) return sort_pairs(a, cols, head, order, tasks, reinterpret_cast<int*>(smem));
  const int row = blockIdx.x - sort;
  const uint16_t* x = (const uint16_t*)a.x + (int64_t)row * a.ldx;
  uint16_t* v = reinterpret_cast<uint16_t*>(smem);
  uint32_t top = 0;
  // loads without conditions, so that none waits for another
  constexpr int AT_ONCE = 4;
  const int up = a.act != QMV_ACT_NONE ? a.K : 0;
  for (int k0 = threadIdx.x; k0 < a.K; k0 += X_NT * AT_ONCE) {
    uint16_t g[AT_ONCE], u[AT_ONCE];
#pragma unroll
    for (int i = 0; i < AT_ONCE; ++i) {
      const int k = min(k0 + i * X_NT, a.K - 1);
      g[i] = x[k], u[i] = x[up + k];
    }
#pragma unroll
    for (int i = 0; i < AT_ONCE; ++i) {
      const int k = k0 + i * X_NT;
      uint32_t b = g[i];
      if (up) b = gated_bits(f16_f(b, a.x_bf16), f16_f(u[i], a.x_bf16), a.act, a.x_bf16);
      if (k < a.K) v[k] = (uint16_t)b, top = max(top, b & 0x7fffu);
    }
  }
  if (!a.x_bf16) {
    for (int k = threadIdx.x; k < a.K; k += X_NT) xh[row * ldxh + k] = v[k];
    return;
  }
  top = __reduce_max_sync(~0u, top);
  if ((threadIdx.x & 31) == 0) atomicMax(&s_top, top);
  __syncthreads();
  const int e = column_exp(s_top);
  const float f = pow2_f(e);
  if (threadIdx.x == 0) exps[row] = e;
  for (int k = threadIdx.x; k < a.K; k += X_NT)
    xh[row * ldxh + k] = __half_as_ushort(__float2half_rn(__uint_as_float((uint32_t)v[k] << 16) * f));
}

// y[m] = sum_j weights[m][j] * part[m][j], in the order of j.  All that came before the products has
// ended when this starts, so ids and weights are read ahead of the wait for those.
__global__ void __launch_bounds__(128) combine_kernel(ExpertsArgs a, const float* part) {
  __shared__ float w[64];
  __shared__ int in[64];
  const int m = blockIdx.y, r = (blockIdx.x * 128 + threadIdx.x) * 4;
  if (threadIdx.x < a.T) {
    in[threadIdx.x] = (unsigned)ld_early(a.ids + m * a.T + threadIdx.x) < (unsigned)a.E;
    w[threadIdx.x] = ld_early(a.weights + m * a.T + threadIdx.x);
  }
  pdl_begin();
  __syncthreads();
  if (r >= a.R) return;
  float4 y = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  // loads without conditions, so that none waits for another
#pragma unroll 8
  for (int j = 0; j < a.T; ++j) {
    const float4 v = *reinterpret_cast<const float4*>(part + (int64_t)(m * a.T + j) * a.R + r);
    const bool is = in[j];
    y.x = is ? fmaf(w[j], v.x, y.x) : y.x, y.y = is ? fmaf(w[j], v.y, y.y) : y.y;
    y.z = is ? fmaf(w[j], v.z, y.z) : y.z, y.w = is ? fmaf(w[j], v.w, y.w) : y.w;
  }
  const int64_t at = (int64_t)m * a.ldy + r;
  store_y(a.y, at, a.y_dtype, y.x), store_y(a.y, at + 1, a.y_dtype, y.y);
  store_y(a.y, at + 2, a.y_dtype, y.z), store_y(a.y, at + 3, a.y_dtype, y.w);
}

bool sorted_before(const ExpertsArgs& a) { return a.M * a.T > X_OWN; }
// x as it is where the copies can take it; otherwise so many rows of it are made.
bool x_as_is(const ExpertsArgs& a) { return !a.x_bf16 && a.act == QMV_ACT_NONE && (uintptr_t)a.x % 16 == 0 && a.ldx % 8 == 0; }
int rows_made(const ExpertsArgs& a) { return x_as_is(a) ? 0 : a.per_pair ? a.M * a.T : a.M; }

// Where things lie in the workspace: the pairs in order where a kernel before sorts them, the rows of x that are
// made, and the products where they are summed afterwards.
struct Places {
  size_t head, order, tasks, exps, x, part, bytes;
  Places(size_t sorted, size_t rows, size_t K, size_t parts, size_t R) {
    const auto up = [](size_t v) { return (v + 255) & ~(size_t)255; };
    head = 0;
    order = sorted ? 256 : 0;
    tasks = order + up(sorted * 4);
    exps = tasks + up(sorted * sizeof(Task));
    x = exps + up(rows * 4);
    part = x + up(rows * K * 2);
    bytes = part + up(parts * R * 4);
  }
  explicit Places(const ExpertsArgs& a)
      : Places(sorted_before(a) ? (size_t)a.M * a.T : 0, rows_made(a), a.K, a.weights ? (size_t)a.M * a.T : 0, a.R) {}
};

// The shared memory of the products with up to `cols` tokens a task, or false where it does not fit.
bool lay_out(const ExpertsArgs& a, int cols, ExpertsPlan* P) {
  const int bb = block_bytes(a.group, a.zeros != 0);
  const auto up = [](int64_t v) { return (v + 127) & ~(int64_t)127; };
  P->KB = cdiv(a.K, BK);
  P->strips = a.R / ROWS;
  P->cols = cols;
  P->pitch = P->KB * 256 + 64;
  P->x_size = (int)up((int64_t)P->pitch * cols);
  P->xs_size = (int)up((int64_t)P->KB * (BK / a.group) * X_COLS * 4);
  const int64_t part = (int64_t)X_W * cols * ROWS * 4;
  const int pairs = a.M * a.T, tasks = std::min(pairs, pairs / cols + std::min(pairs, a.E));
  P->own = !sorted_before(a);
  const int own = P->own ? (int)(up(pairs * 2) + up(tasks * sizeof(OwnTask))) : 0;
  const int64_t left = (int64_t)dev_info().max_smem_optin - 4096 - (2 * P->x_size + 256 + 2 * P->xs_size + part + own);
  const int64_t fit = left / ((int64_t)X_W * bb);         // blocks a warp's ring can hold
  if (left < 0 || fit < 2) return false;
  P->stage = fit >= 4 ? 2 : 1;
  P->slots = (int)(fit / P->stage < X_SLOTS ? fit / P->stage : X_SLOTS);
  P->x_off = (int)up((int64_t)X_W * P->slots * P->stage * bb);
  P->zero_off = P->x_off + 2 * P->x_size;
  P->xs_off = P->zero_off + 256;
  P->part_off = P->xs_off + 2 * P->xs_size;
  P->order_off = P->part_off + (int)part;
  P->tasks_off = P->order_off + (P->own ? (int)up(pairs * 2) : 0);
  P->smem = P->order_off + own;
  return true;
}

}  // namespace

size_t experts_workspace(int K, int R, int M, int T) {
  const size_t P = (size_t)M * T;
  return Places(P, P, K, P, R).bytes;
}
size_t experts_workspace(const ExpertsArgs& a) { return Places(a).bytes; }

cudaError_t launch_experts(const ExpertsArgs& a, cudaStream_t s) {
  ExpertsPlan P;
  int cols = X_COLS;
  while (!lay_out(a, cols, &P))
    if ((cols /= 2) == 0) return cudaErrorInvalidConfiguration;       // not reached: one column of EXPERTS_MAX_K fits
  const Places at(a);
  uint8_t* ws = (uint8_t*)a.ws;
  P.head = (int*)(ws + at.head);
  P.order = (int*)(ws + at.order);
  P.tasks = (Task*)(ws + at.tasks);
  P.exps = (int*)(ws + at.exps);
  P.part = a.weights ? (float*)(ws + at.part) : nullptr;
  uint16_t* xh = (uint16_t*)(ws + at.x);
  const int rows = rows_made(a), sort = !P.own;
  P.x = rows ? xh : (const uint16_t*)a.x;
  P.ldx = rows ? a.K : a.ldx;
  P.prepared = sort || rows;
  cudaError_t e = cudaSuccess;
  if (P.prepared) {
    const size_t counts = sort ? (size_t)X_W * (a.E + 1) * 4 : 0, smem = std::max(counts, (size_t)a.K * 2);
    static thread_local KernCache c;
    e = prep_kernel(prepare_kernel, c, X_NT, smem, nullptr);
    if (e == cudaSuccess)
      e = launch_step(prepare_kernel, dim3(sort + rows), X_NT, smem, s, 1, a, sort, cols, (int*)(ws + at.head),
                      (int*)(ws + at.order), (Task*)(ws + at.tasks), (int*)(ws + at.exps), xh, (int64_t)a.K);
    if (e != cudaSuccess) return e;
  }
  e = a.group == 32 ? run_experts<32>(a, P, s) : a.group == 64 ? run_experts<64>(a, P, s) : run_experts<128>(a, P, s);
  if (e != cudaSuccess || !a.weights) return e;
  return launch_step(combine_kernel, dim3(cdiv(a.R, 512), a.M), 128, 0, s, 1, a, (const float*)P.part);
}

}  // namespace qmv
