// qmv_experts.cuh -- the products of qmv_w4_experts: each expert's 4-bit weights with the tokens
// routed to it, on the packed layout and the tensor instructions of the 4-bit matvec
// (qmv_w4_gemv.cuh).  One translation unit a group size includes it.
//
// A small kernel (qmv_experts.cu) has sorted the pairs of token and expert by expert, in tasks
// of one expert and up to 8 of its tokens, and put x in fp16.  Here a CTA a streaming
// multiprocessor takes an even share of all strips (32 rows) of all tasks, one task after
// another; within a task its warps share the blocks of its strips evenly, and only the
// pieces of strips that cross a warp's range are joined.  Every warp's ring of bulk
// copies runs on into its next task, and so do the columns of x, so that HBM is read
// without a pause.
#pragma once
#include "qmv_token.cuh"
#include "qmv_w4_math.cuh"

namespace qmv {
namespace w4 {

constexpr int X_W = 16, X_NT = X_W * 32, X_COLS = 8, X_SLOTS = 8;

// A task: `count` tokens of one expert, from `first` on in the order of the pairs.
struct alignas(16) Task {
  int expert, first, count, unused;
};

// What the small kernel leaves in the workspace, and how a CTA's shared memory is laid out.
struct ExpertsPlan {
  const int* head;              // tasks; pairs that have an expert
  const int* order;             // pairs by expert; those without one behind them
  const Task* tasks;
  const int* exps;              // a row's power of two (bf16)
  const uint16_t* x;            // rows of x in fp16, ldx apart
  int64_t ldx;
  float* part;                  // products of pairs, where they are summed afterwards
  int strips, KB;               // of an expert
  int cols;                     // tokens a task
  int slots, stage;             // ring slots a warp, blocks a slot
  int pitch, x_size, xs_size;   // bytes between columns of x, of a task's x, of its sums of x
  int x_off, zero_off, xs_off, part_off, smem;
};

// The error word of this translation unit.
static __device__ int g_x_error = 0;

// act(gate) * up, rounded to x's type: its bits, and its value.
__device__ __forceinline__ uint32_t gated_bits(float g, float u, int act, int bf16) {
  float v;
  if (act == QMV_ACT_SILU) {
    v = g / (1.0f + expf(-g)) * u;
  } else {
    const float t = 0.7978845608028654f * (g + 0.044715f * g * g * g);
    v = 0.5f * g * (1.0f + tanhf(t)) * u;
  }
  return bf16 ? __bfloat16_as_ushort(__float2bfloat16_rn(v)) : __half_as_ushort(__float2half_rn(v));
}
__device__ __forceinline__ float gated(float g, float u, int act, int bf16) {
  return f16_f(gated_bits(g, u, act, bf16), bf16);
}

// A product by its definition, for results that are not finite.
static __device__ __noinline__ float plain_product(const ExpertsArgs& a, int pair, int n) {
  const uint16_t* x = (const uint16_t*)a.x + (int64_t)(a.per_pair ? pair : pair / a.T) * a.ldx;
  const int KB = cdiv(a.K, BK), bb = block_bytes(a.group, a.zeros != 0), gpb = BK / a.group;
  const int row = n & 31, r = row >> 4, hi = (row >> 3) & 1;
  float v = 0.0f, sum = 0.0f, s = 0.0f;
  int z = 8;
  for (int k = 0; k < a.K; ++k) {
    const uint8_t* b = a.packed + ((int64_t)(n >> 5) * KB + (k >> 7)) * bb;
    if (k % a.group == 0) {
      v += sum * s;
      sum = 0.0f;
      const uint8_t* meta = b + CODE_BYTES;
      const int at = (k & 127) / a.group * ROWS + meta_slot(row);
      s = f16_f(reinterpret_cast<const uint16_t*>(meta)[at], a.scale_bf16);
      if (a.zeros) z = meta[2 * gpb * ROWS + at];
    }
    const int j = (k >> 6) & 1, h = (k >> 5) & 1, lane = (row & 7) * 4 + ((k >> 3) & 3);
    const uint32_t w = reinterpret_cast<const uint32_t*>(b)[((r * 2 + j) * 32 + lane) * 4 + hi * 2 + h];
    float xv = f16_f(x[k], a.x_bf16);
    if (a.act != QMV_ACT_NONE) xv = gated(xv, f16_f(x[a.K + k], a.x_bf16), a.act, a.x_bf16);
    sum = fmaf(xv, (float)((int)(rot(w, shift_of(k & 7)) & 15u) - z), sum);
  }
  return v + sum * s;
}

// One block (the b-th of k) of a strip, added to tot (as in qmv_w4_gemv.cuh, for 8 columns).
template <int GROUP, bool SB, bool Z>
__device__ __forceinline__ void block_product(const Block<BK / GROUP>& B, int b, const uint8_t* xp, int x_step,
                                              const float* xsum, int t, float (&tot)[2][4]) {
  constexpr int GPB = BK / GROUP, HPG = GROUP / 32;
  const uint8_t* x = xp + b * x_step;
  const float* sxp = xsum + b * (GPB * X_COLS) + 2 * t;
#pragma unroll
  for (int gi = 0; gi < GPB; ++gi) {
    float low[2][4], high[2][4];           // codes times 2^-21 and 2^-17
    const float none[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int hh = 0; hh < HPG; ++hh) {
      const int st = gi * HPG + hh, q = st >> 1, h = st & 1;   // 32 k of the block
      const uint4 xv = *reinterpret_cast<const uint4*>(x + (x_step ? st * 64 : 0));
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const uint32_t u = h ? B.w[r][q].y : B.w[r][q].x, v = h ? B.w[r][q].w : B.w[r][q].z;   // rows g, g + 8
        constexpr uint32_t L = 0x00780078u, H = 0x07800780u;
        const uint32_t u8 = rot(u, 8), v8 = rot(v, 8);
        mma16816(low[r], hh ? low[r] : none, u & L, v & L, u8 & L, v8 & L, xv.x, xv.y);
        mma16816(high[r], hh ? high[r] : none, u & H, v & H, u8 & H, v8 & H, xv.z, xv.w);
      }
    }
    const float2 sx = *reinterpret_cast<const float2*>(sxp + gi * X_COLS);
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const uint32_t s2 = r ? B.sc[gi].y : B.sc[gi].x;
      const float s0 = f16_f(s2 & 0xffffu, SB), s1 = SB ? __uint_as_float(s2 & 0xffff0000u) : f16_f(s2 >> 16, SB);
      const float z0 = Z ? zero_f(B.zp[gi], 2 * r) : 0x1p-18f, z1 = Z ? zero_f(B.zp[gi], 2 * r + 1) : z0;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        float v = fmaf(high[r][e], 0.0625f, low[r][e]);
        v = fmaf(-(e < 2 ? z0 : z1), e & 1 ? sx.y : sx.x, v);
        tot[r][e] = fmaf(e < 2 ? s0 : s1, v, tot[r][e]);
      }
    }
  }
}

template <int GROUP, bool SB>
__global__ void __launch_bounds__(X_NT, 1)
    experts_kernel(const __grid_constant__ ExpertsArgs a, const __grid_constant__ ExpertsPlan P) {
  constexpr int W = X_W, GPB = BK / GROUP, HPG = GROUP / 32;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ uint64_t full[W][X_SLOTS], x_full[2];
  __shared__ int abort_flag;
  const int tid = threadIdx.x, warp = __shfl_sync(~0u, tid >> 5, 0), lane = tid & 31, g = lane >> 2, t = lane & 3;
  const int KB = P.KB, bb = block_bytes(GROUP, a.zeros != 0);
  uint8_t* ring = smem + (size_t)warp * P.slots * P.stage * bb;
  if (tid == 0) abort_flag = 0;
  if (lane == 0) {
    for (int i = 0; i < P.slots; ++i) pipe::mbar_init(&full[warp][i], 1);
    if (warp < 2) pipe::mbar_init(&x_full[warp], 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (tid < 16) reinterpret_cast<uint4*>(smem + P.zero_off)[tid] = make_uint4(0, 0, 0, 0);
  for (int k = a.K + tid; k < KB * BK; k += X_NT)          // up to 96 k past the end
    for (int m = 0; m < 2 * P.cols; ++m)
      reinterpret_cast<uint16_t*>(smem + P.x_off + (m / P.cols) * P.x_size + (m % P.cols) * P.pitch)[k] = 0;
  __syncthreads();
  pdl_begin();                             // the tasks and x come from the kernel before
  // this CTA's strips, counted through all tasks; those of one task are a segment
  const int64_t all = (int64_t)P.head[0] * P.strips;
  const int u0 = (int)(all * blockIdx.x / gridDim.x), u1 = (int)(all * (blockIdx.x + 1) / gridDim.x);
  const int task0 = u0 / P.strips, segs = u1 > u0 ? (u1 - 1) / P.strips - task0 + 1 : 0;
  const auto begin_of = [&](int i) { return i == 0 ? u0 - task0 * P.strips : 0; };     // first strip within the task
  const auto strips_of = [&](int i) { return min(P.strips, u1 - (task0 + i) * P.strips) - begin_of(i); };
  // warp w's blocks of a segment, counted through its strips
  const auto first_of = [&](int i, int w) { return (int)((unsigned)(strips_of(i) * KB) * (unsigned)w / W); };

  // The ring is kept full by lane 0; all lanes follow its course.
  const uint8_t* src = nullptr;
  int p_seg = -1, p_left = 0, p_blk = 0, issued = 0, landed = 0;
  bool dead = false;                       // a wait of this lane ran out
  const auto next_seg = [&]() {
    while (p_left == 0 && ++p_seg < segs) {
      const int lo = first_of(p_seg, warp), st = (int)((unsigned)lo / (unsigned)KB);
      p_left = first_of(p_seg, warp + 1) - lo;
      p_blk = lo - st * KB;
      src = a.packed + (((int64_t)P.tasks[task0 + p_seg].expert * P.strips + begin_of(p_seg)) * KB + lo) * bb;
    }
  };
  const auto issue = [&](int s) {
    const int cnt = min(P.stage, min(p_left, KB - p_blk)), bytes = cnt * bb;
    if (lane == 0 && !dead) {
      pipe::mbar_arrive_tx(&full[warp][s], bytes);
      bulk_g2s(ring + s * P.stage * bb, src, bytes, &full[warp][s]);
    }
    issued += !dead;
    p_left -= cnt;
    p_blk += cnt;
    src += bytes;
    if (p_blk == KB) p_blk = 0;
    if (p_left == 0) next_seg();
  };
  // a task's columns of x, by warp 0; P.pitch is 64 past a multiple of 128, so that the
  // eight lanes of a 128-byte read touch different banks
  int x_issued = 0;
  const auto issue_x = [&](int i) {
    const Task task = P.tasks[task0 + i];
    if (lane == 0) pipe::mbar_arrive_tx(&x_full[i & 1], task.count * a.K * 2);
    __syncwarp();
    if (lane < task.count) {
      const int pair = P.order[task.first + lane], row = a.per_pair ? pair : pair / a.T;
      bulk_g2s(smem + P.x_off + (i & 1) * P.x_size + lane * P.pitch, P.x + row * P.ldx, a.K * 2, &x_full[i & 1]);
    }
    ++x_issued;
  };
  next_seg();
  if (warp == 0 && segs > 0) issue_x(0);
  for (int i = 0; i < P.slots && p_left > 0; ++i) issue(i);

  int slot = 0, parity = 0;
  for (int seg = 0; seg < segs; ++seg) {
    const Task task = P.tasks[task0 + seg];
    const int mc = task.count, s0 = begin_of(seg);
    // after a wait that ran out this CTA copies and stores nothing any more, but keeps to its course
    if (!dead && !pipe::mbar_wait_fast(&x_full[seg & 1], (seg >> 1) & 1, &abort_flag, pipe::ERR_TIMEOUT_TFULL, &g_x_error))
      dead = true;
    if (warp == 0 && seg + 1 < segs && !__any_sync(~0u, dead)) issue_x(seg + 1);   // all are past the segment before
    const uint8_t* xs = smem + P.x_off + (seg & 1) * P.x_size;
    float* xsum = reinterpret_cast<float*>(smem + P.xs_off + (seg & 1) * P.xs_size);    // [group][8]
    // where a lane reads x; lanes past the last column read zeros
    const int x_step = g < mc ? 256 : 0;
    const uint8_t* xp = g < mc ? xs + g * P.pitch + t * 16 : smem + P.zero_off + t * 16;
    // the sums of x over each group, by the same instructions with ones for weights
    for (int b = warp; b < KB; b += W) {
      constexpr uint32_t ONE = 0x3C003C00u;
#pragma unroll
      for (int gi = 0; gi < GPB; ++gi) {
        float d[4] = {};
#pragma unroll
        for (int hh = 0; hh < HPG; ++hh) {
          const uint4 v = *reinterpret_cast<const uint4*>(xp + b * x_step + (x_step ? (gi * HPG + hh) * 64 : 0));
          mma16816(d, d, ONE, ONE, ONE, ONE, v.x, v.y);
          mma16816(d, d, ONE, ONE, ONE, ONE, v.z, v.w);
        }
        if (g == 0) *reinterpret_cast<float2*>(xsum + (b * GPB + gi) * X_COLS + 2 * t) = make_float2(d[0], d[1]);
      }
    }
    __syncthreads();                       // the sums are there, and the segment before is joined

    // Where warp w leaves a partial sum [mc][32]: that of the first strip of its range, or of a later one.
    const auto place = [&](int w, int second) {
      return reinterpret_cast<float*>(smem + P.part_off + (size_t)(2 * w + second) * (P.cols * ROWS * 4));
    };
    const auto emit = [&](int s, int m, float v) {
      const int pair = P.order[task.first + m], row = (s0 + s) * ROWS + lane;
      v *= 2097152.0f;
      if (a.x_bf16) v *= pow2_f(-P.exps[a.per_pair ? pair : pair / a.T]);
      if (!(fabsf(v) <= 3.402823466e38f)) v = plain_product(a, pair, task.expert * a.R + row);
      if (abort_flag) return;
      if (P.part)
        P.part[(int64_t)pair * a.R + row] = v;
      else
        store_y(a.y, (int64_t)pair * a.ldy + row, a.y_dtype, v);
    };
    const int lo = first_of(seg, warp), hi = first_of(seg, warp + 1);
    const int s_lo = (int)((unsigned)lo / (unsigned)KB), F = strips_of(seg) * KB;
    int s = s_lo, blk = lo - s * KB, f = lo, from = blk;
    float tot[2][4] = {};
    float* to = place(warp, 0);
    while (f < hi) {
      const int cnt = min(P.stage, min(hi - f, KB - blk));
      dead |= !pipe::mbar_wait_fast(&full[warp][slot], parity, &abort_flag, pipe::ERR_TIMEOUT_FULL, &g_x_error);
      landed += !dead;
      const uint8_t* p = ring + slot * P.stage * bb;
      Block<GPB> A, B;
      A.load(p, lane, a.zeros);
      if (cnt > 1) B.load(p + bb, lane, a.zeros);
      __syncwarp();                        // every lane has read the slot: fill it again
      if (p_left > 0) issue(slot);
      if (++slot == P.slots) slot = 0, parity ^= 1;
      if (a.zeros) {
        block_product<GROUP, SB, true>(A, blk, xp, x_step, xsum, t, tot);
        if (cnt > 1) block_product<GROUP, SB, true>(B, blk + 1, xp, x_step, xsum, t, tot);
      } else {
        block_product<GROUP, SB, false>(A, blk, xp, x_step, xsum, t, tot);
        if (cnt > 1) block_product<GROUP, SB, false>(B, blk + 1, xp, x_step, xsum, t, tot);
      }
      f += cnt;
      blk += cnt;
      if (blk == KB || f == hi) {          // the end of the strip, or of the range
#pragma unroll
        for (int r = 0; r < 2; ++r)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int m = 2 * t + (e & 1);
            if (m < mc) to[part_at(m, 16 * r + 8 * (e >> 1) + g)] = tot[r][e];
            tot[r][e] = 0.0f;
          }
        if (from == 0 && blk == KB) {      // the whole strip
          __syncwarp();
#pragma unroll 1
          for (int m = 0; m < mc; ++m) emit(s, m, to[part_at(m, lane)]);
          __syncwarp();
        }
        ++s;
        blk = from = 0;
        to = place(warp, 1);
      }
    }
    if (lo == hi && lo < F)                // fewer blocks than warps: nothing to add
      for (int m = 0; m < mc; ++m) to[part_at(m, lane)] = 0.0f;
    __syncthreads();
    // Strips that several warps share: the warps w0 .. w0 + nw - 1 whose ranges begin in the
    // strip share out its columns; where it begins inside a range, one more piece lies in
    // warp w0 - 1's second place.
    if (lo < F) {
      const int begin = s_lo * KB, end = begin + KB;
      const int w0 = (int)(((unsigned)begin * W + F - 1) / F), nw = (int)(((unsigned)end * W + F - 1) / F) - w0;
      const bool inside = first_of(seg, w0) != begin, whole = first_of(seg, w0 + nw - 1) == begin;
      if (!whole) {                        // else one warp had all of it
#pragma unroll 1
        for (int m = warp - w0; m < mc; m += nw) {
          float v = inside ? place(w0 - 1, 1)[part_at(m, lane)] : 0.0f;
          for (int q = 0; q < nw; ++q) v += place(w0 + q, 0)[part_at(m, lane)];
          emit(s_lo, m, v);
        }
      }
    }
  }
  // after a wait that ran out: let the copies in flight land before the CTA ends
  if (lane == 0 && dead)
    for (; landed < issued; ++landed)
      pipe::mbar_drain(&full[warp][landed % P.slots], (landed / P.slots) & 1, &g_x_error);
  if (warp == 0 && lane == 0 && dead)
    for (int i = max(0, x_issued - 2); i < x_issued; ++i) pipe::mbar_drain(&x_full[i & 1], (i >> 1) & 1, &g_x_error);
  // pairs without an expert: zeros, where no sum goes over them afterwards
  if (!P.part)
    for (int i = P.head[1] + blockIdx.x; i < a.M * a.T; i += gridDim.x)
      for (int r = tid; r < a.R; r += X_NT) store_y(a.y, (int64_t)P.order[i] * a.ldy + r, a.y_dtype, 0.0f);
}

template <int GROUP>
cudaError_t run_experts(const ExpertsArgs& a, const ExpertsPlan& P, cudaStream_t s) {
  const auto one = [&](auto kern, KernCache& c) {
    const cudaError_t e = prep_kernel(kern, c, X_NT, P.smem, nullptr);
    return e != cudaSuccess ? e : launch_step(kern, dim3(dev_info().sms), X_NT, P.smem, s, 1, a, P);
  };
  static thread_local KernCache c[2];
  return a.scale_bf16 ? one(experts_kernel<GROUP, true>, c[1]) : one(experts_kernel<GROUP, false>, c[0]);
}

template <int GROUP>
cudaError_t read_x_error(int clear, int* out) {
  cudaError_t e = cudaMemcpyFromSymbol(out, g_x_error, sizeof(int));
  if (e == cudaSuccess && clear && *out) {
    const int z = 0;
    e = cudaMemcpyToSymbol(g_x_error, &z, sizeof(int));
  }
  return e;
}

}  // namespace w4
}  // namespace qmv
