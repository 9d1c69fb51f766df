// qmv_experts.cuh -- the products of qmv_w4_experts: each expert's 4-bit weights with the tokens
// routed to it, on the packed layout and the tensor instructions of the 4-bit matvec
// (qmv_w4_gemv.cuh).  One translation unit a group size includes it.
//
// The pairs of token and expert are sorted by expert into tasks of one expert and up to 8 of its
// tokens, by every CTA for itself where they are few, otherwise by a kernel before (qmv_experts.cu), which
// also puts x in fp16 where it is not.  (One token of eight experts, 2048 x 2048: 12.0 us with that kernel
// always; that and three loads from global memory behind it that wait for each other took 5 of them.)
// Here a CTA a streaming multiprocessor takes an even share of all strips (32 rows) of all tasks, one task after
// another.  Within a task each warp takes the same number of whole strips; the warps then share
// out the blocks of those that are left over, and only these sums are joined.  Every warp's ring of
// bulk copies runs on into its next task, and so do the columns of x, so that HBM is read
// without a pause.
#pragma once
#include "qmv_token.cuh"
#include "qmv_w4_math.cuh"

namespace qmv {
namespace w4 {

constexpr int X_W = 16, X_NT = X_W * 32, X_COLS = 8, X_SLOTS = 8;

// A task: `count` tokens of one expert, from `first` on in the order of the pairs; in global memory and in
// a CTA's own.
struct alignas(16) Task {
  int expert, first, count, unused;
  Task() = default;
  __device__ __forceinline__ Task(int e, int f, int c) : expert(e), first(f), count(c), unused(0) {}
};
struct alignas(8) OwnTask {
  uint16_t expert, first, count, unused;
  OwnTask() = default;
  __device__ __forceinline__ OwnTask(int e, int f, int c) : expert((uint16_t)e), first((uint16_t)f), count((uint16_t)c), unused(0) {}
};
constexpr int X_OWN = 128;      // pairs that a CTA sorts for itself, at most: a comparison of each with each

// Where the kernel before leaves its results, and how a CTA's shared memory is laid out.
struct ExpertsPlan {
  const int* head;              // tasks; pairs that have an expert
  const int* order;             // pairs by expert; those without one behind them
  const Task* tasks;
  const int* exps;              // a row's power of two (bf16)
  const uint16_t* x;            // rows of x in fp16, ldx apart
  int64_t ldx;
  float* part;                  // products of pairs, where they are summed afterwards
  int own;                      // the pairs are sorted here
  int prepared;                 // a kernel before has made x (and sorted): all that came before it has ended
  int strips, KB;               // of an expert
  int cols;                     // tokens a task
  int slots, stage;             // ring slots a warp, blocks a slot
  int pitch, x_size, xs_size;   // bytes between columns of x, of a task's x, of its sums of x
  int x_off, zero_off, xs_off, part_off, order_off, tasks_off, smem;
};

// The error word of this translation unit.
static __device__ int g_x_error = 0;

// act(gate) * up, rounded to x's type: its bits, and its value.  Both are g / (1 + e^-t), t = g or, since
// (1 + tanh s) / 2 = 1 / (1 + e^-2s), twice GELU's argument: no difference takes bits away, and e^-|t|
// does not overflow (1 + tanh s in fp32 has lost all of them at g = -5.5, g / (1 + e^-g) at -89).
__device__ __forceinline__ uint32_t gated_bits(float g, float u, int act, int bf16) {
  const float t = act == QMV_ACT_SILU ? g : 1.5957691216057308f * (g + 0.044715f * g * g * g), e = expf(-fabsf(t));
  const float v = (t >= 0.0f ? g : g * e) / (1.0f + e) * u;
  return bf16 ? __bfloat16_as_ushort(__float2bfloat16_rn(v)) : __half_as_ushort(__float2half_rn(v));
}
__device__ __forceinline__ float gated(float g, float u, int act, int bf16) {
  return f16_f(gated_bits(g, u, act, bf16), bf16);
}

// The same for up to X_OWN pairs, a thread each: a pair's place is the number of those that come
// before it.  keys: 2 * X_OWN ints.
__device__ __forceinline__ void sort_own(const ExpertsArgs& a, int cols, int* head, uint16_t* order, OwnTask* tasks, int* keys) {
  const int P = a.M * a.T, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int* at_place = keys + X_OWN;
  __shared__ int starts[X_OWN / 32], valid[X_OWN / 32];
  int e = INT32_MAX;                       // behind all
  if (tid < X_OWN) {
    if (tid < P) {
      e = ld_early(a.ids + tid);
      if (e < -1 || e >= a.E) atomicCAS(&g_x_error, 0, pipe::ERR_BAD_EXPERT);
      if ((unsigned)e >= (unsigned)a.E) e = a.E;           // those without an expert come last
    }
    keys[tid] = e;
    at_place[tid] = 0;
  }
  __syncthreads();
  if (tid < P) {
    int less = 0, same = 0, before = 0;
#pragma unroll 2
    for (int q = 0; q < P; q += 4) {
      const int4 k = *reinterpret_cast<const int4*>(keys + q);
      less += (k.x < e) + (k.y < e) + (k.z < e) + (k.w < e);
      same += (k.x == e) + (k.y == e) + (k.z == e) + (k.w == e);
      before += (k.x == e && q < tid) + (k.y == e && q + 1 < tid) + (k.z == e && q + 2 < tid) + (k.w == e && q + 3 < tid);
    }
    order[less + before] = (uint16_t)tid;
    // the first of a task: its expert and its count
    if (e < a.E && before % cols == 0) at_place[less + before] = e << 8 | min(cols, same - before);
  }
  __syncthreads();
  int task = 0;
  uint32_t all = 0;
  if (tid < X_OWN) {
    task = at_place[tid];
    all = __ballot_sync(~0u, task != 0);
    const uint32_t in = __ballot_sync(~0u, e < a.E);
    if (lane == 0) starts[warp] = __popc(all), valid[warp] = __popc(in);
  }
  __syncthreads();
  if (tid < X_OWN) {
    int base = __popc(all & ((1u << lane) - 1));
    for (int w = 0; w < warp; ++w) base += starts[w];
    if (task) tasks[base] = OwnTask(task >> 8, tid, task & 255);
    if (tid == 0) {
      int t = 0, v = 0;
      for (int w = 0; w < X_OWN / 32; ++w) t += starts[w], v += valid[w];
      head[0] = t, head[1] = v;
    }
  }
}

// A product by its definition, for results that are not finite: a lane a product, all of K.  (64 tokens of 8 experts,
// 2048 x 2048: 64 us, with NaN in one token's row 7.5 ms, in every row 21 ms.)
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

// OWN: the pairs are sorted here.
template <int GROUP, bool SB, bool OWN>
__global__ void __launch_bounds__(X_NT, 1)
    experts_kernel(const __grid_constant__ ExpertsArgs a, const __grid_constant__ ExpertsPlan P) {
  constexpr int W = X_W, GPB = BK / GROUP, HPG = GROUP / 32;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ uint64_t full[W][X_SLOTS], x_full[2];
  __shared__ int abort_flag, own_head[2];
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
  // Where a kernel before makes x, all that came before that one has ended when this one starts: ids may be
  // read, the pairs sorted and weights fetched meanwhile.
  const uint16_t* own_order = reinterpret_cast<const uint16_t*>(smem + P.order_off);
  const OwnTask* own_tasks = reinterpret_cast<const OwnTask*>(smem + P.tasks_off);
  const bool ahead = OWN && P.prepared;
  if (!ahead) pdl_begin();
  if constexpr (OWN) {
    sort_own(a, P.cols, own_head, reinterpret_cast<uint16_t*>(smem + P.order_off), reinterpret_cast<OwnTask*>(smem + P.tasks_off),
             reinterpret_cast<int*>(smem));                // what it compares lies where the rings will
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  }
  __syncthreads();
  const auto order_of = [&](int i) { return OWN ? (int)own_order[i] : P.order[i]; };
  const auto task_of = [&](int i) {
    return OWN ? Task(own_tasks[i].expert, own_tasks[i].first, own_tasks[i].count) : P.tasks[i];
  };
  const int n_tasks = OWN ? own_head[0] : P.head[0], n_valid = OWN ? own_head[1] : P.head[1];
  // this CTA's strips, counted through all tasks; those of one task are a segment
  const int all = n_tasks * P.strips, share = all / (int)gridDim.x, more = all - share * (int)gridDim.x;
  const int u0 = share * (int)blockIdx.x + min((int)blockIdx.x, more), u1 = u0 + share + ((int)blockIdx.x < more);
  const int task0 = u0 / P.strips, segs = u1 > u0 ? (u1 - 1) / P.strips - task0 + 1 : 0;
  const auto begin_of = [&](int i) { return i == 0 ? u0 - task0 * P.strips : 0; };     // first strip within the task
  const auto strips_of = [&](int i) { return min(P.strips, u1 - (task0 + i) * P.strips) - begin_of(i); };
  // Of a segment's n strips warp w has n / W whole ones, and of the others (rem) the warps from
  // first_warp(j) on share strip j, block by block.
  const auto first_warp = [&](int j, int rem) { return (j * W + rem - 1) / rem; };
  struct Share {
    int strip, b0, b1, w0, nw;             // the strip within the segment, the blocks, and the warps that share it
  };
  const auto share_of = [&](int n, int w) {
    const int rem = n % W;
    if (rem == 0) return Share{0, 0, 0, 0, 0};
    const int j = w * rem / W, w0 = first_warp(j, rem), nw = first_warp(j + 1, rem) - w0;
    return Share{n / W * W + j, (w - w0) * KB / nw, (w - w0 + 1) * KB / nw, w0, nw};
  };

  // The ring is kept full by lane 0; all lanes follow its course.
  const uint8_t* src = nullptr;
  int p_seg = -1, p_left = 0, p_blk = 0, issued = 0, landed = 0;
  bool p_rest = false;                     // at the strip that is shared
  bool dead = false;                       // a wait of this lane ran out
  const auto next_part = [&]() {
    while (p_left == 0) {
      int strip;
      if (p_rest || p_seg < 0) {
        if (++p_seg >= segs) return;
        const int whole = strips_of(p_seg) / W;
        strip = warp * whole;
        p_left = whole * KB;
        p_blk = 0;
        p_rest = false;
      } else {
        const Share s = share_of(strips_of(p_seg), warp);
        strip = s.strip;
        p_left = s.b1 - s.b0;
        p_blk = s.b0;
        p_rest = true;
      }
      src = a.packed + (((int64_t)task_of(task0 + p_seg).expert * P.strips + begin_of(p_seg) + strip) * KB + p_blk) * bb;
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
    if (p_left == 0) next_part();
  };
  // a task's columns of x, by warp 0; P.pitch is 64 past a multiple of 128, so that the
  // eight lanes of a 128-byte read touch different banks
  int x_issued = 0;
  const auto issue_x = [&](int i) {
    const Task task = task_of(task0 + i);
    if (lane == 0) pipe::mbar_arrive_tx(&x_full[i & 1], task.count * a.K * 2);
    __syncwarp();
    if (lane < task.count) {
      const int pair = order_of(task.first + lane), row = a.per_pair ? pair : pair / a.T;
      bulk_g2s(smem + P.x_off + (i & 1) * P.x_size + lane * P.pitch, P.x + row * P.ldx, a.K * 2, &x_full[i & 1]);
    }
    ++x_issued;
  };
  next_part();
  if (!ahead && warp == 0 && segs > 0) issue_x(0);
  for (int i = 0; i < P.slots && p_left > 0; ++i) issue(i);
  if (ahead) {
    pdl_begin();                           // x comes from the kernel before
    if (warp == 0 && segs > 0) issue_x(0);
  }

  int slot = 0, parity = 0;
  for (int seg = 0; seg < segs; ++seg) {
    const Task task = task_of(task0 + seg);
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

    // Where warp w leaves a partial sum [mc][32].
    const auto place = [&](int w) { return reinterpret_cast<float*>(smem + P.part_off + (size_t)w * (P.cols * ROWS * 4)); };
    // column m and row `row` of the segment; what a lane needs of a column comes from global memory once
    const auto emit = [&](int row, int pair, float scale, float v) {
      v = v * 2097152.0f * scale;          // one after the other: their product may be infinite where v's is not
      if (!(fabsf(v) <= 3.402823466e38f)) v = plain_product(a, pair, task.expert * a.R + s0 * ROWS + row);
      if (abort_flag) return;
      if (P.part)
        P.part[(int64_t)pair * a.R + s0 * ROWS + row] = v;
      else
        store_y(a.y, (int64_t)pair * a.ldy + s0 * ROWS + row, a.y_dtype, v);
    };
    const auto pair_of = [&](int m) { return order_of(task.first + m); };
    const auto scale_of = [&](int pair) { return a.x_bf16 ? pow2_f(-P.exps[a.per_pair ? pair : pair / a.T]) : 1.0f; };
    int my_pair[2] = {0, 0};               // of the columns 2 t and 2 t + 1, whose sums this lane has
    float my_scale[2] = {0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < 2; ++i)
      if (2 * t + i < mc) my_pair[i] = pair_of(2 * t + i), my_scale[i] = scale_of(my_pair[i]);
    const int n = strips_of(seg), whole = n / W;
    const Share rest = share_of(n, warp);
    const int rest_n = rest.b1 - rest.b0;
    float tot[2][4] = {};
    int strip = warp * whole, blk = 0, left = whole * KB + rest_n;
    if (whole == 0) strip = rest.strip, blk = rest.b0;
    while (left > 0) {
      const bool last = left <= rest_n;
      const int end = last ? rest.b1 : KB, cnt = min(P.stage, end - blk);
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
      left -= cnt;
      blk += cnt;
      if (blk == end) {                    // the end of the strip, or of this warp's part of it
        const bool joined = last && rest.nw > 1;
        float* to = place(warp);
#pragma unroll
        for (int r = 0; r < 2; ++r)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int m = 2 * t + (e & 1), row = 16 * r + 8 * (e >> 1) + g;
            if (m < mc) {
              if (joined)
                to[part_at(m, row)] = tot[r][e];
              else
                emit(strip * ROWS + row, my_pair[e & 1], my_scale[e & 1], tot[r][e]);
            }
            tot[r][e] = 0.0f;
          }
        ++strip;
        blk = 0;
        if (left == rest_n) strip = rest.strip, blk = rest.b0;
      }
    }
    if (rest.nw > 1 && rest_n == 0)        // fewer blocks than warps: nothing to add
      for (int m = 0; m < mc; ++m) place(warp)[part_at(m, lane)] = 0.0f;
    __syncthreads();
    // the warps of a strip share out its columns
#pragma unroll 1
    for (int m = warp - rest.w0; rest.nw > 1 && m < mc; m += rest.nw) {
      float v = 0.0f;
      for (int q = 0; q < rest.nw; ++q) v += place(rest.w0 + q)[part_at(m, lane)];
      const int pair = pair_of(m);
      emit(rest.strip * ROWS + lane, pair, scale_of(pair), v);
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
    for (int i = n_valid + blockIdx.x; i < a.M * a.T; i += gridDim.x)
      for (int r = tid; r < a.R; r += X_NT) store_y(a.y, (int64_t)order_of(i) * a.ldy + r, a.y_dtype, 0.0f);
}

template <int GROUP>
cudaError_t run_experts(const ExpertsArgs& a, const ExpertsPlan& P, cudaStream_t s) {
  const auto one = [&](auto kern, KernCache& c) {
    const cudaError_t e = prep_kernel(kern, c, X_NT, P.smem, nullptr);
    return e != cudaSuccess ? e : launch_step(kern, dim3(dev_info().sms), X_NT, P.smem, s, 1, a, P);
  };
  static thread_local KernCache c[4];
  if (P.own) return a.scale_bf16 ? one(experts_kernel<GROUP, true, true>, c[3]) : one(experts_kernel<GROUP, false, true>, c[2]);
  return a.scale_bf16 ? one(experts_kernel<GROUP, true, false>, c[1]) : one(experts_kernel<GROUP, false, false>, c[0]);
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
