// qmv_w4_gemv.cuh -- the matvec of the 4-bit weights packed by qmv_w4.cu:
//   y[m][n] = sum_g s[n][g] * (sum_{k in g} x[m][k] * q[n][k] - z[n][g] * sum_{k in g} x[m][k]).
// One translation unit a group size and type of scales includes it.
//
// The products run on m16n8k16 tensor instructions with the weights as the
// 16-row operand, in fp16: products are exact and sums fp32.  The fp16 numbers
// below 2^-13 are evenly spaced, so a masked code in the low 11 bits of a half is,
// read as fp16, the code times 2^-21 (at bit 3) or 2^-17 (at bit 7): the operand
// without any arithmetic, four masks and one rotation for eight codes.  The two
// kinds have sums of their own.  x in bf16 becomes fp16 once a CTA, each column
// scaled by a power of two that puts its largest value at 2^14: what falls off is
// below 2^-39 of that.  (Decoding to bf16 instead, where a code at bit 3 under the
// exponent of 16 is 16 + q, takes four masks and three rotations, all on a pipe of
// half rate: 25.4 us against 24.0 us for 43008x5376 and one token, 57.9 against 56.2
// for 262144x2048 in groups of 32 and five.)
// The zero point comes off a group's sum as z * sum(x), as the library's fast
// form does for its offset; the sums of x are formed once a CTA.
//
// The work is bound by HBM once the instructions per code are few, so a CTA a
// streaming multiprocessor stays for the whole launch and its warps share out
// its strips evenly, block by block and without meeting: a warp's range may
// begin and end inside a strip, and only those partial sums are joined, once,
// at the end.  Every warp keeps a ring of bulk copies of its own in flight.
#pragma once
#include <type_traits>

#include "qmv_pipe.cuh"
#include "qmv_step.cuh"

namespace qmv {
namespace w4 {

static __device__ int g_w4_error = 0;

constexpr int MAX_SLOTS = 8, MAX_CLUSTER = 8, NBMAX = 4;

// Where a warp's partial sum of (column m, row) lies: the rows of a column are
// swapped in eights by column pair, so that the lanes of a warp touch different
// banks both as the products leave them and row by row.
__device__ __forceinline__ int part_at(int m, int row) { return m * ROWS + (row ^ (((m >> 1) & 3) << 3)); }

// Warps a CTA: with many columns fewer, whose partial sums leave room for x.
__host__ __device__ constexpr int warps_of(int nb) { return nb <= 2 ? 16 : 8; }

__device__ __forceinline__ void bulk_g2s(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                   pipe::sa(dst)),
               "l"(src), "r"(bytes), "r"(pipe::sa(bar))
               : "memory");
}

// D = A . B + C on 16 rows x 8 columns x 16 k.
__device__ __forceinline__ void mma16816(float (&d)[4], const float* c, uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%10,%11,%12,%13};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(c[0]), "f"(c[1]), "f"(c[2]), "f"(c[3]));
}

__device__ __forceinline__ uint32_t rot(uint32_t v, int n) { return __funnelshift_r(v, v, n); }

__device__ __forceinline__ float f16_f(uint32_t bits16, int bf16) {
  return bf16 ? __uint_as_float(bits16 << 16) : __half2float(__ushort_as_half((unsigned short)bits16));
}

// The zero point in byte i of v on the scale of a group's sum, 2^-21: placed in the
// mantissa of 4, whose last bit that is.
__device__ __forceinline__ float zero_f(uint32_t v, int i) {
  return __uint_as_float(__byte_perm(v, 0x40800000u, 0x7650u | (uint32_t)i)) - 4.0f;
}

// The power of two that scales a bf16 column, from the bits of its largest
// magnitude (141 minus the exponent field puts that at 2^14), kept where it and its
// inverse are normal: a column below 2^-112 is scaled by 2^126 only, which leaves
// multiples of 2^-7, so that fp16 still holds all of it.
__device__ __forceinline__ int column_exp(uint32_t top) { return min(141 - (int)(top >> 7), 126); }
__device__ __forceinline__ float pow2_f(int e) { return __uint_as_float((uint32_t)(127 + e) << 23); }

__device__ __forceinline__ void store_y(void* y, int64_t at, int dtype, float v) {
  if (dtype == QMV_F32)
    ((float*)y)[at] = v;
  else if (dtype == QMV_F16)
    ((__half*)y)[at] = __float2half_rn(v);
  else
    ((__nv_bfloat16*)y)[at] = __float2bfloat16_rn(v);
}

// How a launch divides the work.  A cluster of ks CTAs takes whole strips, each
// CTA one ks-th of their k.
struct Plan {
  int ks, ks_log, ncl;          // CTAs a cluster (a power of two), clusters
  int k_share, k_more;          // blocks of k a CTA; so many of them have one more
  int s_share, s_more;          // strips a cluster, likewise
  int kbs;                      // blocks of k a CTA, at most
  int cols;                     // columns a launch row (grid.y) takes
  int slots, stage;             // ring slots a warp, blocks a slot
  int rs;                       // strips between two meetings of a cluster
  int vec;                      // x can be read 16 bytes at a time
  int pitch;                    // bytes between the columns of x in shared memory
  int x_off, zero_off, xs_off, part_off, red_off, smem;   // bytes in shared memory; the rings come first
  int second_off, second_step;  // the second places of the warps
};

// A sum by its definition: for results that are not finite, where x * q and z *
// sum(x) apart may give another answer.
static __device__ __noinline__ float plain_sum(const GemvArgs4& a, int m, int n, int k0, int k1) {
  const uint16_t* x = (const uint16_t*)a.x + (int64_t)m * a.ldx;
  const int KB = cdiv(a.K, BK), bb = block_bytes(a.group, a.zeros != 0), gpb = BK / a.group;
  const int row = n & 31, r = row >> 4, hi = (row >> 3) & 1;
  float v = 0.0f, sum = 0.0f, s = 0.0f;
  int z = 8;
  for (int k = k0; k < k1; ++k) {
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
    sum = fmaf(f16_f(x[k], a.x_bf16), (float)((int)(rot(w, shift_of(k & 7)) & 15u) - z), sum);
  }
  return v + sum * s;
}

// A lane's share of a block: the codes of two 16-row halves and two 64-k tiles,
// and for each group the scales and zero points of its rows g, g + 8, g + 16, g + 24.
template <int GPB>
struct Block {
  uint4 w[2][2];
  uint2 sc[GPB];
  uint32_t zp[GPB];
  __device__ __forceinline__ void load(const uint8_t* p, int lane, int zeros) {
#pragma unroll
    for (int r = 0; r < 2; ++r)
#pragma unroll
      for (int q = 0; q < 2; ++q) w[r][q] = *reinterpret_cast<const uint4*>(p + ((r * 2 + q) * 32 + lane) * 16);
    const uint8_t* meta = p + CODE_BYTES + (lane >> 2) * 8;
#pragma unroll
    for (int gi = 0; gi < GPB; ++gi) {
      sc[gi] = *reinterpret_cast<const uint2*>(meta + gi * (2 * ROWS));
      if (zeros) zp[gi] = *reinterpret_cast<const uint32_t*>(p + CODE_BYTES + 2 * GPB * ROWS + gi * ROWS + (lane >> 2) * 4);
    }
  }
};

// SB: the scales are bf16 (fp16 otherwise).
template <int GROUP, int NB, bool SB>
__global__ void __launch_bounds__(warps_of(NB) * 32, 1)
    gemv_kernel(const __grid_constant__ GemvArgs4 a, const __grid_constant__ Plan P) {
  constexpr int W = warps_of(NB), NT = W * 32;
  constexpr int GPB = BK / GROUP, HPG = GROUP / 32;      // groups a block, 32-k steps a group
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ uint64_t full[W][MAX_SLOTS];
  __shared__ uint64_t x_full;
  __shared__ uint32_t colmax[8 * NB];
  __shared__ int abort_flag;
  // the warp's number from one lane, so that what follows from it is known to be uniform
  const int tid = threadIdx.x, warp = __shfl_sync(~0u, tid >> 5, 0), lane = tid & 31, g = lane >> 2, t = lane & 3;
  const int KB = cdiv(a.K, BK), NS = cdiv(a.N, ROWS), bb = block_bytes(GROUP, a.zeros != 0);
  const int m0 = blockIdx.y * P.cols, mc = min(P.cols, a.M - m0);
  const int rank = blockIdx.x & (P.ks - 1), cl = blockIdx.x >> P.ks_log;
  // even shares: the first few CTAs or clusters have one more
  const int kb0 = rank * P.k_share + min(rank, P.k_more), kbn = P.k_share + (rank < P.k_more);
  const int S0 = cl * P.s_share + min(cl, P.s_more), S1 = S0 + P.s_share + (cl < P.s_more);
  const int rounds = P.ks == 1 ? 1 : cdiv(S1 - S0, P.rs);
  // warp w's blocks of round r, counted through the round's strips
  const auto strips_of = [&](int r) { return min(P.rs, S1 - S0 - r * P.rs); };
  const auto first_of = [&](int r, int w) { return (int)((unsigned)(strips_of(r) * kbn) * (unsigned)w / W); };
  uint8_t* ring = smem + (size_t)warp * P.slots * P.stage * bb;
  if (tid == 0) abort_flag = 0;
  if (tid < 8 * NB) colmax[tid] = 0;

  // The ring is kept full by lane 0; all lanes follow its course.  A copy is up to
  // `stage` neighbouring blocks of a strip.
  const uint8_t* src = nullptr;
  int p_round = -1, p_left = 0, p_blk = 0, issued = 0, landed = 0;
  bool dead = false;                       // a wait of this lane ran out
  const auto next_round = [&]() {
    while (p_left == 0 && ++p_round < rounds) {
      const int lo = first_of(p_round, warp);
      p_left = first_of(p_round, warp + 1) - lo;
      const int st = (int)((unsigned)lo / (unsigned)kbn);
      p_blk = lo - st * kbn;
      src = a.packed + ((int64_t)(S0 + p_round * P.rs + st) * KB + kb0 + p_blk) * bb;
    }
  };
  const auto issue = [&](int s) {
    const int cnt = min(P.stage, min(p_left, kbn - p_blk)), bytes = cnt * bb;
    if (lane == 0 && !dead) {
      pipe::mbar_arrive_tx(&full[warp][s], bytes);
      bulk_g2s(ring + s * P.stage * bb, src, bytes, &full[warp][s]);
    }
    issued += !dead;
    p_left -= cnt;
    p_blk += cnt;
    src += bytes;
    if (p_blk == kbn) p_blk = 0, src += (int64_t)(KB - kbn) * bb;
    if (p_left == 0) next_round();
  };
  if (lane == 0) {
    for (int i = 0; i < P.slots; ++i) pipe::mbar_init(&full[warp][i], 1);
    if (warp == 0) pipe::mbar_init(&x_full, 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (!a.early) asm volatile("griddepcontrol.wait;" ::: "memory");
  __syncwarp();
  next_round();
  for (int i = 0; i < P.slots && p_left > 0; ++i) issue(i);

  // x to shared memory as it is, a row a column, P.pitch bytes apart (64 past a
  // multiple of 128, so that the eight lanes of a 128-byte read touch different banks).
  uint8_t* xs = smem + P.x_off;
  const uint16_t* xg = (const uint16_t*)a.x + (int64_t)m0 * a.ldx + (int64_t)kb0 * BK;
  const int klim = min(kbn * BK, a.K - kb0 * BK);
  if (tid < 16) reinterpret_cast<uint4*>(smem + P.zero_off)[tid] = make_uint4(0, 0, 0, 0);
  pdl_begin();                             // x may come from the kernel before
  if (P.vec) {
    if (warp == 0) {
      if (lane == 0) pipe::mbar_arrive_tx(&x_full, mc * klim * 2);
      __syncwarp();
      for (int m = lane; m < mc; m += 32) bulk_g2s(xs + m * P.pitch, xg + (int64_t)m * a.ldx, klim * 2, &x_full);
    }
  } else {
    for (int m = 0; m < mc; ++m)
#pragma unroll 4
      for (int k = tid; k < klim; k += NT) reinterpret_cast<uint16_t*>(xs + m * P.pitch)[k] = xg[(int64_t)m * a.ldx + k];
  }
  if (klim < kbn * BK && tid < kbn * BK - klim)           // up to 96 k past the end
    for (int m = 0; m < mc; ++m) reinterpret_cast<uint16_t*>(xs + m * P.pitch)[klim + tid] = 0;
  __syncthreads();
  if (P.vec && !pipe::mbar_wait_fast(&x_full, 0, &abort_flag, pipe::ERR_TIMEOUT_TFULL, &g_w4_error))
    pipe::mbar_drain(&x_full, 0, &g_w4_error);           // this CTA stores nothing after a wait that ran out

  if (a.x_bf16) {
    // to fp16, in place: 16 lanes take a block of a column, eight values a lane, once
    // for the columns' largest magnitudes and once to scale by them
    const auto each = [&](auto f) {
      for (int b = 2 * warp + (lane >> 4), m = 0;; b += 2 * W) {
        while (b >= kbn && m < mc) b -= kbn, ++m;
        if (__all_sync(~0u, m >= mc)) break;
        f(m, reinterpret_cast<uint4*>(xs + m * P.pitch + b * 256) + (lane & 15));
      }
    };
    each([&](int m, const uint4* p) {
      uint32_t top = 0;
      if (m < mc) {
        const uint4 v = *p;
        constexpr uint32_t ABS = 0x7fff7fffu;
        const uint32_t t2 = __vmaxu2(__vmaxu2(v.x & ABS, v.y & ABS), __vmaxu2(v.z & ABS, v.w & ABS));
        top = max(t2 & 0xffffu, t2 >> 16);
      }
#pragma unroll
      for (int o = 8; o; o >>= 1) top = max(top, __shfl_xor_sync(~0u, top, o));
      if ((lane & 15) == 0 && m < mc) atomicMax(&colmax[m], top);
    });
    __syncthreads();
    each([&](int m, uint4* p) {
      if (m >= mc) return;
      const float f = pow2_f(column_exp(colmax[m]));
      uint4 v = *p;
      const auto two = [&](uint32_t& w) {
        const __half2 h = __floats2half2_rn(__uint_as_float(w << 16) * f, __uint_as_float(w & 0xffff0000u) * f);
        w = *reinterpret_cast<const uint32_t*>(&h);
      };
      two(v.x), two(v.y), two(v.z), two(v.w);
      *p = v;
    });
    __syncthreads();
  }

  // Where a lane reads x; lanes past the last column read zeros.
  const bool in_last = 8 * (NB - 1) + g < mc;
  const uint8_t* xp[NB];
#pragma unroll
  for (int c = 0; c < NB; ++c) xp[c] = xs + (8 * c + g) * P.pitch + t * 16;
  if (!in_last) xp[NB - 1] = smem + P.zero_off + t * 16;
  const int l_step = in_last ? 256 : 0;

  // The sums of x over each group, by the same instructions with ones for weights.
  float* xsum = reinterpret_cast<float*>(smem + P.xs_off);             // [group][8 * NB]
  for (int b = warp; b < kbn; b += W) {
    constexpr uint32_t ONE = 0x3C003C00u;
#pragma unroll
    for (int c = 0; c < NB; ++c)
#pragma unroll
      for (int gi = 0; gi < GPB; ++gi) {
        float d[4] = {};
#pragma unroll
        for (int hh = 0; hh < HPG; ++hh) {
          const uint4 v = *reinterpret_cast<const uint4*>(xp[c] + b * (c < NB - 1 ? 256 : l_step) + (gi * HPG + hh) * 64);
          mma16816(d, d, ONE, ONE, ONE, ONE, v.x, v.y);
          mma16816(d, d, ONE, ONE, ONE, ONE, v.z, v.w);
        }
        if (g == 0) *reinterpret_cast<float2*>(xsum + (b * GPB + gi) * (8 * NB) + 8 * c + 2 * t) = make_float2(d[0], d[1]);
      }
  }
  __syncthreads();

  float* red = reinterpret_cast<float*>(smem + P.red_off);             // [2][rs][mc][32], clusters only
  // Where warp w leaves a partial sum [mc][32]: that of the first strip of its range
  // (place 0), or of a later one (place 1, which may be its own ring, by then read out).
  const auto place = [&](int w, int second) {
    return reinterpret_cast<float*>(second ? smem + P.second_off + (size_t)w * P.second_step
                                           : smem + P.part_off + (size_t)w * (P.cols * ROWS * 4));
  };
  // A finished sum goes out (or to the cluster's sum).  One that is not finite is
  // formed again by its definition.
  const auto emit = [&](int round, int s, int m, float v) {
    v *= 2097152.0f;
    if (a.x_bf16) v *= pow2_f(-column_exp(colmax[m]));
    const int64_t n = (int64_t)(S0 + round * P.rs + s) * ROWS + lane;
    if (!(fabsf(v) <= 3.402823466e38f) && n < a.N)
      v = plain_sum(a, m0 + m, (int)n, kb0 * BK, kb0 * BK + klim);
    if (P.ks > 1)
      red[(((round & 1) * P.rs + s) * mc + m) * 32 + lane] = v;
    else if (n < a.N && !abort_flag)
      store_y(a.y, (int64_t)(m0 + m) * a.ldy + n, a.y_dtype, v);
  };

  // One block (the CTA's b-th of k) of a strip, added to tot.
  const auto product = [&](auto with_zeros, const Block<GPB>& B, int b, float (&tot)[2][NB][4]) {
    constexpr bool Z = decltype(with_zeros)::value;
    const int xo = b * 256, xl = b * l_step;
    const float* sxp = xsum + b * (GPB * 8 * NB) + 2 * t;
#pragma unroll
    for (int gi = 0; gi < GPB; ++gi) {
      float low[2][NB][4], high[2][NB][4];       // codes times 2^-21 and 2^-17
      const float none[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int hh = 0; hh < HPG; ++hh) {
        const int st = gi * HPG + hh, q = st >> 1, h = st & 1;   // 32 k of the block
        uint4 xv[NB];
#pragma unroll
        for (int c = 0; c < NB; ++c) xv[c] = *reinterpret_cast<const uint4*>(xp[c] + (c < NB - 1 ? xo : xl) + st * 64);
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const uint32_t u = h ? B.w[r][q].y : B.w[r][q].x, v = h ? B.w[r][q].w : B.w[r][q].z;   // rows g, g + 8
          constexpr uint32_t L = 0x00780078u, H = 0x07800780u;
          const uint32_t u8 = rot(u, 8), v8 = rot(v, 8);
#pragma unroll
          for (int c = 0; c < NB; ++c) {
            mma16816(low[r][c], hh ? low[r][c] : none, u & L, v & L, u8 & L, v8 & L, xv[c].x, xv[c].y);
            mma16816(high[r][c], hh ? high[r][c] : none, u & H, v & H, u8 & H, v8 & H, xv[c].z, xv[c].w);
          }
        }
      }
      float2 sx[NB];
#pragma unroll
      for (int c = 0; c < NB; ++c) sx[c] = *reinterpret_cast<const float2*>(sxp + gi * (8 * NB) + 8 * c);
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const uint32_t s2 = r ? B.sc[gi].y : B.sc[gi].x;
        const float s0 = f16_f(s2 & 0xffffu, SB), s1 = SB ? __uint_as_float(s2 & 0xffff0000u) : f16_f(s2 >> 16, SB);
        const float z0 = Z ? zero_f(B.zp[gi], 2 * r) : 0x1p-18f, z1 = Z ? zero_f(B.zp[gi], 2 * r + 1) : z0;
#pragma unroll
        for (int c = 0; c < NB; ++c)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            float v = fmaf(high[r][c][e], 0.0625f, low[r][c][e]);
            v = fmaf(-(e < 2 ? z0 : z1), e & 1 ? sx[c].y : sx[c].x, v);
            tot[r][c][e] = fmaf(e < 2 ? s0 : s1, v, tot[r][c][e]);
          }
      }
    }
  };
  int slot = 0, parity = 0;
  for (int round = 0; round < rounds; ++round) {
    const int lo = first_of(round, warp), hi = first_of(round, warp + 1);
    const int s_lo = (int)((unsigned)lo / (unsigned)kbn), F = strips_of(round) * kbn;
    int s = s_lo, blk = lo - s * kbn, f = lo, from = blk;
    float tot[2][NB][4] = {};
    float* to = place(warp, 0);            // the first strip of the range, later ones
    while (f < hi) {
      const int cnt = min(P.stage, min(hi - f, kbn - blk));
      // after a wait that ran out this CTA copies and stores nothing any more, but the warp
      // keeps to its course; with a cluster along k the others still add and store what it
      // had by then (the device error word says that results are incomplete)
      dead |= !pipe::mbar_wait_fast(&full[warp][slot], parity, &abort_flag, pipe::ERR_TIMEOUT_FULL, &g_w4_error);
      landed += !dead;
      const uint8_t* p = ring + slot * P.stage * bb;
      Block<GPB> A, B;
      A.load(p, lane, a.zeros);
      if (cnt > 1) B.load(p + bb, lane, a.zeros);
      __syncwarp();                        // every lane has read the slot: fill it again
      if (p_left > 0) issue(slot);
      if (++slot == P.slots) slot = 0, parity ^= 1;
      if (a.zeros) {
        product(std::true_type(), A, blk, tot);
        if (cnt > 1) product(std::true_type(), B, blk + 1, tot);
      } else {
        product(std::false_type(), A, blk, tot);
        if (cnt > 1) product(std::false_type(), B, blk + 1, tot);
      }
      f += cnt;
      blk += cnt;
      if (blk == kbn || f == hi) {         // the end of the strip, or of the range
#pragma unroll
        for (int r = 0; r < 2; ++r)
#pragma unroll
          for (int c = 0; c < NB; ++c)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int m = 8 * c + 2 * t + (e & 1);
              if (m < mc) to[part_at(m, 16 * r + 8 * (e >> 1) + g)] = tot[r][c][e];
              tot[r][c][e] = 0.0f;
            }
        if (from == 0 && blk == kbn) {     // the whole strip
          __syncwarp();
#pragma unroll 1
          for (int m = 0; m < mc; ++m) emit(round, s, m, to[part_at(m, lane)]);
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
    // Strips that several warps share: the warps w0 .. w0 + nw - 1 whose ranges begin in
    // the strip share out its columns.  Their pieces are in their first places, and
    // where the strip begins inside a range, one more in warp w0 - 1's second.
    if (lo < F) {
      const int begin = s_lo * kbn, end = begin + kbn;
      const int w0 = (int)(((unsigned)begin * W + F - 1) / F), nw = (int)(((unsigned)end * W + F - 1) / F) - w0;
      const bool inside = first_of(round, w0) != begin, whole = first_of(round, w0 + nw - 1) == begin;
      if (!whole) {                        // else one warp had all of it
#pragma unroll 1
        for (int m = warp - w0; m < mc; m += nw) {
          float v = inside ? place(w0 - 1, 1)[part_at(m, lane)] : 0.0f;
          for (int q = 0; q < nw; ++q) v += place(w0 + q, 0)[part_at(m, lane)];
          emit(round, s_lo, m, v);
        }
      }
    }
    if (P.ks > 1) {
      // the CTAs of a cluster add theirs, each finishing a share; two buffers, so that the
      // next round's barrier is the only other one needed
      __syncwarp();
      cluster_arrive();
      cluster_wait();
      const int items = strips_of(round) * mc;
      for (int i = rank + P.ks * warp; i < items; i += P.ks * W) {
        const int st = i / mc, m = i - st * mc;
        float v = 0.0f;
        for (int q = 0; q < P.ks; ++q)
          v += __uint_as_float(ld_cluster32(cluster_addr(red + (((round & 1) * P.rs + st) * mc + m) * 32 + lane, q)));
        const int64_t n = (int64_t)(S0 + round * P.rs + st) * ROWS + lane;
        if (n < a.N && !abort_flag) store_y(a.y, (int64_t)(m0 + m) * a.ldy + n, a.y_dtype, v);
      }
      __syncwarp();
    }
  }
  // after a wait that ran out: let the copies in flight land before the CTA ends
  if (lane == 0 && dead)
    for (; landed < issued; ++landed)
      pipe::mbar_drain(&full[warp][landed % P.slots], (landed / P.slots) & 1, &g_w4_error);
  if (P.ks > 1) {                          // the others may still read this CTA's sums
    __syncwarp();
    cluster_arrive();
    cluster_wait();
  }
}

// How many clusters of ks CTAs the device holds at once (its GPCs need not hold
// a whole number of them).  One CTA fills a streaming multiprocessor whatever the
// shape, so the answer hangs on ks alone.
template <typename Kern>
static int clusters_of(Kern kern, int threads, int ks, const DevInfo& d) {
  struct Seen {
    int dev = -1, n[MAX_CLUSTER + 1] = {};
  };
  static thread_local Seen c;
  if (ks == 1) return d.sms;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return d.sms / ks;
  if (c.dev != dev) c = Seen(), c.dev = dev;
  if (!c.n[ks]) {
    const int smem = d.max_smem_optin - 4096;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = ks;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.gridDim = dim3(ks);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int n = 0, limit = 0;
    if (allow_smem(kern, &limit) != cudaSuccess ||
        cudaOccupancyMaxActiveClusters(&n, kern, &cfg) != cudaSuccess || n < 1) {
      cudaGetLastError();
      n = d.sms / ks;
    }
    c.n[ks] = n;
  }
  return c.n[ks];
}

// The shared memory of a plan with ks CTAs along k, or false where it does not fit.
static bool lay_out(const GemvArgs4& a, int nb, int ks, int ncl, const DevInfo& d, Plan* P) {
  const int KB = cdiv(a.K, BK), NS = cdiv(a.N, ROWS), bb = block_bytes(a.group, a.zeros != 0), W = warps_of(nb);
  P->ks = ks;
  P->ks_log = 0;
  while (1 << P->ks_log < ks) ++P->ks_log;
  P->kbs = cdiv(KB, ks);
  P->ncl = ncl < NS ? ncl : NS;
  P->k_share = KB / ks;
  P->k_more = KB % ks;
  P->s_share = NS / P->ncl;
  P->s_more = NS % P->ncl;
  const int strips = cdiv(NS, P->ncl);
  // a cluster meets after rs strips, whose sums take at most 16 KB a buffer
  int rs = strips;
  if (ks > 1) {
    const int most = 16384 / (P->cols * ROWS * 4);
    rs = cdiv(strips, cdiv(strips, most < 1 ? 1 : most));
  }
  P->rs = rs;
  const auto up = [](int64_t v) { return (v + 127) & ~(int64_t)127; };
  P->pitch = P->kbs * 256 + 64;
  // Only strips that are fewer than warps never lie whole inside a range but at its
  // beginning; then, and with one round, the second place is used once, at the end.
  const bool once = rs >= strips && strips <= W;
  const int64_t x = up((int64_t)P->pitch * P->cols), xs = up((int64_t)P->kbs * (BK / a.group) * 8 * nb * 4),
                places = (int64_t)W * P->cols * ROWS * 4, part = up(places * (once ? 1 : 2)),
                red = ks > 1 ? up((int64_t)(rs < strips ? 2 : 1) * rs * P->cols * ROWS * 4) : 0;
  const int64_t left = (int64_t)d.max_smem_optin - 4096 - (x + 256 + xs + part + red);
  const int64_t fit = left / ((int64_t)W * bb);           // blocks a warp's ring can hold
  if (left < 0 || fit < 2) return false;
  P->stage = fit >= 4 ? 2 : 1;
  P->slots = (int)(fit / P->stage < MAX_SLOTS ? fit / P->stage : MAX_SLOTS);
  P->x_off = (int)up((int64_t)W * P->slots * P->stage * bb);
  P->zero_off = P->x_off + (int)x;
  P->xs_off = P->zero_off + 256;
  P->part_off = P->xs_off + (int)xs;
  P->red_off = P->part_off + (int)part;
  P->second_off = once ? 0 : P->part_off + (int)places;
  P->second_step = once ? P->slots * P->stage * bb : P->cols * ROWS * 4;
  P->smem = P->red_off + (int)red;
  return true;
}

// What joining the sums of a cluster costs, in blocks that a CTA reads meanwhile.
constexpr int CLUSTER_COST = 16;

// The number of CTAs along k with the fewest blocks for the busiest CTA, among
// those whose x fits beside the rings.
template <int NB, typename Kern>
static bool choose(const GemvArgs4& a, Kern kern, int cols, Plan* best) {
  const DevInfo& d = dev_info();
  const int KB = cdiv(a.K, BK), NS = cdiv(a.N, ROWS);
  int64_t least = -1;
  for (int ks = 1; ks <= MAX_CLUSTER && ks <= KB; ks *= 2) {
    Plan P;
    P.cols = cols;
    const int ncl = clusters_of(kern, warps_of(NB) * 32, ks, d);
    if (!lay_out(a, NB, ks, ncl, d, &P)) continue;
    const int64_t cost = (int64_t)cdiv(NS, ncl) * cdiv(KB, ks) + (ks > 1 ? CLUSTER_COST : 0);
    if (least < 0 || cost < least) least = cost, *best = P;
  }
  return least >= 0;
}

template <int GROUP, int NB, bool SB>
static cudaError_t run(const GemvArgs4& a, int cols, cudaStream_t s, bool* fits) {
  const auto kern = gemv_kernel<GROUP, NB, SB>;
  Plan P;
  *fits = choose<NB>(a, kern, cols, &P);
  if (!*fits) return cudaSuccess;
  P.vec = a.ldx % 8 == 0 && (uintptr_t)a.x % 16 == 0;
  static thread_local KernCache c;
  const cudaError_t e = prep_kernel(kern, c, warps_of(NB) * 32, dev_info().max_smem_optin - 4096, nullptr);
  if (e != cudaSuccess) return e;
  return launch_step(kern, dim3(P.ncl * P.ks, cdiv(a.M, cols)), warps_of(NB) * 32, P.smem, s, P.ks, a, P);
}

// Columns in as few launch rows as fit, filled evenly.
template <int GROUP, bool SB>
cudaError_t launch_group(const GemvArgs4& a, cudaStream_t s) {
  for (int top = 8 * NBMAX; top >= 1; top = top > 8 ? top - 8 : top / 2) {
    const int cols = cdiv(a.M, cdiv(a.M, top));
    bool fits = false;
    cudaError_t e;
    switch (cdiv(cols, 8)) {
      case 1: e = run<GROUP, 1, SB>(a, cols, s, &fits); break;
      case 2: e = run<GROUP, 2, SB>(a, cols, s, &fits); break;
      case 3: e = run<GROUP, 3, SB>(a, cols, s, &fits); break;
      default: e = run<GROUP, 4, SB>(a, cols, s, &fits); break;
    }
    if (fits || e != cudaSuccess) return e;
  }
  return cudaErrorInvalidConfiguration;    // not reached: one column of MAX_K fits
}

template <int GROUP, bool SB>
cudaError_t read_error(int clear, int* out) {
  cudaError_t e = cudaMemcpyFromSymbol(out, g_w4_error, sizeof(int));
  if (e == cudaSuccess && clear && *out) {
    const int z = 0;
    e = cudaMemcpyToSymbol(g_w4_error, &z, sizeof(int));
  }
  return e;
}

}  // namespace w4
}  // namespace qmv
