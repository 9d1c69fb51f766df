// qmv_w4.cu -- 4-bit weights with a scale and a zero point a group:
//   y[m][n] = sum_g s[n][g] * sum_{k in g} x[m][k] * (q[n][k] - z[n][g]).
//
// The packed layout is the order in which the tensor cores read the weights:
// one 16-byte word of a lane holds, for a 16-row half and 64 k, the codes of
// rows g and g + 8 (g = lane / 4) at k = 32 h + 8 t + 0..7 (t = lane % 4,
// h = 0, 1), so the words of a warp are 512 consecutive bytes and no code
// moves between lanes.  Inside a 32-bit word code i sits at nibble
// i / 2 + 4 * (i % 2), so that one mask yields a pair (k, k + 1).
#include "qmv_pipe.cuh"
#include "qmv_step.cuh"

namespace qmv {

__device__ int g_w4_error = 0;

int read_w4_error(int clear, int* out) {
  cudaError_t e = cudaMemcpyFromSymbol(out, g_w4_error, sizeof(int));
  if (e == cudaSuccess && clear && *out) {
    const int z = 0;
    e = cudaMemcpyToSymbol(g_w4_error, &z, sizeof(int));
  }
  return (int)e;
}

namespace w4 {

__host__ __device__ constexpr int nibble_of(int i) { return (i >> 1) + 4 * (i & 1); }

// One thread a 16-byte word: block b of strip s, half r, tile j, lane.
__global__ void __launch_bounds__(256) pack_kernel(const uint8_t* __restrict__ codes,
                                                   uint8_t* __restrict__ packed, int N, int K,
                                                   int KB, int64_t words, int bbytes) {
  const int64_t stride = (int64_t)gridDim.x * blockDim.x;
  for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < words; i += stride) {
    const int lane = (int)(i & 31), j = (int)(i >> 5) & 1, r = (int)(i >> 6) & 1;
    const int64_t blk = i >> 7;
    const int64_t n0 = (blk / KB) * ROWS + 16 * r + (lane >> 2);
    const int k0 = (int)(blk % KB) * BK + 64 * j + 8 * (lane & 3);
    uint32_t w[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {            // (row g, h 0), (g, 1), (g + 8, 0), (g + 8, 1)
      const int64_t n = n0 + 8 * (q >> 1);
      const int k = k0 + 32 * (q & 1);
      uint2 c = make_uint2(0, 0);
      if (n < N && k < K) c = *reinterpret_cast<const uint2*>(codes + n * K + k);
      w[q] = 0;
#pragma unroll
      for (int e = 0; e < 8; ++e)
        w[q] |= (((e < 4 ? c.x : c.y) >> (8 * (e & 3))) & 15u) << (4 * nibble_of(e));
    }
    *reinterpret_cast<uint4*>(packed + blk * bbytes + ((r * 2 + j) * 32 + lane) * 16) =
        make_uint4(w[0], w[1], w[2], w[3]);
  }
}

// One thread a (block, group, row): its scale and zero point; zero scales past the end.
__global__ void __launch_bounds__(256) pack_meta_kernel(const uint16_t* __restrict__ scales,
                                                        const uint8_t* __restrict__ zeros,
                                                        uint8_t* __restrict__ packed, int N, int G,
                                                        int KB, int GPB, int64_t items, int bbytes) {
  const int64_t stride = (int64_t)gridDim.x * blockDim.x;
  for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < items; i += stride) {
    const int row = (int)(i & 31);
    const int gi = (int)((i >> 5) % GPB);
    const int64_t blk = (i >> 5) / GPB;
    const int64_t n = (blk / KB) * ROWS + row;
    const int g = (int)(blk % KB) * GPB + gi;
    const bool in = n < N && g < G;
    uint8_t* meta = packed + blk * bbytes + CODE_BYTES;
    const int at = gi * ROWS + meta_slot(row);
    reinterpret_cast<uint16_t*>(meta)[at] = in ? scales[n * G + g] : (uint16_t)0;
    if (zeros) meta[2 * GPB * ROWS + at] = in ? (uint8_t)(zeros[n * G + g] & 15) : (uint8_t)8;
  }
}

__global__ void __launch_bounds__(256) unpack_kernel(const uint8_t* __restrict__ packed,
                                                     uint8_t* __restrict__ codes, int N, int K,
                                                     int KB, int bbytes) {
  const int64_t items = (int64_t)N * K, stride = (int64_t)gridDim.x * blockDim.x;
  for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < items; i += stride) {
    const int64_t n = i / K;
    const int k = (int)(i - n * K), row = (int)(n & 31);
    const int r = row >> 4, hi = (row >> 3) & 1, j = (k >> 6) & 1, h = (k >> 5) & 1;
    const int lane = (row & 7) * 4 + ((k >> 3) & 3);
    const uint8_t* b = packed + ((n >> 5) * KB + (k >> 7)) * (int64_t)bbytes;
    const uint32_t w = reinterpret_cast<const uint32_t*>(b)[((r * 2 + j) * 32 + lane) * 4 + hi * 2 + h];
    codes[i] = (uint8_t)((w >> (4 * nibble_of(k & 7))) & 15u);
  }
}

static int flat_grid(int64_t n) {
  const int64_t b = (n + 255) / 256, cap = 152 * 16;
  return (int)(b < cap ? b : cap);
}

cudaError_t launch_w4_pack(const qmv_w4pack& p, const uint8_t* codes, const uint16_t* scales,
                           const uint8_t* zeros, uint8_t* packed, cudaStream_t s) {
  const int KB = cdiv(p.K, BK), GPB = BK / p.group, bb = block_bytes(p.group, p.zeros != 0);
  const int64_t blocks = (int64_t)cdiv(p.N, ROWS) * KB;
  pack_kernel<<<flat_grid(blocks * 128), 256, 0, s>>>(codes, packed, p.N, p.K, KB, blocks * 128, bb);
  const int64_t items = blocks * GPB * ROWS;
  pack_meta_kernel<<<flat_grid(items), 256, 0, s>>>(scales, zeros, packed, p.N, p.G, KB, GPB, items, bb);
  return cudaGetLastError();
}

cudaError_t launch_w4_unpack(const qmv_w4pack& p, uint8_t* codes, cudaStream_t s) {
  unpack_kernel<<<flat_grid((int64_t)p.N * p.K), 256, 0, s>>>(p.d_packed, codes, p.N, p.K, cdiv(p.K, BK),
                                                              block_bytes(p.group, p.zeros != 0));
  return cudaGetLastError();
}

// ------------------------------------------------------------------ matvec --
//
// The products run on m16n8k16 tensor instructions with the weights as the
// 16-row operand.  A masked nibble of a 32-bit word is, read as a pair of
// fp16, the subnormal pair q * 2^-24 (nibbles 0 and 4) or q * 2^-20 (nibbles 1
// and 5): the operand without any arithmetic, four masks and one shift for
// eight codes.  The products x * q are exact and their sums fp32; the zero
// point comes off a group's sum as z * sum(x), as the library's fast form does
// for its offset.  For that x is brought once per CTA into shared memory as
// fp16, in the order the instructions read it, each column scaled by a power
// of two that puts its largest value at 2^14 (so that bf16 fits, and the
// values that meet a 2^-20 nibble can be taken 16 times smaller): what falls
// off is below 2^-35 of the column's largest value.

constexpr int WARPS = 16, NT = WARPS * 32, MAX_SLOTS = 8;
constexpr int PART_LD = 36;     // floats between the columns of a warp's sums: no bank conflicts
constexpr int PART_FLOATS = 8 * PART_LD;

__device__ __forceinline__ void bulk_g2s(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                   pipe::sa(dst)),
               "l"(src), "r"(bytes), "r"(pipe::sa(bar))
               : "memory");
}

__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ float scale_f(uint32_t bits16, int bf16) {
  return bf16 ? __uint_as_float(bits16 << 16) : __half2float(__ushort_as_half((unsigned short)bits16));
}

// A small whole number as fp32: placed in the mantissa of 2^23.
__device__ __forceinline__ float whole_f(uint32_t v) {
  return __uint_as_float(0x4B000000u | v) - 8388608.0f;
}

__device__ __forceinline__ void store_y(void* y, int64_t at, int dtype, float v) {
  if (dtype == QMV_F32)
    ((float*)y)[at] = v;
  else if (dtype == QMV_F16)
    ((__half*)y)[at] = __float2half_rn(v);
  else
    ((__nv_bfloat16*)y)[at] = __float2bfloat16_rn(v);
}

// Eight activations of a column as they are stored.
__device__ __forceinline__ uint4 load_x8(const uint16_t* p, int vec) {
  if (vec) return *reinterpret_cast<const uint4*>(p);
  uint32_t v[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) v[e] = (uint32_t)p[2 * e] | ((uint32_t)p[2 * e + 1] << 16);
  return make_uint4(v[0], v[1], v[2], v[3]);
}

__device__ __forceinline__ float x_f(uint32_t bits16, int bf16) { return scale_f(bits16, bf16); }

// The power of two that a column is scaled by, from the bits of its largest
// magnitude: 141 minus the exponent field puts that value at 2^14 (a bit lower
// where it is subnormal in fp32; any power serves a column of zeros).  Between
// -113 and 141, so it is applied in two halves.
__device__ __forceinline__ int column_exp(uint32_t top, int bf16) {
  return 141 - (int)(__float_as_uint(x_f(top, bf16)) >> 23);
}
__device__ __forceinline__ float pow2_f(int e) { return __uint_as_float((uint32_t)(127 + e) << 23); }

// How a launch divides the work.  A cluster of ks CTAs takes whole strips, each
// CTA one ks-th of k; in a CTA, kw warps share a strip and 16 / kw strips run
// side by side.
struct Plan {
  int ks, kw, slots;     // CTAs along k, warps along k, ring slots a warp
  int kbs;               // blocks of k a CTA (the last CTA of a cluster may have fewer)
  int cols;              // columns a launch row (grid.y) takes
  int vec;               // x can be read 16 bytes at a time
  int x_off, xs_off, part_off, red_off, smem;   // bytes in shared memory; the rings come first
};

// All warps that share a strip.
__device__ __forceinline__ void strip_sync(int sw, int kw) {
  if (kw > 1)
    pipe::named_bar(1 + sw, kw * 32);
  else
    __syncwarp();
}

// The non-finite activations of a column, left out of the products, against row
// n as the definition has them (inf * 0 and inf - inf are NaN).
__device__ __noinline__ float nonfinite_part(const GemvArgs4& a, int m, int n, int k0, int k1) {
  const uint16_t* x = (const uint16_t*)a.x + (int64_t)m * a.ldx;
  const uint32_t inf = a.x_bf16 ? 0x7f80u : 0x7c00u;
  const int KB = cdiv(a.K, BK), bb = block_bytes(a.group, a.zeros != 0), gpb = BK / a.group;
  const int row = n & 31, lane4 = (row & 7) * 4, r = row >> 4, hi = (row >> 3) & 1;
  float v = 0.0f;
  for (int k = k0; k < k1; ++k) {
    if ((x[k] & 0x7fffu) < inf) continue;
    const uint8_t* b = a.packed + ((int64_t)(n >> 5) * KB + (k >> 7)) * bb;
    const int j = (k >> 6) & 1, h = (k >> 5) & 1, lane = lane4 + ((k >> 3) & 3);
    const uint32_t w = reinterpret_cast<const uint32_t*>(b)[((r * 2 + j) * 32 + lane) * 4 + hi * 2 + h];
    const int q = (w >> (4 * nibble_of(k & 7))) & 15, gi = (k & 127) / a.group;
    const uint8_t* meta = b + CODE_BYTES;
    const int at = gi * ROWS + meta_slot(row);
    const int z = a.zeros ? meta[2 * gpb * ROWS + at] : 8;
    v += x_f(x[k], a.x_bf16) * ((float)(q - z) * scale_f(reinterpret_cast<const uint16_t*>(meta)[at], a.scale_bf16));
  }
  return v;
}

template <int GROUP, int NB>
__global__ void __launch_bounds__(NT, 1) gemv_kernel(const __grid_constant__ GemvArgs4 a, const __grid_constant__ Plan P) {
  constexpr int GPB = BK / GROUP, HPG = GROUP / 32;      // groups a block, 32-k steps a group
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ uint64_t full[WARPS][MAX_SLOTS];
  __shared__ uint32_t colmax[8 * NB];
  __shared__ int bad[8 * NB];
  __shared__ int abort_flag;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  const int KB = cdiv(a.K, BK), NS = cdiv(a.N, ROWS), bb = block_bytes(GROUP, a.zeros != 0);
  const int m0 = blockIdx.y * P.cols, mc = min(P.cols, a.M - m0);
  const int rank = blockIdx.x % P.ks, cl = blockIdx.x / P.ks, ncl = gridDim.x / P.ks;
  const int kb0 = min(KB, rank * P.kbs), kbn = min(KB - kb0, P.kbs);   // this CTA's blocks of k
  const int SW = WARPS / P.kw, sw = warp / P.kw, kw = warp % P.kw;
  const int per = kw < kbn ? (kbn - kw + P.kw - 1) / P.kw : 0;         // this warp's blocks of a strip
  const int rounds = cdiv(NS, ncl * SW), strip0 = cl * SW + sw, dstrip = ncl * SW;
  const int mine_strips = strip0 < NS ? (NS - strip0 + dstrip - 1) / dstrip : 0;
  const int64_t n = (int64_t)per * mine_strips;                        // this warp's copies
  uint8_t* ring = smem + (size_t)warp * P.slots * bb;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (tid < 8 * NB) colmax[tid] = 0, bad[tid] = 0;
  if (tid == 0) abort_flag = 0;
  // Lane 0 keeps the ring full: copy i is block i % per of the warp's strip i / per.
  int64_t issued = 0;
  const uint8_t* src = a.packed + ((int64_t)strip0 * KB + kb0 + kw) * bb;
  int src_j = 0;
  const auto issue = [&](int s) {
    pipe::mbar_arrive_tx(&full[warp][s], bb);
    bulk_g2s(ring + s * bb, src, bb, &full[warp][s]);
    ++issued;
    if (++src_j == per) {
      src_j = 0;
      src += ((int64_t)dstrip * KB - (int64_t)(per - 1) * P.kw) * bb;
    } else {
      src += (int64_t)P.kw * bb;
    }
  };
  if (lane == 0) {
    for (int i = 0; i < P.slots; ++i) pipe::mbar_init(&full[warp][i], 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    for (int i = 0; i < P.slots && issued < n; ++i) issue(i);
  }
  __syncthreads();
  asm volatile("griddepcontrol.wait;" ::: "memory");     // x may come from the kernel before

  // x to shared memory.  Chunks of eight k: chunk c of a column is step c / 4, lane
  // part c % 4; 16 chunks a block, so 16 neighbouring lanes share column and block.
  uint4* xs4 = reinterpret_cast<uint4*>(smem + P.x_off);               // [step][column][4]
  float* xsum = reinterpret_cast<float*>(smem + P.xs_off);             // [group][8 * NB]
  const int nch = kbn * 16, total = nch * mc;
  const uint32_t inf = a.x_bf16 ? 0x7f80u : 0x7c00u;
  const uint16_t* xg = (const uint16_t*)a.x + (int64_t)m0 * a.ldx;
  const int klim = a.K - kb0 * BK;
  for (int i0 = 0; i0 < total; i0 += NT) {               // total is a multiple of 16
    const int i = i0 + tid, m = i / nch, c = i - m * nch;
    uint32_t mx = 0;
    if (i < total && c * 8 < klim) {
      const uint4 v = load_x8(xg + (int64_t)m * a.ldx + (int64_t)kb0 * BK + c * 8, P.vec);
      const uint32_t w[4] = {v.x & 0x7fff7fffu, v.y & 0x7fff7fffu, v.z & 0x7fff7fffu, v.w & 0x7fff7fffu};
      const uint32_t p = __vmaxu2(__vmaxu2(w[0], w[1]), __vmaxu2(w[2], w[3]));
      mx = max(p & 0xffffu, p >> 16);
      if (mx >= inf) {
        bad[m] = 1;
        mx = 0;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const uint32_t b = (w[e >> 1] >> (16 * (e & 1))) & 0xffffu;
          if (b < inf) mx = max(mx, b);
        }
      }
    }
#pragma unroll
    for (int o = 8; o; o >>= 1) mx = max(mx, __shfl_xor_sync(~0u, mx, o));
    if ((lane & 15) == 0 && i < total) atomicMax(&colmax[m], mx);
  }
  __syncthreads();
  for (int i0 = 0; i0 < total; i0 += NT) {
    const int i = i0 + tid, m = i / nch, c = i - m * nch;
    float sum = 0.0f;
    if (i < total) {
      uint4 v = make_uint4(0, 0, 0, 0);
      if (c * 8 < klim) v = load_x8(xg + (int64_t)m * a.ldx + (int64_t)kb0 * BK + c * 8, P.vec);
      const int ex = column_exp(colmax[m], a.x_bf16);
      const float f1 = pow2_f(ex / 2), f2 = pow2_f(ex - ex / 2);
      const uint32_t in[4] = {v.x, v.y, v.z, v.w};
      uint32_t o[4];
#pragma unroll
      for (int p = 0; p < 4; ++p) {                      // pairs 1 and 3 meet the 2^-20 nibbles
        float u[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const uint32_t b = e ? in[p] >> 16 : in[p] & 0xffffu;
          u[e] = (b & 0x7fffu) < inf ? x_f(b, a.x_bf16) * f1 * f2 : 0.0f;
          if (p & 1) u[e] *= 0.0625f;
        }
        const __half2 h = __floats2half2_rn(u[0], u[1]);
        o[p] = *reinterpret_cast<const uint32_t*>(&h);
        sum += (__low2float(h) + __high2float(h)) * (p & 1 ? 16.0f : 1.0f);
      }
      xs4[((c >> 2) * mc + m) * 4 + (c & 3)] = make_uint4(o[0], o[1], o[2], o[3]);
    }
#pragma unroll
    for (int q = GROUP / 16; q; q >>= 1) sum += __shfl_xor_sync(~0u, sum, q);
    if (i < total && c % (GROUP / 8) == 0) xsum[(c / (GROUP / 8)) * (8 * NB) + m] = sum * 5.9604644775390625e-08f;
  }
  __syncthreads();

  float* part = reinterpret_cast<float*>(smem + P.part_off) + warp * PART_FLOATS;
  int slot = 0, parity = 0;
  int64_t used = 0;
  for (int round = 0; round < rounds; ++round) {
    const int strip = strip0 + round * dstrip;
    float tot[2][NB][4] = {};
    const int todo = strip < NS ? per : 0;
    for (int j = 0; j < todo; ++j) {
      const int b = kw + j * P.kw;
      if (!__all_sync(~0u, pipe::mbar_wait_fast(&full[warp][slot], parity, &abort_flag, pipe::ERR_TIMEOUT_FULL, &g_w4_error)))
        break;
      const uint8_t* blk = ring + slot * bb;
      uint4 w[2][2];
#pragma unroll
      for (int r = 0; r < 2; ++r)
#pragma unroll
        for (int q = 0; q < 2; ++q) w[r][q] = *reinterpret_cast<const uint4*>(blk + ((r * 2 + q) * 32 + lane) * 16);
      const uint8_t* meta = blk + CODE_BYTES;
      uint2 sc[GPB];
      uint32_t zp[GPB];
#pragma unroll
      for (int gi = 0; gi < GPB; ++gi) {
        sc[gi] = *reinterpret_cast<const uint2*>(meta + 2 * (gi * ROWS + g * 4));
        zp[gi] = a.zeros ? *reinterpret_cast<const uint32_t*>(meta + 2 * GPB * ROWS + gi * ROWS + g * 4) : 0x08080808u;
      }
      ++used;
      __syncwarp();                       // every lane has read the slot
      if (lane == 0 && issued < n) issue(slot);
      if (++slot == P.slots) slot = 0, parity ^= 1;
#pragma unroll
      for (int gi = 0; gi < GPB; ++gi) {
        float acc[2][NB][4] = {};
#pragma unroll
        for (int hh = 0; hh < HPG; ++hh) {
          const int st = gi * HPG + hh, q = st >> 1, h = st & 1;   // 32 k of the block
          uint4 xv[NB];
#pragma unroll
          for (int c = 0; c < NB; ++c) {
            xv[c] = make_uint4(0, 0, 0, 0);
            if (8 * c + g < mc) xv[c] = xs4[((b * 4 + st) * mc + 8 * c + g) * 4 + t];
          }
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const uint32_t u = h ? w[r][q].y : w[r][q].x, v = h ? w[r][q].w : w[r][q].z;   // rows g, g + 8
            const uint32_t u8 = u >> 8, v8 = v >> 8;
#pragma unroll
            for (int c = 0; c < NB; ++c) {
              mma16816(acc[r][c], u & 0x000f000fu, v & 0x000f000fu, u & 0x00f000f0u, v & 0x00f000f0u, xv[c].x, xv[c].y);
              mma16816(acc[r][c], u8 & 0x000f000fu, v8 & 0x000f000fu, u8 & 0x00f000f0u, v8 & 0x00f000f0u, xv[c].z, xv[c].w);
            }
          }
        }
        float2 sx[NB];
#pragma unroll
        for (int c = 0; c < NB; ++c)
          sx[c] = *reinterpret_cast<const float2*>(xsum + (b * GPB + gi) * (8 * NB) + 8 * c + 2 * t);
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const uint32_t s2 = r ? sc[gi].y : sc[gi].x, z2 = zp[gi] >> (16 * r);
          const float s0 = scale_f(s2 & 0xffffu, a.scale_bf16), s1 = scale_f(s2 >> 16, a.scale_bf16);
          const float z0 = whole_f(z2 & 255u), z1 = whole_f((z2 >> 8) & 255u);
#pragma unroll
          for (int c = 0; c < NB; ++c) {
            tot[r][c][0] = fmaf(s0, fmaf(-z0, sx[c].x, acc[r][c][0]), tot[r][c][0]);
            tot[r][c][1] = fmaf(s0, fmaf(-z0, sx[c].y, acc[r][c][1]), tot[r][c][1]);
            tot[r][c][2] = fmaf(s1, fmaf(-z1, sx[c].x, acc[r][c][2]), tot[r][c][2]);
            tot[r][c][3] = fmaf(s1, fmaf(-z1, sx[c].y, acc[r][c][3]), tot[r][c][3]);
          }
        }
      }
    }
    // the warps of a strip add their sums, eight columns at a time
    float* red = reinterpret_cast<float*>(smem + P.red_off) + ((round & 1) * SW + sw) * (mc * 32);
    const int64_t nn = (int64_t)strip * ROWS + lane;
#pragma unroll
    for (int c = 0; c < NB; ++c) {
      if (8 * c >= mc) break;
#pragma unroll
      for (int r = 0; r < 2; ++r)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int col = 2 * t + (e & 1);
          if (8 * c + col < mc) part[col * PART_LD + 16 * r + 8 * (e >> 1) + g] = tot[r][c][e];
        }
      strip_sync(sw, P.kw);
      for (int m = 8 * c + kw; m < min(mc, 8 * c + 8); m += P.kw) {
        float v = 0.0f;
        for (int q = 0; q < P.kw; ++q) v += part[(q - kw) * PART_FLOATS + (m - 8 * c) * PART_LD + lane];
        const int ex = 24 - column_exp(colmax[m], a.x_bf16);
        v = v * pow2_f(ex / 2) * pow2_f(ex - ex / 2);
        if (bad[m] && nn < a.N) v += nonfinite_part(a, m0 + m, (int)nn, kb0 * BK, min(a.K, (kb0 + kbn) * BK));
        if (P.ks > 1)
          red[m * 32 + lane] = v;
        else if (nn < a.N && !abort_flag)
          store_y(a.y, (int64_t)(m0 + m) * a.ldy + nn, a.y_dtype, v);
      }
      strip_sync(sw, P.kw);              // the sums have been read
    }
    if (P.ks > 1) {
      // the CTAs of a cluster add theirs: each finishes a share of the columns; two
      // buffers, so that the next round's barrier is the only other one needed
      __syncwarp();
      cluster_arrive();
      cluster_wait();
      for (int m = rank * P.kw + kw; m < mc; m += P.ks * P.kw) {
        float v = 0.0f;
        for (int q = 0; q < P.ks; ++q) v += __uint_as_float(ld_cluster32(cluster_addr(red + m * 32 + lane, q)));
        if (nn < a.N && !abort_flag) store_y(a.y, (int64_t)(m0 + m) * a.ldy + nn, a.y_dtype, v);
      }
      __syncwarp();
    }
  }
  // after a wait that ran out: let the copies in flight land before the CTA ends
  if (lane == 0)
    for (; used < issued; ++used) {
      pipe::mbar_drain(&full[warp][slot], parity, &g_w4_error);
      if (++slot == P.slots) slot = 0, parity ^= 1;
    }
  if (P.ks > 1) {                          // the others may still read this CTA's sums
    cluster_arrive();
    cluster_wait();
  }
}

// Blocks of k a warp should have at least, so that the sums of a strip are
// added once per so many blocks.
constexpr int MIN_PER = 4;

static bool plan_for(const GemvArgs4& a, int nb, int cols, int ks, const DevInfo& d, Plan* P) {
  const int KB = cdiv(a.K, BK), NS = cdiv(a.N, ROWS), bb = block_bytes(a.group, a.zeros != 0);
  P->ks = ks;
  P->kbs = cdiv(KB, ks);
  P->cols = cols;
  const int ncl = d.sms / ks;
  int kw = 1;
  while (kw < WARPS && kw * 2 * MIN_PER <= P->kbs) kw *= 2;
  // fewer strips than warps to take them: more warps a strip
  while (kw < WARPS && kw < P->kbs && (int64_t)ncl * (WARPS / kw) > NS) kw *= 2;
  P->kw = kw;
  const int64_t x = (int64_t)P->kbs * BK * cols * 2, xs = (int64_t)P->kbs * (BK / a.group) * 8 * nb * 4,
                part = (int64_t)WARPS * PART_FLOATS * 4, red = ks > 1 ? (int64_t)2 * (WARPS / kw) * cols * 32 * 4 : 0;
  const int64_t left = d.max_smem_optin - 2048 - (x + xs + part + red) - 4 * 128;
  const int64_t fit = left / ((int64_t)WARPS * bb);
  if (left < 0 || fit < 2) return false;
  P->slots = (int)(fit < MAX_SLOTS ? fit : MAX_SLOTS);
  const auto up = [](int64_t v) { return (int)((v + 127) & ~(int64_t)127); };
  P->x_off = up((int64_t)WARPS * P->slots * bb);
  P->xs_off = P->x_off + up(x);
  P->part_off = P->xs_off + up(xs);
  P->red_off = P->part_off + up(part);
  P->smem = P->red_off + up(red);
  return true;
}

// Columns of one launch row: the fewest rows of at most 8 * NBMAX, filled evenly.
constexpr int NBMAX = 4;

// How many clusters of ks CTAs the device holds at once (GPCs need not hold a
// whole number of them), cached for the last shape asked.
template <typename Kern>
static int max_clusters(Kern kern, int ks, int smem, int sms) {
  struct Seen {
    int dev = -1, ks = 0, smem = 0, n = 0;
  };
  static thread_local Seen c;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return sms / ks;
  if (c.dev != dev || c.ks != ks || c.smem != smem) {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = ks;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.gridDim = dim3(ks);
    cfg.blockDim = dim3(NT);
    cfg.dynamicSmemBytes = smem;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int n = 0;
    if (cudaOccupancyMaxActiveClusters(&n, kern, &cfg) != cudaSuccess || n < 1) n = sms / ks;
    c.dev = dev, c.ks = ks, c.smem = smem, c.n = n;
  }
  return c.n;
}

// The division of k over a cluster for this many columns, or false where x does
// not fit beside the rings: the fewest CTAs along k that leave three ring slots
// (two at eight CTAs); where strips are fewer than CTAs, more of them while
// each warp still has a block.
static bool choose(const GemvArgs4& a, int nb, int cols, const DevInfo& d, Plan* P) {
  const int KB = cdiv(a.K, BK), NS = cdiv(a.N, ROWS);
  int ks = 1;
  bool ok = plan_for(a, nb, cols, ks, d, P);
  while ((!ok || P->slots < 3) && ks < 8 && ks * 2 <= KB) {
    ks *= 2;
    ok = plan_for(a, nb, cols, ks, d, P);
  }
  if (!ok) return false;
  while (ks < 8 && (int64_t)NS * ks * 2 <= d.sms && KB >= ks * 2 * WARPS) {
    ks *= 2;
    ok = plan_for(a, nb, cols, ks, d, P);
  }
  return ok;
}

template <int GROUP, int NB>
static cudaError_t run(const GemvArgs4& a, Plan P, cudaStream_t s) {
  const DevInfo& d = dev_info();
  P.vec = a.ldx % 8 == 0 && (uintptr_t)a.x % 16 == 0;
  static thread_local KernCache c;
  const cudaError_t e = prep_kernel(gemv_kernel<GROUP, NB>, c, NT, P.smem, nullptr);
  if (e != cudaSuccess) return e;
  const int need = cdiv(cdiv(a.N, ROWS), WARPS / P.kw);
  int ncl = P.ks == 1 ? d.sms : max_clusters(gemv_kernel<GROUP, NB>, P.ks, P.smem, d.sms);
  if (ncl > need) ncl = need;
  return launch_step(gemv_kernel<GROUP, NB>, dim3(ncl * P.ks, cdiv(a.M, P.cols)), NT, P.smem, s, P.ks, a, P);
}

template <int GROUP>
static cudaError_t run_m(const GemvArgs4& a, cudaStream_t s) {
  const DevInfo& d = dev_info();
  for (int top = 8 * NBMAX; top >= 1; top = top > 8 ? top - 8 : top / 2) {
    const int rows = cdiv(a.M, top), cols = cdiv(a.M, rows), nb = cdiv(cols, 8);
    Plan P;
    if (!choose(a, nb, cols, d, &P)) continue;
    switch (nb) {
      case 1: return run<GROUP, 1>(a, P, s);
      case 2: return run<GROUP, 2>(a, P, s);
      case 3: return run<GROUP, 3>(a, P, s);
      default: return run<GROUP, 4>(a, P, s);
    }
  }
  return cudaErrorInvalidConfiguration;    // not reached: one column of MAX_K fits
}

cudaError_t launch_w4_gemv(const GemvArgs4& a, cudaStream_t s) {
  if (a.group == 32) return run_m<32>(a, s);
  if (a.group == 64) return run_m<64>(a, s);
  return run_m<128>(a, s);
}

}  // namespace w4
}  // namespace qmv
