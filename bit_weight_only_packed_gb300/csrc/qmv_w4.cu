// qmv_w4.cu -- 4-bit weights with a scale and a zero point a group:
//   y[m][n] = sum_g s[n][g] * sum_{k in g} x[m][k] * (q[n][k] - z[n][g]).
//
// The packed layout is the order in which the tensor cores read the weights:
// one 16-byte word of a lane holds, for a 16-row half and 64 k, the codes of
// rows g and g + 8 (g = lane / 4) at k = 32 h + 8 t + 0..7 (t = lane % 4,
// h = 0, 1), so the words of a warp are 512 consecutive bytes and no code
// moves between lanes.  Inside a 32-bit word code i sits at nibble
// i / 2 + 4 * (i % 2), so that one mask yields a pair (k, k + 1).
#include "qmv_step.cuh"

namespace qmv {
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

// ------------------------------------------------------------------ decode --

__device__ __forceinline__ uint32_t and_or(uint32_t w, uint32_t mask, uint32_t magic) {
  return (w & mask) | magic;
}
__device__ __forceinline__ uint32_t hsub2_f16(uint32_t a, uint32_t negz) {
  uint32_t d;
  asm("add.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(negz));
  return d;
}
__device__ __forceinline__ uint32_t hfma2_f16(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t d;
  asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
  return d;
}
__device__ __forceinline__ uint32_t hsub2_bf16(uint32_t a, uint32_t negz) {
  uint32_t d;
  asm("add.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(negz));
  return d;
}

// The constants that take a zero point off, for one row.  fp16: a nibble under
// the exponent of 1024 reads 1024 + q, one nibble higher 1024 + 16 q, so that
// q - z = (1024 + q) - (1024 + z) = (1024 + 16 q) / 16 - (64 + z).  bf16 has 7
// mantissa bits: 128 + q only.  All of these are exact.
template <bool BF16>
__device__ __forceinline__ void zero_consts(uint32_t z, uint32_t& lo, uint32_t& hi) {
  if (BF16) {
    lo = (0xC300u | z) * 0x10001u;
    hi = lo;
  } else {
    lo = (0xE400u | z) * 0x10001u;
    hi = (0xD400u | (z << 4)) * 0x10001u;
  }
}

// The eight codes of a word minus the zero point, as four pairs in k order.
template <bool BF16>
__device__ __forceinline__ void decode(uint32_t w, uint32_t lo, uint32_t hi, uint32_t (&v)[4]) {
  if (BF16) {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = hsub2_bf16(and_or(w >> (4 * i), 0x000f000fu, 0x43004300u), lo);
  } else {
    const uint32_t w8 = w >> 8;
    v[0] = hsub2_f16(and_or(w, 0x000f000fu, 0x64006400u), lo);
    v[1] = hfma2_f16(and_or(w, 0x00f000f0u, 0x64006400u), 0x2c002c00u, hi);
    v[2] = hsub2_f16(and_or(w8, 0x000f000fu, 0x64006400u), lo);
    v[3] = hfma2_f16(and_or(w8, 0x00f000f0u, 0x64006400u), 0x2c002c00u, hi);
  }
}

// D = A . B + D on 16 rows x 8 columns x 16 k, fp32 sums.
template <bool BF16>
__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  if (BF16)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ float scale_f(uint32_t bits16, int bf16) {
  return bf16 ? __uint_as_float(bits16 << 16) : __half2float(__ushort_as_half((unsigned short)bits16));
}

__device__ __forceinline__ void store_y(void* y, int64_t at, int dtype, float v) {
  if (dtype == QMV_F32)
    ((float*)y)[at] = v;
  else if (dtype == QMV_F16)
    ((__half*)y)[at] = __float2half_rn(v);
  else
    ((__nv_bfloat16*)y)[at] = __float2bfloat16_rn(v);
}

// One CTA a strip of 32 rows and 8 columns; its warps take every WARPS-th
// block of k and their sums meet in shared memory.
constexpr int WARPS = 8;

template <bool BF16, int GROUP>
__global__ void __launch_bounds__(WARPS * 32) gemv_kernel(GemvArgs4 a) {
  constexpr int GPB = BK / GROUP, HPG = GROUP / 32;      // groups a block, 32-k steps a group
  __shared__ float part[WARPS][ROWS][8];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int KB = cdiv(a.K, BK), strip = blockIdx.x, m0 = blockIdx.y * 8;
  const int bb = block_bytes(GROUP, a.zeros != 0);
  const uint16_t* x = (const uint16_t*)a.x + (int64_t)(m0 + g) * a.ldx;
  const bool col = m0 + g < a.M;
  float tot[2][4] = {};
  for (int b = warp; b < KB; b += WARPS) {
    const uint8_t* blk = a.packed + ((int64_t)strip * KB + b) * bb;
    const uint8_t* meta = blk + CODE_BYTES;
    uint4 w[2][2];
#pragma unroll
    for (int r = 0; r < 2; ++r)
#pragma unroll
      for (int j = 0; j < 2; ++j) w[r][j] = *reinterpret_cast<const uint4*>(blk + ((r * 2 + j) * 32 + lane) * 16);
#pragma unroll
    for (int gi = 0; gi < GPB; ++gi) {
      const uint2 sc = *reinterpret_cast<const uint2*>(meta + 2 * (gi * ROWS + g * 4));
      uint32_t z = 0x08080808u;
      if (a.zeros) z = *reinterpret_cast<const uint32_t*>(meta + 2 * GPB * ROWS + gi * ROWS + g * 4);
      uint32_t lo[4], hi[4];     // rows g, g + 8, g + 16, g + 24
#pragma unroll
      for (int i = 0; i < 4; ++i) zero_consts<BF16>((z >> (8 * i)) & 255u, lo[i], hi[i]);
      float acc[2][4] = {};
#pragma unroll
      for (int hh = 0; hh < HPG; ++hh) {
        const int step = gi * HPG + hh, j = step >> 1, h = step & 1;   // 32 k of the block
        const int k = b * BK + 32 * step + 8 * t;
        uint32_t xv[4] = {};
        if (col && k < a.K) {
#pragma unroll
          for (int e = 0; e < 4; ++e) xv[e] = (uint32_t)x[k + 2 * e] | ((uint32_t)x[k + 2 * e + 1] << 16);
        }
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          uint32_t p[4], q[4];
          decode<BF16>(h ? w[r][j].y : w[r][j].x, lo[2 * r], hi[2 * r], p);
          decode<BF16>(h ? w[r][j].w : w[r][j].z, lo[2 * r + 1], hi[2 * r + 1], q);
          mma16816<BF16>(acc[r], p[0], q[0], p[1], q[1], xv[0], xv[1]);
          mma16816<BF16>(acc[r], p[2], q[2], p[3], q[3], xv[2], xv[3]);
        }
      }
      const float s[4] = {scale_f(sc.x & 0xffffu, a.scale_bf16), scale_f(sc.x >> 16, a.scale_bf16),
                          scale_f(sc.y & 0xffffu, a.scale_bf16), scale_f(sc.y >> 16, a.scale_bf16)};
#pragma unroll
      for (int r = 0; r < 2; ++r)
#pragma unroll
        for (int i = 0; i < 4; ++i) tot[r][i] = fmaf(s[2 * r + (i >> 1)], acc[r][i], tot[r][i]);
    }
  }
#pragma unroll
  for (int r = 0; r < 2; ++r)
#pragma unroll
    for (int i = 0; i < 4; ++i) part[warp][16 * r + g + 8 * (i >> 1)][2 * t + (i & 1)] = tot[r][i];
  __syncthreads();
  // one thread an output: 32 rows x 8 columns
  const int row = threadIdx.x & 31, m = threadIdx.x >> 5;
  float v = 0.0f;
#pragma unroll
  for (int w = 0; w < WARPS; ++w) v += part[w][row][m];
  const int64_t n = (int64_t)strip * ROWS + row;
  if (n < a.N && m0 + m < a.M) store_y(a.y, (int64_t)(m0 + m) * a.ldy + n, a.y_dtype, v);
}

template <bool BF16>
static void run(const GemvArgs4& a, cudaStream_t s) {
  const dim3 grid(cdiv(a.N, ROWS), cdiv(a.M, 8));
  switch (a.group) {
    case 32: gemv_kernel<BF16, 32><<<grid, WARPS * 32, 0, s>>>(a); break;
    case 64: gemv_kernel<BF16, 64><<<grid, WARPS * 32, 0, s>>>(a); break;
    default: gemv_kernel<BF16, 128><<<grid, WARPS * 32, 0, s>>>(a); break;
  }
}

cudaError_t launch_w4_gemv(const GemvArgs4& a, cudaStream_t s) {
  if (a.x_bf16)
    run<true>(a, s);
  else
    run<false>(a, s);
  return cudaGetLastError();
}

}  // namespace w4
}  // namespace qmv
