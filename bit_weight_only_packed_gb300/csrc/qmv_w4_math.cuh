// qmv_w4_math.cuh -- what the products of 4-bit weights share: a warp's tensor instructions, its
// part of a packed block, copies, and the scaling of bf16 columns (qmv_w4_gemv.cuh says why).
#pragma once
#include "qmv_pipe.cuh"
#include "qmv_step.cuh"

namespace qmv {
namespace w4 {

// Where a warp's partial sum of (column m, row) lies: the rows of a column are
// swapped in eights by column pair, so that the lanes of a warp touch different
// banks both as the products leave them and row by row.
__device__ __forceinline__ int part_at(int m, int row) { return m * ROWS + (row ^ (((m >> 1) & 3) << 3)); }

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

}  // namespace w4
}  // namespace qmv
