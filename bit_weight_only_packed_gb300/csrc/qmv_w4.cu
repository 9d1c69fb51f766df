// qmv_w4.cu -- 4-bit weights with a scale and a zero point a group:
//   y[m][n] = sum_g s[n][g] * sum_{k in g} x[m][k] * (q[n][k] - z[n][g]).
//
// The packed layout is the order in which the tensor cores read the weights:
// one 16-byte word of a lane holds, for a 16-row half and 64 k, the codes of
// rows g and g + 8 (g = lane / 4) at k = 32 h + 8 t + 0..7 (t = lane % 4,
// h = 0, 1), so the words of a warp are 512 consecutive bytes and no code
// moves between lanes.  Inside a 32-bit word the pairs (k, k + 1) lie at the
// same bits of the two halves: (0, 1) at bit 3, (4, 5) at 7, (2, 3) at 11 and
// (6, 7) at 15, wrapping around.  One mask, after a rotation of the word, yields
// a pair in place for the matvec's operand: fp16 reads a code at bit 3 or 7
// evenly spaced.
#include "qmv_step.cuh"

namespace qmv {

namespace w4 {

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
      {
        const uint32_t v = ((e < 4 ? c.x : c.y) >> (8 * (e & 3))) & 15u;
        w[q] |= __funnelshift_l(v, v, shift_of(e));
      }
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
    codes[i] = (uint8_t)(__funnelshift_r(w, w, shift_of(k & 7)) & 15u);
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

cudaError_t launch_w4_gemv(const GemvArgs4& a, cudaStream_t s) {
  if (a.group == 32) return a.scale_bf16 ? launch_group<32, true>(a, s) : launch_group<32, false>(a, s);
  if (a.group == 64) return a.scale_bf16 ? launch_group<64, true>(a, s) : launch_group<64, false>(a, s);
  return a.scale_bf16 ? launch_group<128, true>(a, s) : launch_group<128, false>(a, s);
}

}  // namespace w4

int read_w4_error(int clear, int* out) {
  cudaError_t (*const read[])(int, int*) = {w4::read_error<32, false>, w4::read_error<32, true>,
                                            w4::read_error<64, false>, w4::read_error<64, true>,
                                            w4::read_error<128, false>, w4::read_error<128, true>};
  *out = 0;
  for (const auto f : read) {
    int v = 0;
    const cudaError_t e = f(clear, &v);
    if (e != cudaSuccess) return (int)e;
    if (v) *out = v;
  }
  return 0;
}

}  // namespace qmv
