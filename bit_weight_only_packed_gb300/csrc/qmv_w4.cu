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

// ------------------------------------------------------------------ matvec --

__device__ __forceinline__ void bulk_g2s(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                   pipe::sa(dst)),
               "l"(src), "r"(bytes), "r"(pipe::sa(bar))
               : "memory");
}

constexpr int WARPS = 8, NT = WARPS * 32, MAX_SLOTS = 3;
constexpr int PART_LD = 36;     // floats between the columns of a warp's sums: no bank conflicts

// Eight activations of a column, k .. k + 7, as the tensor cores take them.
__device__ __forceinline__ uint4 load_x8(const uint16_t* p, bool vec) {
  if (vec) return *reinterpret_cast<const uint4*>(p);
  uint32_t v[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) v[e] = (uint32_t)p[2 * e] | ((uint32_t)p[2 * e + 1] << 16);
  return make_uint4(v[0], v[1], v[2], v[3]);
}

// One CTA a strip of 32 rows and 8 * NB columns; warp w takes blocks w, w + 8,
// ... of the strip's k through a ring of its own: lane 0 keeps `slots` bulk
// copies in flight, one block each, and refills a slot as soon as its codes are
// in registers.  Warps meet only once, to add their sums.
template <bool BF16, int GROUP, int NB>
__global__ void __launch_bounds__(NT) gemv_kernel(GemvArgs4 a, int slots, int vec) {
  constexpr int GPB = BK / GROUP, HPG = GROUP / 32;      // groups a block, 32-k steps a group
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ uint64_t full[WARPS][MAX_SLOTS];
  __shared__ int abort_flag;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int KB = cdiv(a.K, BK), strip = blockIdx.x, m0 = blockIdx.y * 8 * NB;
  const int bb = block_bytes(GROUP, a.zeros != 0);
  const int n = warp < KB ? (KB - warp + WARPS - 1) / WARPS : 0;
  const uint8_t* src = a.packed + ((int64_t)strip * KB + warp) * bb;
  uint8_t* ring = smem + (size_t)warp * slots * bb;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (threadIdx.x == 0) abort_flag = 0;
  if (lane == 0) {
    for (int i = 0; i < slots; ++i) pipe::mbar_init(&full[warp][i], 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    for (int i = 0; i < slots && i < n; ++i) {
      pipe::mbar_arrive_tx(&full[warp][i], bb);
      bulk_g2s(ring + i * bb, src + (int64_t)i * WARPS * bb, bb, &full[warp][i]);
    }
  }
  __syncthreads();
  asm volatile("griddepcontrol.wait;" ::: "memory");     // x may come from the kernel before
  const uint16_t* x = (const uint16_t*)a.x + (int64_t)(m0 + g) * a.ldx + 8 * t;
  float tot[2][NB][4] = {};
  int slot = 0, parity = 0, i = 0;
  for (; i < n; ++i) {
    const int k0 = (warp + i * WARPS) * BK;
    uint4 xv[4][NB];
#pragma unroll
    for (int st = 0; st < 4; ++st)
#pragma unroll
      for (int c = 0; c < NB; ++c) {
        xv[st][c] = make_uint4(0, 0, 0, 0);
        if (m0 + 8 * c + g < a.M && k0 + 32 * st + 8 * t < a.K)
          xv[st][c] = load_x8(x + (int64_t)(8 * c) * a.ldx + k0 + 32 * st, vec);
      }
    if (!pipe::mbar_wait_fast(&full[warp][slot], parity, &abort_flag, pipe::ERR_TIMEOUT_FULL, &g_w4_error)) break;
    const uint8_t* blk = ring + slot * bb;
    uint4 w[2][2];
#pragma unroll
    for (int r = 0; r < 2; ++r)
#pragma unroll
      for (int j = 0; j < 2; ++j) w[r][j] = *reinterpret_cast<const uint4*>(blk + ((r * 2 + j) * 32 + lane) * 16);
    const uint8_t* meta = blk + CODE_BYTES;
    uint2 sc[GPB];
    uint32_t zp[GPB];
#pragma unroll
    for (int gi = 0; gi < GPB; ++gi) {
      sc[gi] = *reinterpret_cast<const uint2*>(meta + 2 * (gi * ROWS + g * 4));
      zp[gi] = a.zeros ? *reinterpret_cast<const uint32_t*>(meta + 2 * GPB * ROWS + gi * ROWS + g * 4) : 0x08080808u;
    }
    __syncwarp();
    if (lane == 0 && i + slots < n) {
      pipe::mbar_arrive_tx(&full[warp][slot], bb);
      bulk_g2s(ring + slot * bb, src + (int64_t)(i + slots) * WARPS * bb, bb, &full[warp][slot]);
    }
    if (++slot == slots) slot = 0, parity ^= 1;
#pragma unroll
    for (int gi = 0; gi < GPB; ++gi) {
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        uint32_t lo[2], hi[2];     // rows g and g + 8 of the half
        zero_consts<BF16>((zp[gi] >> (16 * r)) & 255u, lo[0], hi[0]);
        zero_consts<BF16>((zp[gi] >> (16 * r + 8)) & 255u, lo[1], hi[1]);
        float acc[NB][4] = {};
#pragma unroll
        for (int hh = 0; hh < HPG; ++hh) {
          const int st = gi * HPG + hh, j = st >> 1, h = st & 1;   // 32 k of the block
          uint32_t p[4], q[4];
          decode<BF16>(h ? w[r][j].y : w[r][j].x, lo[0], hi[0], p);
          decode<BF16>(h ? w[r][j].w : w[r][j].z, lo[1], hi[1], q);
#pragma unroll
          for (int c = 0; c < NB; ++c) {
            mma16816<BF16>(acc[c], p[0], q[0], p[1], q[1], xv[st][c].x, xv[st][c].y);
            mma16816<BF16>(acc[c], p[2], q[2], p[3], q[3], xv[st][c].z, xv[st][c].w);
          }
        }
        const uint32_t s2 = r ? sc[gi].y : sc[gi].x;
        const float s0 = scale_f(s2 & 0xffffu, a.scale_bf16), s1 = scale_f(s2 >> 16, a.scale_bf16);
#pragma unroll
        for (int c = 0; c < NB; ++c) {
          tot[r][c][0] = fmaf(s0, acc[c][0], tot[r][c][0]);
          tot[r][c][1] = fmaf(s0, acc[c][1], tot[r][c][1]);
          tot[r][c][2] = fmaf(s1, acc[c][2], tot[r][c][2]);
          tot[r][c][3] = fmaf(s1, acc[c][3], tot[r][c][3]);
        }
      }
    }
  }
  // a wait that ran out: let the copies in flight land before the CTA ends
  if (i < n && lane == 0)
    for (int j = i; j < n && j < i + slots; ++j) {
      pipe::mbar_drain(&full[warp][slot], parity, &g_w4_error);
      if (++slot == slots) slot = 0, parity ^= 1;
    }
  __syncthreads();                 // every copy has been read: the rings hold the sums now
  if (abort_flag) return;
  float* part = reinterpret_cast<float*>(smem);
  float* mine = part + warp * (8 * NB * PART_LD);
  const int cols = min(8 * NB, a.M - m0);
#pragma unroll
  for (int r = 0; r < 2; ++r)
#pragma unroll
    for (int c = 0; c < NB; ++c)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int col = 8 * c + 2 * t + (e & 1);
        if (col < cols) mine[col * PART_LD + 16 * r + 8 * (e >> 1) + g] = tot[r][c][e];
      }
  __syncthreads();
  for (int o = threadIdx.x; o < 32 * cols; o += NT) {
    const int row = o & 31, m = o >> 5;
    const int64_t nn = (int64_t)strip * ROWS + row;
    if (nn >= a.N) continue;
    float v = 0.0f;
#pragma unroll
    for (int w = 0; w < WARPS; ++w) v += part[(w * 8 * NB + m) * PART_LD + row];
    store_y(a.y, (int64_t)(m0 + m) * a.ldy + nn, a.y_dtype, v);
  }
}

template <bool BF16, int GROUP, int NB>
static cudaError_t run(const GemvArgs4& a, cudaStream_t s) {
  static thread_local KernCache c;
  const int KB = cdiv(a.K, BK), bb = block_bytes(GROUP, a.zeros != 0);
  const int per = cdiv(KB, WARPS), slots = per < MAX_SLOTS ? per : MAX_SLOTS;
  size_t smem = (size_t)WARPS * slots * bb;
  const size_t part = (size_t)WARPS * 8 * NB * PART_LD * sizeof(float);
  if (part > smem) smem = part;
  const cudaError_t e = prep_kernel(gemv_kernel<BF16, GROUP, NB>, c, NT, smem, nullptr);
  if (e != cudaSuccess) return e;
  const int vec = a.ldx % 8 == 0 && (uintptr_t)a.x % 16 == 0;
  return launch_step(gemv_kernel<BF16, GROUP, NB>, dim3(cdiv(a.N, ROWS), cdiv(a.M, 8 * NB)), NT, smem, s, 1, a,
                     slots, vec);
}

template <bool BF16, int GROUP>
static cudaError_t run_m(const GemvArgs4& a, cudaStream_t s) {
  if (a.M <= 8) return run<BF16, GROUP, 1>(a, s);
  if (a.M <= 16) return run<BF16, GROUP, 2>(a, s);
  return run<BF16, GROUP, 4>(a, s);
}

template <bool BF16>
static cudaError_t run_g(const GemvArgs4& a, cudaStream_t s) {
  if (a.group == 32) return run_m<BF16, 32>(a, s);
  if (a.group == 64) return run_m<BF16, 64>(a, s);
  return run_m<BF16, 128>(a, s);
}

cudaError_t launch_w4_gemv(const GemvArgs4& a, cudaStream_t s) {
  return a.x_bf16 ? run_g<true>(a, s) : run_g<false>(a, s);
}

}  // namespace w4
}  // namespace qmv
