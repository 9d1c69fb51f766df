// qmv_step.cuh -- declarations of the verification-step operators: the 4-bit
// matvec with group scales and zero points (qmv_w4.cu), the norms between two
// blocks (qmv_norm.cu), and logits to probabilities to accepted tokens
// (qmv_sample.cu).  Arguments are checked in qmv_step_abi.cu.
#pragma once
#include <cuda_bf16.h>

#include "qmv_internal.cuh"

#define QMV_W4_MAGIC 0x514D3450u

struct qmv_w4pack {
  uint32_t magic;
  int N, K, group, scale_bf16, zeros;
  int G;                      // groups per row: ceil(K / group)
  size_t bytes;
  const uint8_t* d_packed;    // bound by qmv_w4_pack or qmv_w4_bind
};

namespace qmv {
namespace w4 {

// The packed layout (qmv.h): blocks of ROWS x BK codes, strips of ROWS rows,
// the blocks of a strip one after another in k.
constexpr int ROWS = 32, BK = 128, CODE_BYTES = ROWS * BK / 2;
// The longest row: an eighth of one column of x fits beside the rings.
constexpr int MAX_K = 131072;

__host__ __device__ constexpr int block_bytes(int group, bool zeros) {
  return CODE_BYTES + (BK / group) * ROWS * (zeros ? 3 : 2);
}
__host__ __device__ constexpr int cdiv(int a, int b) { return (a + b - 1) / b; }

// The bit of a 32-bit word where code i of its eight begins: the low halves hold
// codes 0, 4, 2, 6 at bits 3, 7, 11 and 15 (wrapping around), the high halves
// their odd neighbours.
__host__ __device__ constexpr int shift_of(int i) {
  return (3 + 8 * ((i >> 1) & 1) + 4 * (i >> 2) + 16 * (i & 1)) & 31;
}

// Where row r (0..31) of a block keeps its scale and zero point inside a
// group's 32: the four rows that one lane of a warp holds (g, g + 8, g + 16,
// g + 24 for g = lane / 4) lie side by side.
__host__ __device__ constexpr int meta_slot(int r) { return (r & 7) * 4 + (r >> 3); }

struct GemvArgs4 {
  const uint8_t* packed;
  int N, K, scale_bf16, group, zeros;
  int M;
  const void* x;
  int ldx, x_bf16;
  void* y;
  int ldy, y_dtype;
  int early;                  // the weights may be read before the kernel before has ended
};

cudaError_t launch_w4_pack(const qmv_w4pack& p, const uint8_t* codes, const uint16_t* scales,
                           const uint8_t* zeros, uint8_t* packed, cudaStream_t s);
cudaError_t launch_w4_unpack(const qmv_w4pack& p, uint8_t* codes, cudaStream_t s);
cudaError_t launch_w4_gemv(const GemvArgs4& a, cudaStream_t s);
template <int GROUP, bool SB>
cudaError_t launch_group(const GemvArgs4& a, cudaStream_t s);
template <int GROUP, bool SB>
cudaError_t read_error(int clear, int* out);

}  // namespace w4

struct NormArgs {
  int M, D;
  const void* y;
  int ldy, y_dtype;
  const void* r;
  int ldr;
  const void *gamma_post, *gate;
  int ldg;
  float rs, bs;
  const void* gamma_pre;
  float goff, eps;
  void* h;
  int ldh;
  void* out;
  int ldo;
  int bf16;
};
cudaError_t launch_block_norm(const NormArgs& a, cudaStream_t s);

struct SoftmaxArgs {
  int rows, V;
  const void* x;
  int ldx, dtype;
  const float* t;
  float t0;
  float* out;
  int ldo;
};
cudaError_t launch_softmax(const SoftmaxArgs& a, cudaStream_t s);

struct VerifyArgs {
  int B, S, V;
  const float *p, *q;
  const int *draft, *n_draft;
  const float *ua, *us;
  int *tokens, *n_acc;
};
cudaError_t launch_verify(const VerifyArgs& a, cudaStream_t s);

// A launch on s in clusters of `cluster` CTAs along x, as a programmatic
// dependent of the kernel before it: its CTAs may start while that one still
// drains, and every kernel launched here waits for it (griddepcontrol.wait)
// before it touches global memory, so that only the launch itself overlaps.  Each lets
// its own dependents start after that wait and not before, so what runs early runs ahead
// of one kernel only: all before that one have ended.  Three read something before their
// wait, and so need a kernel right before them that waits before it lets them start:
//   the matvec with early weights (qmv_set_pdl): packed weights, by bulk copies;
//   the experts' products behind the kernel that makes x: ids (ld_early) and packed weights, by bulk copies;
//   the sums of the experts' products: ids and their weights (ld_early).
// None of these is what the kernel right before writes.  Ids and their weights change at every
// step, in place, so they are read from L2, where all that has ended has left its writes.
// (43008x5376 for one token, call after call: 28.7 us without, 25.8 us with.)
template <typename... P, typename... A>
inline cudaError_t launch_step(void (*kern)(P...), dim3 grid, int threads, size_t smem, cudaStream_t s, int cluster,
                               A... args) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  int n = 0;
  if (cluster > 1) {
    attr[n].id = cudaLaunchAttributeClusterDimension;
    attr[n].val.clusterDim.x = cluster;
    attr[n].val.clusterDim.y = 1;
    attr[n].val.clusterDim.z = 1;
    ++n;
  }
  attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[n].val.programmaticStreamSerializationAllowed = 1;
  ++n;
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = n;
  return cudaLaunchKernelEx(&cfg, kern, args...);
}

// Waits for the kernel before, then lets the next one of the stream start.  (The other way
// round, call after call: verification of 1 x 4 tokens 5.6 for 5.8 us, softmax of 5 x 262144
// 4.9 for 4.6, the norms and the matvec the same.)
__device__ __forceinline__ void pdl_begin() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// Clusters: a barrier of all their threads, and a CTA's shared memory as the others see it.
__device__ __forceinline__ void cluster_arrive() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
// For warps that publish nothing (no fence; what they read must have arrived).
__device__ __forceinline__ void cluster_arrive_relaxed() {
  asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t cluster_addr(const void* p, int rank) {
  uint32_t d;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(d) : "r"((uint32_t)__cvta_generic_to_shared(p)), "r"(rank));
  return d;
}
__device__ __forceinline__ uint32_t ld_cluster32(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
  return v;
}
// Stores to another CTA's shared memory that complete on its mbarrier `bar`.
__device__ __forceinline__ void st_async128(uint32_t to, uint32_t bar, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.v4.b32 [%0], {%1, %2, %3, %4}, [%5];" ::"r"(to),
               "r"(a), "r"(b), "r"(c), "r"(d), "r"(bar)
               : "memory");
}
__device__ __forceinline__ void st_async64(uint32_t to, uint32_t bar, long long v) {
  asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.b64 [%0], %1, [%2];" ::"r"(to), "l"(v), "r"(bar)
               : "memory");
}

// The device error words of the 4-bit matvec and of softmax and verification (bounded waits).
int read_w4_error(int clear, int* out);
int read_sample_error(int clear, int* out);

// 16-bit elements as fp32 and back (round to nearest even).
template <typename T>
__device__ __forceinline__ float to_f(T v);
template <>
__device__ __forceinline__ float to_f<float>(float v) { return v; }
template <>
__device__ __forceinline__ float to_f<__half>(__half v) { return __half2float(v); }
template <>
__device__ __forceinline__ float to_f<__nv_bfloat16>(__nv_bfloat16 v) { return __bfloat162float(v); }
template <typename T>
__device__ __forceinline__ T from_f(float v);
template <>
__device__ __forceinline__ float from_f<float>(float v) { return v; }
template <>
__device__ __forceinline__ __half from_f<__half>(float v) { return __float2half_rn(v); }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

}  // namespace qmv
