// qmv_step_abi.cu -- the C ABI of the verification-step operators declared in
// include/qmv.h: argument checks on the host and dispatch to the kernels.
#include <new>

#include "qmv_span.cuh"
#include "qmv_step.cuh"

using namespace qmv::span_of;

namespace {

bool pack_ok(const qmv_w4pack* p) { return p && p->magic == QMV_W4_MAGIC; }
bool dtype16(int d) { return d == QMV_F16 || d == QMV_BF16; }
bool dtype_ok(int d) { return d == QMV_F32 || dtype16(d); }
size_t dsize(int d) { return d == QMV_F32 ? 4 : 2; }

int done(cudaError_t e) { return e == cudaSuccess ? QMV_OK : qmv::record_cuda_error(e); }

}  // namespace

extern "C" {

int qmv_w4_create(qmv_w4pack** out, int N, int K, int group, int scale_dtype, int has_zeros,
                  size_t* packed_bytes) {
  if (!out) return QMV_ERR_INVALID_ARG;
  *out = nullptr;
  if (group != 32 && group != 64 && group != 128) return QMV_ERR_INVALID_ARG;
  if (!dtype16(scale_dtype)) return QMV_ERR_INVALID_ARG;
  // strips are counted in int; the padded size must not pass it
  if (N < 1 || K < 32 || K % 32 != 0 || N > INT32_MAX - 31)
    return QMV_ERR_SHAPE;
  if (K > qmv::w4::MAX_K) return QMV_ERR_UNSUPPORTED;
  qmv_w4pack* p = new (std::nothrow) qmv_w4pack;
  if (!p) return QMV_ERR_INVALID_ARG;
  memset(p, 0, sizeof(*p));
  p->magic = QMV_W4_MAGIC;
  p->N = N;
  p->K = K;
  p->group = group;
  p->scale_bf16 = scale_dtype == QMV_BF16;
  p->zeros = has_zeros != 0;
  p->G = qmv::w4::cdiv(K, group);
  p->bytes = (size_t)qmv::w4::cdiv(N, qmv::w4::ROWS) * (size_t)qmv::w4::cdiv(K, qmv::w4::BK) *
             (size_t)qmv::w4::block_bytes(group, p->zeros != 0);
  if (packed_bytes) *packed_bytes = p->bytes;
  *out = p;
  return QMV_OK;
}

int qmv_w4_pack(qmv_w4pack* p, const uint8_t* d_codes_in, const void* d_scales_in,
                const uint8_t* d_zeros_in, void* d_packed, void* stream) {
  if (!pack_ok(p) || !d_codes_in || !d_scales_in || !d_packed) return QMV_ERR_INVALID_ARG;
  if ((d_zeros_in != nullptr) != (p->zeros != 0)) return QMV_ERR_INVALID_ARG;
  if (!aligned(d_codes_in, 8) || !aligned(d_scales_in, 2) || !aligned(d_packed, 16))
    return QMV_ERR_ALIGNMENT;
  if (meets(flat(d_packed, p->bytes, 1), flat(d_codes_in, (int64_t)p->N * p->K, 1),
            flat(d_scales_in, (int64_t)p->N * p->G, 2), flat(d_zeros_in, (int64_t)p->N * p->G, 1)))
    return QMV_ERR_INVALID_ARG;
  const cudaError_t e = qmv::w4::launch_w4_pack(*p, d_codes_in, (const uint16_t*)d_scales_in,
                                                d_zeros_in, (uint8_t*)d_packed, (cudaStream_t)stream);
  if (e != cudaSuccess) return qmv::record_cuda_error(e);
  p->d_packed = (const uint8_t*)d_packed;
  return QMV_OK;
}

int qmv_w4_bind(qmv_w4pack* p, void* d_packed) {
  if (!pack_ok(p) || !d_packed) return QMV_ERR_INVALID_ARG;
  if (!aligned(d_packed, 16)) return QMV_ERR_ALIGNMENT;
  p->d_packed = (const uint8_t*)d_packed;
  return QMV_OK;
}

int qmv_w4_unpack(const qmv_w4pack* p, uint8_t* d_codes_out, void* stream) {
  if (!pack_ok(p) || !p->d_packed || !d_codes_out) return QMV_ERR_INVALID_ARG;
  if (meet(flat(d_codes_out, (int64_t)p->N * p->K, 1), flat(p->d_packed, p->bytes, 1))) return QMV_ERR_INVALID_ARG;
  return done(qmv::w4::launch_w4_unpack(*p, d_codes_out, (cudaStream_t)stream));
}

int qmv_w4_info(const qmv_w4pack* p, int* N, int* K, int* group, int* scale_dtype, int* has_zeros) {
  if (!pack_ok(p)) return QMV_ERR_INVALID_ARG;
  if (N) *N = p->N;
  if (K) *K = p->K;
  if (group) *group = p->group;
  if (scale_dtype) *scale_dtype = p->scale_bf16 ? QMV_BF16 : QMV_F16;
  if (has_zeros) *has_zeros = p->zeros;
  return QMV_OK;
}

int qmv_w4_destroy(qmv_w4pack* p) {
  if (!pack_ok(p)) return QMV_ERR_INVALID_ARG;
  p->magic = 0;
  delete p;
  return QMV_OK;
}

int qmv_w4_gemv(const qmv_w4pack* p, int M, const void* x, int ldx, int x_dtype, void* y, int ldy,
                int y_dtype, void* stream) {
  if (!pack_ok(p) || !p->d_packed || !x || !y) return QMV_ERR_INVALID_ARG;
  if (M < 1 || M > 4096 || !dtype16(x_dtype) || !dtype_ok(y_dtype)) return QMV_ERR_INVALID_ARG;
  if (ldx < p->K || ldy < p->N) return QMV_ERR_SHAPE;
  if (!aligned(x, 2) || !aligned(y, dsize(y_dtype))) return QMV_ERR_ALIGNMENT;
  if (meets(span(y, M, ldy, p->N, dsize(y_dtype)), span(x, M, ldx, p->K, 2), flat(p->d_packed, p->bytes, 1)))
    return QMV_ERR_INVALID_ARG;
  qmv::w4::GemvArgs4 a;
  a.packed = p->d_packed;
  a.N = p->N;
  a.K = p->K;
  a.scale_bf16 = p->scale_bf16;
  a.group = p->group;
  a.zeros = p->zeros;
  a.M = M;
  a.x = x;
  a.ldx = ldx;
  a.x_bf16 = x_dtype == QMV_BF16;
  a.y = y;
  a.ldy = ldy;
  a.y_dtype = y_dtype;
  a.early = qmv::pdl_enabled();
  return done(qmv::w4::launch_w4_gemv(a, (cudaStream_t)stream));
}

int qmv_block_norm(int M, int D, const void* y, int ldy, int y_dtype, const void* residual, int ldr,
                   const void* gamma_post, const void* gate, int ldg, float residual_scale,
                   float branch_scale, const void* gamma_pre, float gamma_offset, float eps,
                   void* h_out, int ldh, void* out, int ldo, int dtype, void* stream) {
  if (!y || !residual || !gamma_pre || !out || M < 1 || D < 1) return QMV_ERR_INVALID_ARG;
  if (!dtype_ok(y_dtype) || !dtype16(dtype) || !(eps >= 0.0f)) return QMV_ERR_INVALID_ARG;
  if (D > 65536) return QMV_ERR_UNSUPPORTED;
  if (ldy < D || ldr < D || ldo < D || (h_out && ldh < D) || (gate && ldg != 0 && ldg < D))
    return QMV_ERR_SHAPE;
  if (h_out == residual && ldh != ldr) return QMV_ERR_SHAPE;
  if (out == y || out == residual || out == h_out || h_out == y || out == gate) return QMV_ERR_INVALID_ARG;
  if (!aligned(y, dsize(y_dtype)) || !aligned(residual, 2) || !aligned(gamma_post, 2) ||
      !aligned(gate, 2) || !aligned(gamma_pre, 2) || !aligned(h_out, 2) || !aligned(out, 2))
    return QMV_ERR_ALIGNMENT;
  const Span h = span(h_out, M, ldh, D, 2), o = span(out, M, ldo, D, 2), in = span(y, M, ldy, D, dsize(y_dtype)),
             res = span(residual, M, ldr, D, 2), gt = ldg ? span(gate, M, ldg, D, 2) : flat(gate, D, 2),
             g1 = flat(gamma_pre, D, 2), g2 = flat(gamma_post, D, 2);
  if (meets(o, in, res, gt, g1, g2, h) || meets(h, in, gt, g1, g2) || (h_out != residual && meet(h, res)))
    return QMV_ERR_INVALID_ARG;
  qmv::NormArgs a{M, D, y, ldy, y_dtype, residual, ldr, gamma_post, gate, ldg, residual_scale,
                  branch_scale, gamma_pre, gamma_offset, eps, h_out, ldh, out, ldo,
                  dtype == QMV_BF16};
  return done(qmv::launch_block_norm(a, (cudaStream_t)stream));
}

int qmv_softmax(int rows, int V, const void* logits, int ldl, int dtype, const float* d_temperature,
                float temperature, float* out, int ldo, void* stream) {
  if (!logits || !out || rows < 1 || V < 1 || !dtype_ok(dtype)) return QMV_ERR_INVALID_ARG;
  if (!d_temperature && !(temperature >= 0.0f)) return QMV_ERR_INVALID_ARG;
  if (ldl < V || ldo < V || ((const void*)out == logits && (ldo != ldl || dtype != QMV_F32)))
    return QMV_ERR_SHAPE;
  if (!aligned(logits, dsize(dtype)) || !aligned(out, 4) || !aligned(d_temperature, 4))
    return QMV_ERR_ALIGNMENT;
  const Span o = span(out, rows, ldo, V, 4);
  if (meet(o, flat(d_temperature, rows, 4)) ||
      ((const void*)out != logits && meet(o, span(logits, rows, ldl, V, dsize(dtype)))))
    return QMV_ERR_INVALID_ARG;
  qmv::SoftmaxArgs a{rows, V, logits, ldl, dtype, d_temperature, temperature, out, ldo};
  return done(qmv::launch_softmax(a, (cudaStream_t)stream));
}

int qmv_verify_draft(int B, int S, int V, const float* target, const float* draft_probs,
                     const int* draft, const int* n_draft, const float* u_accept,
                     const float* u_sample, int* tokens, int* n_accepted, void* stream) {
  if (!target || !u_sample || !tokens || !n_accepted || B < 1 || S < 0 || V < 1)
    return QMV_ERR_INVALID_ARG;
  if (S > 0 && (!draft || !u_accept)) return QMV_ERR_INVALID_ARG;
  // V bounds the integer total below 2^62; B is a grid dimension
  if (B > 65535 || S > 1024 || V > (1 << 20)) return QMV_ERR_UNSUPPORTED;
  if (!aligned(target, 4) || !aligned(draft_probs, 4) || !aligned(draft, 4) || !aligned(n_draft, 4) ||
      !aligned(u_accept, 4) || !aligned(u_sample, 4) || !aligned(tokens, 4) || !aligned(n_accepted, 4))
    return QMV_ERR_ALIGNMENT;
  const int64_t drafted = (int64_t)B * S;
  const Span in[] = {flat(target, (drafted + B) * V, 4), flat(u_sample, B, 4), flat(n_draft, B, 4),
                     flat(S ? draft_probs : nullptr, drafted * V, 4), flat(S ? draft : nullptr, drafted, 4),
                     flat(S ? u_accept : nullptr, drafted, 4)};
  const Span to = flat(tokens, drafted + B, 4), na = flat(n_accepted, B, 4);
  bool shared = meet(to, na);
  for (const Span& i : in) shared = shared || meets(i, to, na);
  if (shared) return QMV_ERR_INVALID_ARG;
  qmv::VerifyArgs a{B, S, V, target, draft_probs, draft, n_draft, u_accept, u_sample, tokens, n_accepted};
  return done(qmv::launch_verify(a, (cudaStream_t)stream));
}

}  // extern "C"
