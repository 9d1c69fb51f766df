// qmv_token_abi.cu -- the C ABI of the decode-step operators declared in include/qmv.h:
// argument checks on the host, rotary frequencies, and dispatch to the kernels.
#include <math.h>

#include "qmv_span.cuh"
#include "qmv_token.cuh"

using namespace qmv::span_of;

namespace {

bool dtype16(int d) { return d == QMV_F16 || d == QMV_BF16; }
bool dtype_ok(int d) { return d == QMV_F32 || dtype16(d); }
size_t dsize(int d) { return d == QMV_F32 ? 4 : 2; }
int done(cudaError_t e) { return e == cudaSuccess ? QMV_OK : qmv::record_cuda_error(e); }

// The experts of a pack in rows of R, or 0 where it does not hold whole ones.
int experts_of(const qmv_w4pack* p, int R) {
  return R > 0 && R % qmv::w4::ROWS == 0 && p->N % R == 0 ? p->N / R : 0;
}

bool experts_fit(const qmv_w4pack* p, int E, int M, int T) {
  return M <= 4096 && T <= 64 && (int64_t)M * T <= qmv::EXPERTS_MAX_PAIRS && E <= qmv::EXPERTS_MAX_E &&
         p->K <= qmv::EXPERTS_MAX_K && p->N / E <= qmv::EXPERTS_MAX_R;
}

// form: the workspace has to hold this call's own scratch only.
int experts_call(const qmv_w4pack* p, int rows_per_expert, int M, int T, const int* ids, const float* weights, const void* x,
                 int ldx, int per_pair, int x_dtype, int act, void* y, int ldy, int y_dtype, void* d_workspace,
                 size_t workspace_bytes, bool form, void* stream) {
  if (!p || p->magic != QMV_W4_MAGIC || !p->d_packed || !ids || !x || !y || M < 1 || T < 1) return QMV_ERR_INVALID_ARG;
  if (!dtype16(x_dtype) || !dtype_ok(y_dtype) || act < QMV_ACT_NONE || act > QMV_ACT_GELU) return QMV_ERR_INVALID_ARG;
  const int E = experts_of(p, rows_per_expert), R = rows_per_expert;
  if (!E) return QMV_ERR_SHAPE;
  if (!experts_fit(p, E, M, T)) return QMV_ERR_UNSUPPORTED;
  const int width = act == QMV_ACT_NONE ? p->K : 2 * p->K;
  if (ldx < width || ldy < R) return QMV_ERR_SHAPE;
  const qmv::ExpertsArgs a{p->d_packed, p->K, p->scale_bf16, p->group, p->zeros, E, R, M, T, ids, weights, x, ldx, per_pair != 0,
                           x_dtype == QMV_BF16, act, y, ldy, y_dtype, d_workspace};
  const size_t need = form ? qmv::experts_workspace(a) : qmv::experts_workspace(p->K, R, M, T);
  if (!aligned(ids, 4) || !aligned(weights, 4) || !aligned(x, 2) || !aligned(y, dsize(y_dtype)) ||
      (need && d_workspace && !aligned(d_workspace, 256)))
    return QMV_ERR_ALIGNMENT;
  if (need && (!d_workspace || workspace_bytes < need)) return QMV_ERR_WORKSPACE;
  const int64_t pairs = (int64_t)M * T;
  const Span in = span(x, per_pair ? pairs : M, ldx, width, 2), i = flat(ids, pairs, 4), w = flat(weights, pairs, 4),
             packed = flat(p->d_packed, p->bytes, 1), out = span(y, weights ? M : pairs, ldy, R, dsize(y_dtype)),
             ws = flat(need ? d_workspace : nullptr, need, 1);
  if (meets(out, in, i, w, packed, ws) || meets(ws, in, i, w, packed)) return QMV_ERR_INVALID_ARG;
  return done(qmv::launch_experts(a, (cudaStream_t)stream));
}
constexpr float NO_WEIGHT = 0.0f;          // stands for weights in a question for sizes

}  // namespace

extern "C" {

int qmv_rope_inv_freq(int rot, double base, int scaling, double factor, double original_length, double beta_fast,
                      double beta_slow, double* inv_freq, float* amplitude) {
  if (!inv_freq || !(base > 1.0) || !(base <= 1e300) || scaling < QMV_SCALE_NONE || scaling > QMV_SCALE_YARN)
    return QMV_ERR_INVALID_ARG;
  if (scaling != QMV_SCALE_NONE && (!(factor > 0.0) || !(factor <= 1e100))) return QMV_ERR_INVALID_ARG;
  if (rot < 2 || rot > 1024 || rot % 2 != 0 || (scaling == QMV_SCALE_NTK && rot == 2)) return QMV_ERR_SHAPE;
  if (scaling == QMV_SCALE_NTK) base *= pow(factor, (double)rot / (rot - 2));
  double lo = 0.0, hi = 0.0;
  float amp = 1.0f;
  if (scaling == QMV_SCALE_YARN) {
    if (!(original_length > 0.0) || !(beta_fast > 0.0) || !(beta_slow > 0.0) || !isfinite(original_length) ||
        !isfinite(beta_fast) || !isfinite(beta_slow))
      return QMV_ERR_INVALID_ARG;
    // the pair that turns so many times in the original length
    const auto pair_of = [&](double turns) { return rot * log(original_length / (turns * 2.0 * M_PI)) / (2.0 * log(base)); };
    lo = fmax(floor(pair_of(beta_fast)), 0.0);
    hi = fmin(ceil(pair_of(beta_slow)), (double)rot - 1.0);
    if (factor > 1.0) amp = (float)(0.1 * log(factor) + 1.0);
  }
  for (int i = 0; i < rot / 2; ++i) {
    double w = pow(base, -2.0 * i / rot);
    if (scaling == QMV_SCALE_LINEAR) w /= factor;
    if (scaling == QMV_SCALE_YARN) {
      const double r = fmin(fmax((i - lo) / fmax(hi - lo, 1e-3), 0.0), 1.0);
      w = w / factor * r + w * (1.0 - r);
    }
    inv_freq[i] = w;
  }
  if (amplitude) *amplitude = amp;
  return QMV_OK;
}

int qmv_rope_turns(int n, const double* inv_freq, int64_t* turns) {
  if (n < 1 || !inv_freq || !turns) return QMV_ERR_INVALID_ARG;
  for (int i = 0; i < n; ++i)
    if (!isfinite(inv_freq[i])) return QMV_ERR_INVALID_ARG;
  for (int i = 0; i < n; ++i) {
    const double t = inv_freq[i] / (2.0 * M_PI), part = t - floor(t);
    // 2^64 * part fits unless part was rounded up to a whole turn
    turns[i] = part >= 1.0 ? 0 : (int64_t)(uint64_t)ldexp(part, 64);
  }
  return QMV_OK;
}

int qmv_qk_norm_rope(int M, int n_q, int n_k, int D, const void* qkv, int ld, int x_dtype, const int* positions,
                     const int64_t* turns, int rot, int layout, float amplitude, const void* gamma_q,
                     const void* gamma_k, float gamma_offset, float eps, void* q, int ldq, void* k, int ldk, int dtype,
                     void* stream) {
  if (!qkv || M < 1 || n_q < 0 || n_k < 0 || (n_q == 0 && n_k == 0) || D < 1) return QMV_ERR_INVALID_ARG;
  if ((q != nullptr) != (n_q > 0) || (k != nullptr) != (n_k > 0)) return QMV_ERR_INVALID_ARG;
  if (!dtype_ok(x_dtype) || !dtype16(dtype) || !(eps >= 0.0f)) return QMV_ERR_INVALID_ARG;
  if (layout != QMV_ROPE_HALF && layout != QMV_ROPE_INTERLEAVED) return QMV_ERR_INVALID_ARG;
  if ((positions != nullptr) != (rot != 0) || (turns != nullptr) != (rot != 0)) return QMV_ERR_INVALID_ARG;
  if (n_q > 4096 || n_k > 4096 || D > 1024) return QMV_ERR_UNSUPPORTED;
  if (rot < 0 || rot > D || rot % 2 != 0) return QMV_ERR_SHAPE;
  const int wq = n_q * D, wk = n_k * D;
  if (ld < wq + wk || (q && ldq < wq) || (k && ldk < wk)) return QMV_ERR_SHAPE;
  const size_t xs = dsize(x_dtype);
  if (!aligned(qkv, xs) || !aligned(q, 2) || !aligned(k, 2) || !aligned(gamma_q, 2) || !aligned(gamma_k, 2) ||
      !aligned(positions, 4) || !aligned(turns, 8))
    return QMV_ERR_ALIGNMENT;
  const Span in = span(qkv, M, ld, wq + wk, xs), gq = flat(gamma_q, D, 2), gk = flat(gamma_k, D, 2),
             ps = flat(positions, M, 4), tn = flat(turns, rot / 2, 8), oq = span(q, M, ldq, wq, 2),
             ok = span(k, M, ldk, wk, 2);
  // each head is read whole before it is written, so it may stay where it is
  const bool q_stays = q == qkv && dtype == x_dtype && (M == 1 || ldq == ld),
             k_stays = k && k == (const char*)qkv + (size_t)wq * xs && dtype == x_dtype && (M == 1 || ldk == ld);
  if (meets(oq, gq, gk, ps, tn, ok) || meets(ok, gq, gk, ps, tn) || (!q_stays && meet(oq, in)) || (!k_stays && meet(ok, in)))
    return QMV_ERR_INVALID_ARG;
  qmv::RopeArgs a{M, n_q, n_k, D, qkv, ld, x_dtype, positions, turns, rot, layout, amplitude, gamma_q, gamma_k,
                  gamma_offset, eps, q, ldq, k, ldk, dtype == QMV_BF16};
  return done(qmv::launch_rope(a, (cudaStream_t)stream));
}

int qmv_route(int M, int E, int T, const void* logits, int ldl, int dtype, int score, const float* bias, int groups,
              int group_k, int group_top, int renormalise, float scale, int* ids, float* weights, void* stream) {
  if (!logits || !ids || !weights || M < 1 || E < 1 || T < 1 || !dtype_ok(dtype)) return QMV_ERR_INVALID_ARG;
  if (score != QMV_SCORE_SOFTMAX && score != QMV_SCORE_SIGMOID) return QMV_ERR_INVALID_ARG;
  if (groups < 1 || group_k < 1 || (group_top != 1 && group_top != 2)) return QMV_ERR_INVALID_ARG;
  if (E > 1024 || T > 64 || groups > 32) return QMV_ERR_UNSUPPORTED;
  if (E % groups != 0 || group_k > groups || T > group_k * (E / groups) || (groups > 1 && group_top > E / groups) || ldl < E)
    return QMV_ERR_SHAPE;
  if (!aligned(logits, dsize(dtype)) || !aligned(bias, 4) || !aligned(ids, 4) || !aligned(weights, 4))
    return QMV_ERR_ALIGNMENT;
  const Span in = span(logits, M, ldl, E, dsize(dtype)), b = flat(bias, E, 4), oi = flat(ids, (int64_t)M * T, 4),
             ow = flat(weights, (int64_t)M * T, 4);
  if (meets(oi, in, b, ow) || meets(ow, in, b)) return QMV_ERR_INVALID_ARG;
  qmv::RouteArgs a{M, E, T, logits, ldl, dtype, score, bias, groups, group_k, group_top, renormalise != 0, scale, ids, weights,
                   E / groups, E == groups ? 0 : (uint32_t)(((uint64_t)1 << 32) / (E / groups) + 1)};
  return done(qmv::launch_route(a, (cudaStream_t)stream));
}

size_t qmv_w4_experts_workspace_bytes(const qmv_w4pack* p, int rows_per_expert, int M, int T) {
  if (!p || p->magic != QMV_W4_MAGIC || M < 1 || T < 1) return 0;
  const int E = experts_of(p, rows_per_expert);
  if (!E || !experts_fit(p, E, M, T)) return 0;
  return qmv::experts_workspace(p->K, rows_per_expert, M, T);
}

size_t qmv_w4_experts_form_bytes(const qmv_w4pack* p, int rows_per_expert, int M, int T, int weighted, const void* x, int ldx,
                                 int per_pair, int x_dtype, int act) {
  if (qmv_w4_experts_workspace_bytes(p, rows_per_expert, M, T) == 0) return 0;
  qmv::ExpertsArgs a = {};
  a.K = p->K, a.R = rows_per_expert, a.M = M, a.T = T;
  a.weights = weighted ? &NO_WEIGHT : nullptr;
  a.x = x, a.ldx = ldx, a.per_pair = per_pair != 0, a.x_bf16 = x_dtype == QMV_BF16, a.act = act;
  return qmv::experts_workspace(a);
}

int qmv_w4_experts(const qmv_w4pack* p, int rows_per_expert, int M, int T, const int* ids, const float* weights,
                   const void* x, int ldx, int per_pair, int x_dtype, int act, void* y, int ldy, int y_dtype,
                   void* d_workspace, size_t workspace_bytes, void* stream) {
  return experts_call(p, rows_per_expert, M, T, ids, weights, x, ldx, per_pair, x_dtype, act, y, ldy, y_dtype, d_workspace,
                      workspace_bytes, false, stream);
}

int qmv_w4_experts_form(const qmv_w4pack* p, int rows_per_expert, int M, int T, const int* ids, const float* weights,
                        const void* x, int ldx, int per_pair, int x_dtype, int act, void* y, int ldy, int y_dtype,
                        void* d_workspace, size_t workspace_bytes, void* stream) {
  return experts_call(p, rows_per_expert, M, T, ids, weights, x, ldx, per_pair, x_dtype, act, y, ldy, y_dtype, d_workspace,
                      workspace_bytes, true, stream);
}

int qmv_sample(int rows, int V, const void* logits, int ldl, int dtype, const float* d_temperature, float temperature,
               const int* d_top_k, int top_k, const float* d_top_p, float top_p, const float* d_min_p, float min_p,
               const float* u, int* tokens, void* stream) {
  if (!logits || !u || !tokens || rows < 1 || V < 1 || !dtype_ok(dtype)) return QMV_ERR_INVALID_ARG;
  if ((!d_temperature && !(temperature >= 0.0f)) || (!d_top_k && top_k < 0) ||
      (!d_top_p && !(top_p >= 0.0f && top_p <= 1.0f)) || (!d_min_p && !(min_p >= 0.0f && min_p <= 1.0f)))
    return QMV_ERR_INVALID_ARG;
  if (V > (1 << 20)) return QMV_ERR_UNSUPPORTED;         // the whole sum stays below 2^62
  if (ldl < V) return QMV_ERR_SHAPE;
  if (!aligned(logits, dsize(dtype)) || !aligned(d_temperature, 4) || !aligned(d_top_k, 4) || !aligned(d_top_p, 4) ||
      !aligned(d_min_p, 4) || !aligned(u, 4) || !aligned(tokens, 4))
    return QMV_ERR_ALIGNMENT;
  if (meets(flat(tokens, rows, 4), span(logits, rows, ldl, V, dsize(dtype)), flat(d_temperature, rows, 4),
            flat(d_top_k, rows, 4), flat(d_top_p, rows, 4), flat(d_min_p, rows, 4), flat(u, rows, 4)))
    return QMV_ERR_INVALID_ARG;
  qmv::DrawArgs a{rows, V, logits, ldl, dtype, d_temperature, temperature, d_top_k, top_k, d_top_p, top_p, d_min_p, min_p, u, tokens};
  return done(qmv::launch_draw(a, (cudaStream_t)stream));
}

}  // extern "C"
