// kda_qk_api.cpp -- C ABI of the query / key preparation (include/kda.h, kda_qk_norm_rope*).
#include <stddef.h>
#include <stdint.h>

#include "../../include/kda.h"
#include "kda_check.h"
#include "kda_qk.h"

namespace {

int check_qk(const kda_qk_shape* s, int* es) {
  if (!s) return KDA_ERR_NULL;
  if (s->dtype != KDA_BF16 && s->dtype != KDA_F32) return KDA_ERR_DTYPE;
  if (s->tokens < 0 || s->q_heads < 1 || s->k_heads < 0 || s->d < 1) return KDA_ERR_SHAPE;
  if (s->q_heads > 65535 || s->k_heads > 65535 || s->tokens >= (int64_t(1) << 28))
    return KDA_ERR_SHAPE;
  if (!supported_width(s->d)) return KDA_ERR_UNSUPPORTED;
  if (s->norm < KDA_NORM_NONE || s->norm > KDA_NORM_L2) return KDA_ERR_UNSUPPORTED;
  if (!(s->eps >= 0.f)) return KDA_ERR_SHAPE;
  if (s->rotary_dim < 0 || s->rotary_dim > s->d) return KDA_ERR_SHAPE;
  if (s->rotary_dim % 16 != 0) return KDA_ERR_UNSUPPORTED;
  if (s->rotary_dim > 0) {
    if (s->n_axes < 1 || s->n_axes > 4) return KDA_ERR_UNSUPPORTED;
    int sum = 0;
    for (int i = 0; i < s->n_axes; ++i) {
      if (s->sections[i] < 0 || s->sections[i] > s->rotary_dim) return KDA_ERR_SHAPE;
      sum += s->sections[i];
    }
    if (sum != s->rotary_dim / 2) return KDA_ERR_SHAPE;
  }
  *es = s->dtype == KDA_BF16 ? 2 : 4;
  const int64_t ev = 16 / *es;  // rows move in 16-byte vectors
  const int64_t qd = (int64_t)s->q_heads * s->d, kd = (int64_t)s->k_heads * s->d;
  if (s->q_stride != 0 && (s->q_stride < qd || s->q_stride > (int64_t(1) << 31))) return KDA_ERR_SHAPE;
  if (s->k_stride != 0 && (s->k_stride < kd || s->k_stride > (int64_t(1) << 31))) return KDA_ERR_SHAPE;
  if (s->q_stride % ev != 0 || s->k_stride % ev != 0) return KDA_ERR_ALIGN;
  return KDA_OK;
}

int64_t span(int64_t tokens, int64_t stride, int64_t row, int es) {
  return tokens > 0 ? ((tokens - 1) * stride + row) * es : 0;
}

struct QkPtrs {
  const void *q, *k;
  const float *wq, *wk;
  const double* inv;
  const void* pos;
  void *oq, *ok;  // outputs (backward: dq, dk)
  // backward
  const void *dyq = nullptr, *dyk = nullptr;
  float *dwq = nullptr, *dwk = nullptr;
  void* ws = nullptr;
  size_t ws_bytes = 0;
};

size_t partial_bytes(const kda_qk_shape& s) { return (size_t)kda::kQkMaxBlocks * 2 * s.d * 4; }

int run(const kda_qk_shape* shape, const QkPtrs& p, bool bwd, void* stream) {
  int es = 0;
  int rc = check_qk(shape, &es);
  if (rc) return rc;
  const kda_qk_shape& s = *shape;
  // the forward's blocks hold 2048 / d tokens each, the last one whole: a launch counts 2^32 - 1 threads at most
  if (!bwd && (s.tokens + 2048 / s.d - 1) / (2048 / s.d) * 256 > 0xFFFFFFFFll) return KDA_ERR_SHAPE;
  const int64_t qd = (int64_t)s.q_heads * s.d, kd = (int64_t)s.k_heads * s.d;
  const int64_t qs = s.q_stride ? s.q_stride : qd, ks = s.k_stride ? s.k_stride : kd;
  const bool any = s.tokens > 0, keys = s.k_heads > 0;
  if (any) {
    if (!p.q || !p.oq || (keys && (!p.k || !p.ok))) return KDA_ERR_NULL;
    if (s.rotary_dim > 0 && (!p.inv || !p.pos)) return KDA_ERR_NULL;
    if (bwd && (!p.dyq || (keys && !p.dyk))) return KDA_ERR_NULL;
  }
  if ((p.dwq && !p.wq) || (p.dwk && !p.wk)) return KDA_ERR_NULL;
  for (const void* x : {p.q, p.k, p.dyq, p.dyk, (const void*)p.oq, (const void*)p.ok})
    if (x && misaligned(x)) return KDA_ERR_ALIGN;
  if (misaligned(p.wq, 4) || misaligned(p.wk, 4) || misaligned(p.inv, 8) || misaligned(p.pos, s.positions_64 ? 8 : 4) ||
      misaligned(p.dwq, 4) || misaligned(p.dwk, 4))
    return KDA_ERR_ALIGN;
  const bool sums = bwd && (p.dwq || p.dwk);
  const size_t need = sums ? partial_bytes(s) : 0;
  if (sums) {
    if (!p.ws) return KDA_ERR_NULL;
    if (p.ws_bytes < need) return KDA_ERR_WORKSPACE;
    if (misaligned(p.ws, 256)) return KDA_ERR_ALIGN;
  }
  const Range in[] = {range_of(p.q, p.q ? span(s.tokens, qs, qd, es) : 0),
                      range_of(p.k, p.k ? span(s.tokens, ks, kd, es) : 0),
                      range_of(p.dyq, p.dyq ? s.tokens * qd * es : 0), range_of(p.dyk, p.dyk ? s.tokens * kd * es : 0),
                      range_of(p.wq, p.wq ? s.d * 4 : 0), range_of(p.wk, p.wk ? s.d * 4 : 0),
                      range_of(p.inv, p.inv ? s.rotary_dim * 4 : 0),
                      range_of(p.pos, p.pos ? (int64_t)s.n_axes * s.tokens * (s.positions_64 ? 8 : 4) : 0)};
  const Range out[] = {range_of(p.oq, p.oq ? s.tokens * qd * es : 0), range_of(p.ok, p.ok ? s.tokens * kd * es : 0),
                       range_of(p.dwq, p.dwq ? s.d * 4 : 0), range_of(p.dwk, p.dwk ? s.d * 4 : 0),
                       range_of(p.ws, (int64_t)need)};
  // in place: a row is read whole before it is written, by the lanes that write it
  const bool in_q = p.oq == p.q && qs == qd, in_k = p.ok == p.k && ks == kd;
  const bool in_dyq = bwd && p.oq == p.dyq, in_dyk = bwd && p.ok == p.dyk;
  for (int i = 0; i < 5; ++i) {
    for (int j = 0; j < 8; ++j) {
      const bool same = (i == 0 && ((j == 0 && in_q) || (j == 2 && in_dyq))) ||
                        (i == 1 && ((j == 1 && in_k) || (j == 3 && in_dyk)));
      if (!same && overlap(out[i], in[j])) return KDA_ERR_ALIAS;
    }
    for (int j = i + 1; j < 5; ++j)
      if (overlap(out[i], out[j])) return KDA_ERR_ALIAS;
  }
  kda::QkArgs a;
  a.q = {p.q, p.dyq, p.oq, p.wq, p.dwq, s.q_heads, qs};
  a.k = {p.k, p.dyk, p.ok, p.wk, p.dwk, s.k_heads, ks};
  a.tokens = s.tokens;
  a.d = s.d;
  a.norm = s.norm;
  a.eps = s.eps;
  a.w_offset = s.weight_offset;
  a.rotary = s.rotary_dim;
  a.interleaved = s.interleaved != 0;
  a.axes = s.n_axes;
  int end = 0;
  for (int i = 0; i < 4; ++i) {
    end += s.rotary_dim > 0 && i < s.n_axes ? s.sections[i] : 0;
    a.ends[i] = s.rotary_dim > 0 && i < s.n_axes - 1 ? end : (1 << 30);  // past the last axis: never reached
  }
  a.inv = p.inv;
  a.pos = p.pos;
  a.pos64 = s.positions_64 != 0;
  a.bf16 = s.dtype == KDA_BF16;
  a.partial = sums ? (float*)p.ws : nullptr;
  a.stream = stream;
  if (!any && !sums) return KDA_OK;  // with weights, their gradients are written as zeros
  return (bwd ? kda::launch_qk_bwd(a) : kda::launch_qk(a)) == hipSuccess ? KDA_OK : KDA_ERR_HIP;
}

}  // namespace

extern "C" {

int kda_qk_norm_rope(const kda_qk_shape* shape, const void* q, const void* k, const float* q_weight,
                     const float* k_weight, const double* inv_freq, const void* positions, void* q_out, void* k_out,
                     void* stream) {
  const QkPtrs p{q, k, q_weight, k_weight, inv_freq, positions, q_out, k_out};
  return run(shape, p, false, stream);
}

size_t kda_qk_norm_rope_bwd_workspace_size(const kda_qk_shape* shape) {
  int es = 0;
  return check_qk(shape, &es) == KDA_OK ? partial_bytes(*shape) : 0;
}

int kda_qk_norm_rope_bwd(const kda_qk_shape* shape, const void* d_q_out, const void* d_k_out, const void* q,
                         const void* k, const float* q_weight, const float* k_weight, const double* inv_freq,
                         const void* positions, void* dq, void* dk, float* d_q_weight, float* d_k_weight,
                         void* workspace, size_t workspace_bytes, void* stream) {
  const QkPtrs p{q,       k,       q_weight,   k_weight,   inv_freq,  positions,      dq, dk,
                 d_q_out, d_k_out, d_q_weight, d_k_weight, workspace, workspace_bytes};
  return run(shape, p, true, stream);
}

}  // extern "C"
