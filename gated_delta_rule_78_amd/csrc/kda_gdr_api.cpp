// kda_gdr_api.cpp -- C ABI of the gated delta rule with one decay per head (include/kda.h, kda_gdr_*):
// argument checks on the host, then the kernels' launches.
#include <stddef.h>
#include <stdint.h>
#include <stdlib.h>

#include <algorithm>

#include "../../include/kda.h"
#include "kda_check.h"
#include "kda_gdr.h"

namespace {

size_t up(size_t x) { return (x + 255) / 256 * 256; }

int check_gdr_shape(const kda_shape* s, int qk_heads, bool decode, int n_seqs, int* es) {
  if (!s) return KDA_ERR_NULL;
  if (s->dtype != KDA_BF16 && s->dtype != KDA_F32) return KDA_ERR_DTYPE;
  if (s->B < 0 || s->H < 1 || s->H > 65535 || qk_heads < 1 || s->dk < 1 || s->dv < 1 || s->T < 0) return KDA_ERR_SHAPE;
  if (s->H % qk_heads != 0) return KDA_ERR_SHAPE;
  if (n_seqs >= 0 && (s->B != 1 || n_seqs > (1 << 24))) return KDA_ERR_SHAPE;
  if (too_many_rows(s->B, s->T, s->H)) return KDA_ERR_SHAPE;
  if (!supported_width(s->dk) || !supported_width(s->dv)) return KDA_ERR_UNSUPPORTED;
  if (!decode && s->chunk != 0 && s->chunk != 64) return KDA_ERR_UNSUPPORTED;
  *es = s->dtype == KDA_BF16 ? 2 : 4;
  return KDA_OK;
}

struct Plan {
  int L;  // chunks of a segment
  bool split;
  int64_t nseg, chunks;
  int64_t ends, states;  // segments that another one starts from; with the copies of the caller's start states
};

// KDA_GDR_SEGMENT=n pins the chunks of a segment (tuning aid, and the tests' forced splits).
int segment_override() {
  static const int v = [] {
    const char* e = getenv("KDA_GDR_SEGMENT");
    return e ? atoi(e) : 0;
  }();
  return v;
}

// A chain (sequence, head, 64 value columns) is walked in order.  With few chains it is cut into segments,
// which costs a first pass over all but the last (the value columns and the transfer's, about 0.7 of a
// step each) and the links between them (counted as 1.5 steps each, one after another); a cut is taken where this sum of steps on
// 256 compute units is least.  As it chooses, whole and in segments of 16 chunks: 131,072 tokens, 16 heads 2,205, 5,698 and
// 3,602 us; 8,192 tokens, 16 heads 206, 370 and 206; 2 x 8,192, 32 heads 429, 431 (whole) and 607; 2,048 tokens, 8 heads 103,
// 108 and 113.  Packed chains are cut, or not, where their lengths are known
// (lina_offsets_kernel); L is then the least that their segments may have, a compute unit's share of all steps.
// What a link takes is its product's: 7.5 us at d_k = 128, 1.6 at 64, of a step (bf16 3.0 and 2.0 us, fp32 8.7 and 4.8)
// 2.5, 0.8, 0.9 and 0.35.  1.5 is between them and suits both directions: at 3 the forward of 131,072 tokens, one head, takes
// 577 us instead of 597, the backward 1,537 instead of 1,482.
Plan gdr_plan(const kda_shape& s, int n_seqs) {
  const bool packed = n_seqs >= 0;
  const int nv = s.dv / 64, nk = s.dk / 64;
  const int64_t nch = std::max<int64_t>(1, ((int64_t)s.T + 63) / 64);
  const int64_t n = packed ? n_seqs : s.B, heads = std::max<int64_t>(1, n * s.H);
  int64_t L = nch;
  if (packed) {
    L = std::max<int64_t>(8, ((nch + n) * s.H * nv + 255) / 256);
  } else {
    static const int cuts[] = {1, 2, 3, 4, 6, 8, 12, 16, 24, 32, 48, 64};
    double best = 0.;
    for (int c : cuts) {
      const int64_t len = (nch + c - 1) / c, segs = (nch + len - 1) / len;
      auto rounds = [](int64_t wgs) { return (double)((wgs + 255) / 256); };
      const double t = segs == 1 ? rounds(heads * nv) * nch
                                 : (rounds(heads * (nv + nk) * (segs - 1)) * 0.7 + rounds(heads * nv * segs)) * len + 1.5 * segs + 2.;
      if (c == 1 || t < best) {
        best = t;
        L = len;
      }
    }
  }
  if (segment_override() > 0) L = segment_override();
  L = std::max<int64_t>(1, std::min(L, nch));
  Plan p;
  p.L = (int)L;
  p.split = L < nch;
  p.nseg = packed ? kda::lina_pieces(s.T, n, L) : n * ((nch + L - 1) / L);
  p.chunks = kda::gdr_chunks(packed, s.T, n);
  p.ends = p.split ? kda::lina_ends(packed, s.T, n, L) : 0;
  p.states = kda::lina_seg_states(p.ends, n);
  return p;
}

// A launch counts its threads in 32 bits.
bool launchable(const Plan& p, const kda_shape& s, int qk_heads) {
  const int tiles = (s.dv + s.dk) / 64;
  return ((p.nseg * qk_heads + 7) / 8 * 8) * (s.H / qk_heads) * tiles <= 0xFFFFFFFFll / 512 &&
         p.chunks * ((s.H + 3) / 4) <= 0xFFFFFFFFll / 256 && p.chunks * qk_heads <= 0xFFFFFFFFll / 256;
}

// What either direction's walk needs.
struct Layout {
  Plan plan;
  size_t off_score, off_token, off_seg, off_transfer, off_cs, off_list, bytes;
};

Layout layout(const kda_shape& s, int n_seqs) {
  Layout l;
  l.plan = gdr_plan(s, n_seqs);
  const size_t tri = (size_t)l.plan.chunks * s.H * kda::kTriBlocks * 256 * 4;
  l.off_score = up(tri);
  l.off_token = up(l.off_score + tri);
  l.off_seg = up(l.off_token + (size_t)l.plan.chunks * s.H * kda::kTokenFloats * 4);
  l.off_transfer = up(l.off_seg + (size_t)l.plan.states * s.H * s.dk * s.dv * 4);
  l.off_cs = up(l.off_transfer + (size_t)l.plan.ends * s.H * s.dk * s.dk * 4);
  l.off_list = up(l.off_cs + (n_seqs >= 0 ? ((size_t)n_seqs + 2) * 4 : 0));
  l.bytes = up(l.off_list + (n_seqs >= 0 ? (size_t)l.plan.nseg * 8 : 0));
  return l;
}

// Batch, widths and workspace of a walk; the offsets of a packed batch.
int start(kda::GdrWalk& a, const kda_shape& s, const Layout& l, int n_seqs, const int* cu, char* ws, void* stream) {
  kda::LinaWalk& w = a.walk;
  w.n = n_seqs >= 0 ? n_seqs : s.B;
  w.T = s.T;
  w.H = s.H;
  w.dk = s.dk;
  w.dv = s.dv;
  w.L = l.plan.L;
  w.split = l.plan.split;
  w.bf16 = s.dtype == KDA_BF16;
  w.stream = stream;
  w.seg_state = (float*)(ws + l.off_seg);
  a.inv = (float*)ws;
  a.score = (float*)(ws + l.off_score);
  a.token = (float*)(ws + l.off_token);
  a.transfer = (float*)(ws + l.off_transfer);
  if (n_seqs < 0) return KDA_OK;
  w.cs = (const int*)(ws + l.off_cs);
  w.list = (const int*)(ws + l.off_list);
  // A link against both walks' steps of a segment, in tenths.  One sequence of 131,072 tokens, one head, without and with it:
  // bf16, 128 x 128 1,042 and 576 us, 128 x 64 1,809 and 574, 64 x 64 485 and 265; fp32, 32,768 tokens 620 and 502.
  const int link = segment_override() > 0 ? 0 : s.dk == 128 ? (w.bf16 ? 12 : 5) : (w.bf16 ? 4 : 2);
  // cut chains take three times the steps, so chains of up to 3 shares are walked whole: 20,011 tokens in 24 sequences, 8 heads,
  // the longest 0.15 of them (2.2 shares) 168 us whole, 174 cut, 0.3 (4.5 shares) 292 and 181; 32 heads, one of half (1.8 shares)
  // 523 and 537
  return kda::launch_lina_offsets(cu, n_seqs, s.T, w.L, s.H * (s.dv / 64), (int*)(ws + l.off_cs),
                                  (int*)(ws + l.off_list), stream, 85, link) == hipSuccess
             ? KDA_OK
             : KDA_ERR_HIP;
}

bool walk(const kda::GdrWalk& a, int64_t toks) {
  return (toks == 0 || (kda::launch_gdr_prep(a) == hipSuccess && kda::launch_gdr_segments(a) == hipSuccess)) &&
         kda::launch_gdr_walk(a) == hipSuccess;
}

int fwd_impl(const kda_shape* shape, int Hk, const int* cu, int n_seqs, const void* q, const void* k, const void* v,
             const float* g, const void* beta, const float* s0, void* o, float* sT, void* ws, size_t ws_bytes,
             void* stream) {
  int es = 0;
  int rc = check_gdr_shape(shape, Hk, false, n_seqs, &es);
  if (rc) return rc;
  const kda_shape& s = *shape;
  const bool packed = n_seqs >= 0;
  if (packed && !cu) return KDA_ERR_NULL;
  const int64_t n = packed ? n_seqs : s.B, toks = (int64_t)s.B * s.T;
  if (toks > 0 && (!q || !k || !v || !g || !beta || !o)) return KDA_ERR_NULL;
  for (const void* x : {q, k, v, (const void*)o, (const void*)s0, (const void*)sT})
    if (x && misaligned(x)) return KDA_ERR_ALIGN;
  if (misaligned(g, 4) || misaligned(beta, es) || misaligned(cu, 4)) return KDA_ERR_ALIGN;
  const Layout l = layout(s, n_seqs);
  if (!launchable(l.plan, s, Hk)) return KDA_ERR_SHAPE;
  if (l.bytes > 0 && !ws) return KDA_ERR_NULL;
  if (ws_bytes < l.bytes) return KDA_ERR_WORKSPACE;
  if (misaligned(ws, 256)) return KDA_ERR_ALIGN;
  const int64_t st = n * s.H * s.dk * s.dv * 4;
  const Range in[] = {range_of(q, q ? toks * Hk * s.dk * es : 0), range_of(k, k ? toks * Hk * s.dk * es : 0),
                      range_of(v, v ? toks * s.H * s.dv * es : 0), range_of(g, g ? toks * s.H * 4 : 0),
                      range_of(beta, beta ? toks * s.H * es : 0), range_of(cu, packed ? (int64_t)(n_seqs + 1) * 4 : 0),
                      range_of(s0, s0 ? st : 0)};
  const Range out[] = {range_of(o, o ? toks * s.H * s.dv * es : 0), range_of(sT, sT ? st : 0),
                       range_of(ws, (int64_t)l.bytes)};
  for (int i = 0; i < 3; ++i) {
    for (int j = 0; j < 7; ++j)
      if (overlap(out[i], in[j]) && !(i == 1 && j == 6 && s0 == sT)) return KDA_ERR_ALIAS;
    for (int j = i + 1; j < 3; ++j)
      if (overlap(out[i], out[j])) return KDA_ERR_ALIAS;
  }
  if (n == 0) return KDA_OK;
  kda::GdrWalk a;
  a.beta = beta;
  kda::LinaWalk& w = a.walk;
  w.q = {q, Hk};
  w.k = {k, Hk};
  w.v = {v, s.H};
  w.out = o;
  w.g = g;
  w.s0 = s0;
  w.sT = sT;
  rc = start(a, s, l, n_seqs, cu, (char*)ws, stream);
  if (rc) return rc;
  return walk(a, toks) ? KDA_OK : KDA_ERR_HIP;
}

struct BwdLayout {
  Layout fwd;
  int64_t groups;
  size_t off_r, off_kept, off_kept_r, off_snap, off_anchor, off_a, off_b, off_c, bytes;
};

BwdLayout bwd_layout(const kda_shape& s, int n_seqs) {
  BwdLayout l;
  l.fwd = layout(s, n_seqs);
  const bool packed = n_seqs >= 0;
  const int64_t n = packed ? n_seqs : s.B, toks = (int64_t)s.B * s.T;
  const size_t es = s.dtype == KDA_BF16 ? 2 : 4, state = (size_t)s.H * s.dk * s.dv;
  const int64_t per = 64 * kda::kLinaGroup, keep = kda::lina_keep(s.dtype == KDA_BF16);
  l.groups = packed ? kda::lina_pieces(s.T, n, kda::kLinaGroup) : n * ((s.T + per - 1) / per);
  const int64_t anchors = packed ? kda::lina_pieces(s.T, n, keep) : n * ((s.T + 64 * keep - 1) / (64 * keep));
  const int64_t snaps = kda::lina_ends(packed, s.T, n, keep);
  const size_t chunks = (size_t)l.fwd.plan.chunks, dots = (size_t)toks * s.H * 4 * (s.dv / 64);
  l.off_r = up(l.fwd.bytes);
  l.off_kept = up(l.off_r + (size_t)toks * s.H * s.dv * es);
  l.off_kept_r = up(l.off_kept + chunks * state * es);
  l.off_snap = up(l.off_kept_r + chunks * state * es);
  l.off_anchor = up(l.off_snap + (size_t)snaps * state * 4);
  l.off_a = up(l.off_anchor + (size_t)anchors * s.H * (s.dv / 64) * 4 * 4);
  l.off_b = up(l.off_a + dots);
  l.off_c = up(l.off_b + dots);
  l.bytes = up(l.off_c + dots);
  return l;
}

struct BwdPtrs {
  const void *q, *k, *v;
  const float* g;
  const void* beta;
  const float* s0;
  const void* d_o;
  const float* dsT;
  void *dq, *dk, *dv;
  float* dg;
  void* dbeta;
  float* ds0;
  void* ws;
  size_t ws_bytes;
};

int bwd_impl(const kda_shape* shape, int Hk, const int* cu, int n_seqs, const BwdPtrs& p, void* stream) {
  int es = 0;
  int rc = check_gdr_shape(shape, Hk, false, n_seqs, &es);
  if (rc) return rc;
  const kda_shape& s = *shape;
  const bool packed = n_seqs >= 0;
  if (packed && !cu) return KDA_ERR_NULL;
  const int64_t n = packed ? n_seqs : s.B, toks = (int64_t)s.B * s.T;
  if (toks > 0 && (!p.q || !p.k || !p.v || !p.g || !p.beta || !p.d_o || !p.dq || !p.dk || !p.dv || !p.dbeta))
    return KDA_ERR_NULL;
  for (const void* x : {p.q, p.k, p.v, p.d_o, (const void*)p.s0, (const void*)p.dsT, (const void*)p.dq,
                        (const void*)p.dk, (const void*)p.dv, (const void*)p.ds0})
    if (x && misaligned(x)) return KDA_ERR_ALIGN;
  if (misaligned(p.g, 4) || misaligned(p.dg, 4) || misaligned(p.beta, es) || misaligned(p.dbeta, es) || misaligned(cu, 4))
    return KDA_ERR_ALIGN;
  const BwdLayout l = bwd_layout(s, n_seqs);
  if (!launchable(l.fwd.plan, s, Hk) || l.groups > 0xFFFFFFFFll / kda::kLinaDecayThreads) return KDA_ERR_SHAPE;
  if (l.bytes > 0 && !p.ws) return KDA_ERR_NULL;
  if (p.ws_bytes < l.bytes) return KDA_ERR_WORKSPACE;
  if (misaligned(p.ws, 256)) return KDA_ERR_ALIGN;
  const int64_t st = n * s.H * s.dk * s.dv * 4, qk = toks * Hk * s.dk * es, vo = toks * s.H * s.dv * es;
  const int64_t gb = toks * s.H * 4, bb = toks * s.H * es;
  const Range in[] = {range_of(p.q, p.q ? qk : 0),     range_of(p.k, p.k ? qk : 0),   range_of(p.v, p.v ? vo : 0),
                      range_of(p.g, p.g ? gb : 0),     range_of(p.s0, p.s0 ? st : 0), range_of(p.d_o, p.d_o ? vo : 0),
                      range_of(p.dsT, p.dsT ? st : 0), range_of(p.beta, p.beta ? bb : 0),
                      range_of(cu, packed ? (int64_t)(n_seqs + 1) * 4 : 0)};
  const Range out[] = {range_of(p.dq, p.dq ? qk : 0),   range_of(p.dk, p.dk ? qk : 0),       range_of(p.dv, p.dv ? vo : 0),
                       range_of(p.dg, p.dg ? gb : 0),   range_of(p.dbeta, p.dbeta ? bb : 0), range_of(p.ds0, p.ds0 ? st : 0),
                       range_of(p.ws, (int64_t)l.bytes)};
  for (int i = 0; i < 7; ++i) {
    for (const Range& r : in)
      if (overlap(out[i], r)) return KDA_ERR_ALIAS;
    for (int j = i + 1; j < 7; ++j)
      if (overlap(out[i], out[j])) return KDA_ERR_ALIAS;
  }
  if (n == 0) return KDA_OK;
  char* ws = (char*)p.ws;
  const kda::LinaOp q{p.q, Hk}, k{p.k, Hk}, v{p.v, s.H}, d_o{p.d_o, s.H}, r{ws + l.off_r, s.H};
  kda::GdrWalk f;
  f.beta = p.beta;
  kda::LinaWalk& w = f.walk;
  w.q = q;
  w.k = k;
  w.v = v;
  w.x = d_o;
  w.out = ws + l.off_r;
  w.g = p.g;
  w.s0 = p.s0;
  w.snap = (float*)(ws + l.off_snap);
  w.dots = (float*)(ws + l.off_a);
  f.train = true;
  f.kept = ws + l.off_kept;
  f.r = r;
  rc = start(f, s, l.fwd, n_seqs, cu, ws, stream);
  if (rc) return rc;
  kda::GdrWalk b = f;
  b.walk.v = d_o;
  b.walk.x = v;
  b.walk.out = p.dv;
  b.walk.s0 = p.dsT;
  b.walk.sT = p.ds0;
  b.walk.rev = true;
  b.walk.snap0 = p.s0;
  b.walk.anchor = p.dg ? (float*)(ws + l.off_anchor) : nullptr;
  b.walk.dots = (float*)(ws + l.off_b);
  b.dots2 = (float*)(ws + l.off_c);
  b.kept = ws + l.off_kept_r;
  if (toks == 0) return kda::launch_gdr_walk(b) == hipSuccess ? KDA_OK : KDA_ERR_HIP;
  if (!walk(f, toks) || !walk(b, toks)) return KDA_ERR_HIP;
  kda::GdrGrad gr;
  gr.f = f;
  gr.d_o = d_o;
  gr.y = {p.dv, s.H};
  gr.kept_r = b.kept;
  gr.dots2 = b.dots2;
  gr.dq = p.dq;
  gr.dk = p.dk;
  gr.dbeta = p.dbeta;
  if (kda::launch_gdr_grad(gr) != hipSuccess) return KDA_ERR_HIP;
  // a token's decay scales all that was before it: its gradient falls by do . o - dv . v from token to token
  if (p.dg && kda::launch_lina_ddecay(b.walk, f.walk.dots, b.walk.dots, nullptr, s.dv / 64, 0, b.walk.anchor, p.dg,
                                      nullptr, nullptr) != hipSuccess)
    return KDA_ERR_HIP;
  return KDA_OK;
}

int decode_impl(const kda_shape* shape, int Hk, int ntok, const int* counts, int update, const void* q, const void* k,
                const void* v, const float* g, const void* beta, float* state, void* o, void* stream) {
  if (!shape) return KDA_ERR_NULL;
  if (ntok < 0) return KDA_ERR_SHAPE;
  kda_shape s = *shape;
  s.T = ntok;
  int es = 0;
  int rc = check_gdr_shape(&s, Hk, true, -1, &es);
  if (rc) return rc;
  if ((int64_t)s.B * s.H * (s.dv / 64) > 0xFFFFFFFFll / 512) return KDA_ERR_SHAPE;
  const int64_t toks = (int64_t)s.B * ntok, st = (int64_t)s.B * s.H * s.dk * s.dv * 4;
  if (toks > 0 && (!k || !v || !g || !beta || !state)) return KDA_ERR_NULL;
  if ((q == nullptr) != (o == nullptr) && toks > 0) return KDA_ERR_NULL;
  if (state && misaligned(state)) return KDA_ERR_ALIGN;
  if (misaligned(q, es) || misaligned(k, es) || misaligned(v, es) || misaligned(o, es) || misaligned(beta, es) ||
      misaligned(g, 4) || misaligned(counts, 4))
    return KDA_ERR_ALIGN;
  const Range in[] = {range_of(q, q ? toks * Hk * s.dk * es : 0), range_of(k, k ? toks * Hk * s.dk * es : 0),
                      range_of(v, v ? toks * s.H * s.dv * es : 0), range_of(g, g ? toks * s.H * 4 : 0),
                      range_of(beta, beta ? toks * s.H * es : 0), range_of(counts, counts ? (int64_t)s.B * 4 : 0)};
  const Range ro = range_of(o, o ? toks * s.H * s.dv * es : 0), rs = range_of(state, state ? st : 0);
  for (const Range& r : in)
    if (overlap(ro, r) || overlap(rs, r)) return KDA_ERR_ALIAS;
  if (overlap(ro, rs)) return KDA_ERR_ALIAS;
  if (toks == 0 || (!o && !update)) return KDA_OK;
  const kda::GdrDecodeArgs a{q,    k,   v,  g,    beta, state, counts, update != 0, o, (int64_t)s.B * s.H,
                             ntok, s.H, Hk, s.dk, s.dv, s.dtype == KDA_BF16, stream};
  return kda::launch_gdr_decode(a) == hipSuccess ? KDA_OK : KDA_ERR_HIP;
}

}  // namespace

extern "C" {

size_t kda_gdr_chunk_fwd_workspace_size(const kda_shape* shape) {
  int es = 0;
  return check_gdr_shape(shape, 1, false, -1, &es) == KDA_OK ? layout(*shape, -1).bytes : 0;
}

int kda_gdr_chunk_fwd(const kda_shape* shape, int qk_heads, const void* q, const void* k, const void* v,
                      const float* log_decay, const void* beta, const float* initial_state, void* o,
                      float* final_state, void* workspace, size_t workspace_bytes, void* stream) {
  return fwd_impl(shape, qk_heads, nullptr, -1, q, k, v, log_decay, beta, initial_state, o, final_state, workspace,
                  workspace_bytes, stream);
}

size_t kda_gdr_chunk_fwd_varlen_workspace_size(const kda_shape* shape, int n_seqs) {
  int es = 0;
  return n_seqs >= 0 && check_gdr_shape(shape, 1, false, n_seqs, &es) == KDA_OK ? layout(*shape, n_seqs).bytes : 0;
}

int kda_gdr_chunk_fwd_varlen(const kda_shape* shape, int qk_heads, const int* cu_seqlens, int n_seqs, const void* q,
                             const void* k, const void* v, const float* log_decay, const void* beta,
                             const float* initial_state, void* o, float* final_state, void* workspace,
                             size_t workspace_bytes, void* stream) {
  if (!shape) return KDA_ERR_NULL;
  if (n_seqs < 0) return KDA_ERR_SHAPE;
  return fwd_impl(shape, qk_heads, cu_seqlens, n_seqs, q, k, v, log_decay, beta, initial_state, o, final_state,
                  workspace, workspace_bytes, stream);
}

size_t kda_gdr_chunk_bwd_workspace_size(const kda_shape* shape) {
  int es = 0;
  return check_gdr_shape(shape, 1, false, -1, &es) == KDA_OK ? bwd_layout(*shape, -1).bytes : 0;
}

int kda_gdr_chunk_bwd(const kda_shape* shape, int qk_heads, const void* q, const void* k, const void* v,
                      const float* log_decay, const void* beta, const float* initial_state, const void* d_o,
                      const float* d_final_state, void* dq, void* dk, void* dv, float* d_log_decay, void* d_beta,
                      float* d_initial_state, void* workspace, size_t workspace_bytes, void* stream) {
  const BwdPtrs p{q,  k,  v,  log_decay,   beta,   initial_state,   d_o,       d_final_state,
                  dq, dk, dv, d_log_decay, d_beta, d_initial_state, workspace, workspace_bytes};
  return bwd_impl(shape, qk_heads, nullptr, -1, p, stream);
}

size_t kda_gdr_chunk_bwd_varlen_workspace_size(const kda_shape* shape, int n_seqs) {
  int es = 0;
  return n_seqs >= 0 && check_gdr_shape(shape, 1, false, n_seqs, &es) == KDA_OK ? bwd_layout(*shape, n_seqs).bytes : 0;
}

int kda_gdr_chunk_bwd_varlen(const kda_shape* shape, int qk_heads, const int* cu_seqlens, int n_seqs, const void* q,
                             const void* k, const void* v, const float* log_decay, const void* beta,
                             const float* initial_state, const void* d_o, const float* d_final_state, void* dq,
                             void* dk, void* dv, float* d_log_decay, void* d_beta, float* d_initial_state,
                             void* workspace, size_t workspace_bytes, void* stream) {
  if (!shape) return KDA_ERR_NULL;
  if (n_seqs < 0) return KDA_ERR_SHAPE;
  const BwdPtrs p{q,  k,  v,  log_decay,   beta,   initial_state,   d_o,       d_final_state,
                  dq, dk, dv, d_log_decay, d_beta, d_initial_state, workspace, workspace_bytes};
  return bwd_impl(shape, qk_heads, cu_seqlens, n_seqs, p, stream);
}

int kda_gdr_decode_step(const kda_shape* shape, int qk_heads, const void* q, const void* k, const void* v,
                        const float* log_decay, const void* beta, float* state, void* o, void* stream) {
  return decode_impl(shape, qk_heads, 1, nullptr, 1, q, k, v, log_decay, beta, state, o, stream);
}

int kda_gdr_decode_tokens(const kda_shape* shape, int qk_heads, const int* counts, int update, const void* q,
                          const void* k, const void* v, const float* log_decay, const void* beta, float* state,
                          void* o, void* stream) {
  if (!shape) return KDA_ERR_NULL;
  return decode_impl(shape, qk_heads, shape->T, counts, update, q, k, v, log_decay, beta, state, o, stream);
}

}  // extern "C"
