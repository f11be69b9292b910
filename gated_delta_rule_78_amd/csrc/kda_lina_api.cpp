// kda_lina_api.cpp -- C ABI of linear attention with a decay per head (include/kda.h,
// kda_lina_*): argument checks on the host, then the walks' launches.
#include <stddef.h>
#include <stdint.h>
#include <stdlib.h>

#include <algorithm>
#include <cmath>

#include "../../include/kda.h"
#include "kda_check.h"
#include "kda_lina.h"

namespace {

size_t up(size_t x) { return (x + 255) / 256 * 256; }

int check_lina_shape(const kda_shape* s, int qk_heads, bool decode, int n_seqs, int* es) {
  if (!s) return KDA_ERR_NULL;
  if (s->dtype != KDA_BF16 && s->dtype != KDA_F32) return KDA_ERR_DTYPE;
  if (s->B < 0 || s->H < 1 || s->H > 65535 || qk_heads < 1 || s->dk < 1 || s->dv < 1 || (!decode && s->T < 0))
    return KDA_ERR_SHAPE;
  if (s->H % qk_heads != 0) return KDA_ERR_SHAPE;
  if (n_seqs >= 0 && (s->B != 1 || n_seqs > (1 << 24))) return KDA_ERR_SHAPE;
  if (too_many_rows(s->B, decode && s->T < 1 ? 1 : s->T, s->H)) return KDA_ERR_SHAPE;
  if (!supported_width(s->dk) || !supported_width(s->dv)) return KDA_ERR_UNSUPPORTED;
  if (!decode && s->chunk != 0 && s->chunk != 64) return KDA_ERR_UNSUPPORTED;
  *es = s->dtype == KDA_BF16 ? 2 : 4;
  return KDA_OK;
}

struct Plan {
  int L;  // chunks of a segment
  bool split;
  bool replay;  // the forward's segments make their start states themselves
  int64_t nseg;
  int64_t ends, states;  // end states of segments; with the kept start states
};

// KDA_LINA_SEGMENT=n pins the chunks of a segment (tuning aid, and the tests' forced splits).
int segment_override() {
  static const int v = [] {
    const char* e = getenv("KDA_LINA_SEGMENT");
    return e ? atoi(e) : 0;
  }();
  return v;
}

// A chain (sequence, head, 64 value columns) is walked in order; with too few chains for the 256 compute
// units it is cut into segments of L chunks, whose start states cost one more read of k and v
// (the segments' end states first, then every segment from its own start).  Measured, us, cut and
// whole, bf16, d = 128, T = 8,192:
//   chains     96         112        128        144        158        176          192          240
//   forward    208, 255   204, 249   210, 239   251, 252   279, 241   347, 267     338, 253     458, 294
//   backward   603, 950   678, 959   715, 953   849, 978   903, 959   1198, 1001   1134, 987    1404, 1030
// (T = 32,768 with 144: 955, 980 and 3249, 3868; with 158: 1059, 939 and 3503, 3766; fp32, d = 64, T = 2,048, with
// 158: 221, 220 and 680, 840; with 192: 304, 221 and 880, 842), so that a forward cuts up to 144 chains and a
// backward up to 160.  Where chains are cut, one segment per compute
// unit (work / 256: 512 chunks of 8 chains 74 us at L = 16, 87 at 8, 90 at 24), or two where
// segments stay long, for the sake of the first pass (128 chunks of 64 chains 115 us at L = 16,
// 116 at 32, 234 whole; 2,048 of 32 chains 860 at 128, 889 at 256, 3,620 whole).  Short segments
// cost their successors a state to add, nch / L of them in a row: with a step of s and an
// addition of f, 2 L s + f nch / L is least at L = sqrt(nch f / 2 s) (64 chunks of 8 chains: 28 us
// at L = 3, 51 at 1, 60 at 16; fp32, 16 chunks: 22.7 us at 1, 45 at 4, 110 whole).  Packed chains
// are cut, or not, where their lengths are known (lina_offsets_kernel): L is the least that their
// segments may have, and half a compute unit's share of the steps is right where one chain is long
// (24 prompts of 20,011 tokens, H = 32, one 0.6 of all: 283 us at 42, half the share; 317 at 80).
// Of the shortest chains every segment makes its start state itself, from the chunks before it,
// which saves the first pass and its launch: bf16, 8 heads, d = 128: 3 chunks 10.3 us against
// 12.9, 8 chunks 16.8 and 17.4, 10 chunks 19.1 and 17.6; fp32, whose steps are dearer, 4 heads,
// d = 64: 3 chunks 16.0 and 17.2, 4 chunks 18.8 and 17.7.
Plan lina_plan(const kda_shape& s, int n_seqs, int nv, int most) {
  const bool packed = n_seqs >= 0;
  const int64_t nch = std::max<int64_t>(1, ((int64_t)s.T + 63) / 64);
  const int64_t n = packed ? n_seqs : s.B;
  const int64_t chains = std::max<int64_t>(1, n * s.H * nv);
  const int64_t work = (packed ? nch + n : nch * n) * s.H * nv;  // chunk steps in all
  int64_t L = nch;
  if (packed || chains <= most) {
    L = (work + 255) / 256;
    if (chains >= 256 || L >= 32) L = (work + 511) / 512;
    L = std::max<int64_t>(L, (int64_t)std::ceil(std::sqrt((double)nch * (s.dtype == KDA_BF16 ? 0.16 : 0.06))));
  }
  if (segment_override() > 0) L = segment_override();
  L = std::max<int64_t>(1, std::min(L, nch));
  Plan p;
  p.L = (int)L;
  p.split = L < nch;
  p.replay = p.split && nch <= (s.dtype == KDA_BF16 ? 8 : 3);
  p.nseg = packed ? kda::lina_pieces(s.T, n, L) : n * ((nch + L - 1) / L);
  p.ends = p.split ? kda::lina_ends(packed, s.T, n, L) : 0;
  p.states = kda::lina_seg_states(p.ends, n);
  return p;
}

// A launch counts its threads in 32 bits: no walk of this plan may have more workgroups.
bool launchable(const Plan& p, const kda_shape& s, int qk_heads, int nv) {
  return ((p.nseg * qk_heads + 7) / 8 * 8) * (s.H / qk_heads) * nv <= 0xFFFFFFFFll / kda::kLinaThreads;
}

struct FwdLayout {
  Plan plan;
  size_t off_dec, off_cs, off_list, bytes;
};

FwdLayout fwd_layout(const kda_shape& s, int n_seqs) {
  FwdLayout l;
  l.plan = lina_plan(s, n_seqs, s.dv / 64, 144);
  const size_t some = l.plan.replay ? 0 : 1;
  l.off_dec = up(some * l.plan.states * s.H * s.dk * s.dv * 4);
  l.off_cs = up(l.off_dec + some * l.plan.ends * s.H * 4);
  l.off_list = up(l.off_cs + (n_seqs >= 0 ? ((size_t)n_seqs + 2) * 4 : 0));
  l.bytes = up(l.off_list + (n_seqs >= 0 ? (size_t)l.plan.nseg * 8 : 0));
  return l;
}

int fwd_impl(const kda_shape* shape, int Hk, const int* cu, int n_seqs, const void* q, const void* k, const void* v,
             const float* g, int per_head, const float* s0, void* o, float* sT, void* ws, size_t ws_bytes,
             void* stream) {
  int es = 0;
  int rc = check_lina_shape(shape, Hk, false, n_seqs, &es);
  if (rc) return rc;
  const kda_shape& s = *shape;
  const bool packed = n_seqs >= 0;
  if (packed && !cu) return KDA_ERR_NULL;
  const int64_t n = packed ? n_seqs : s.B, toks = (int64_t)s.B * s.T;
  if (toks > 0 && (!q || !k || !v || !g || !o)) return KDA_ERR_NULL;
  for (const void* x : {q, k, v, (const void*)o, (const void*)s0, (const void*)sT})
    if (x && misaligned(x)) return KDA_ERR_ALIGN;
  if (misaligned(g, 4) || misaligned(cu, 4)) return KDA_ERR_ALIGN;
  const FwdLayout l = fwd_layout(s, n_seqs);
  if (!launchable(l.plan, s, Hk, s.dv / 64)) return KDA_ERR_SHAPE;
  if (l.bytes > 0 && !ws) return KDA_ERR_NULL;
  if (ws_bytes < l.bytes) return KDA_ERR_WORKSPACE;
  if (misaligned(ws, 256)) return KDA_ERR_ALIGN;
  const int64_t st = n * s.H * s.dk * s.dv * 4;
  const Range in[] = {range_of(q, q ? toks * Hk * s.dk * es : 0), range_of(k, k ? toks * Hk * s.dk * es : 0),
                      range_of(v, v ? toks * s.H * s.dv * es : 0),
                      range_of(g, g ? (per_head ? (int64_t)s.H : toks * s.H) * 4 : 0),
                      range_of(cu, packed ? (int64_t)(n_seqs + 1) * 4 : 0), range_of(s0, s0 ? st : 0)};
  const Range out[] = {range_of(o, o ? toks * s.H * s.dv * es : 0), range_of(sT, sT ? st : 0),
                       range_of(ws, (int64_t)l.bytes)};
  for (int i = 0; i < 3; ++i) {
    for (int j = 0; j < 6; ++j)
      if (overlap(out[i], in[j]) && !(i == 1 && j == 5 && s0 == sT)) return KDA_ERR_ALIAS;
    for (int j = i + 1; j < 3; ++j)
      if (overlap(out[i], out[j])) return KDA_ERR_ALIAS;
  }
  if (n == 0) return KDA_OK;
  char* w = (char*)ws;
  kda::LinaWalk a;
  a.q = {q, Hk};
  a.k = {k, Hk};
  a.v = {v, s.H};
  a.out = o;
  a.g = g;
  a.g_fixed = per_head != 0;
  a.s0 = s0;
  a.sT = sT;
  a.n = (int)n;
  a.T = s.T;
  a.H = s.H;
  a.dk = s.dk;
  a.dv = s.dv;
  a.L = l.plan.L;
  a.split = l.plan.split && !l.plan.replay;
  a.replay = l.plan.replay;
  if (a.replay && s0 && s0 == sT) {  // others would read what the last segment writes: chains whole
    a.L = (s.T + 63) / 64;
    a.replay = false;
  }
  a.seg_state = (float*)w;
  a.seg_dec = (float*)(w + l.off_dec);
  a.bf16 = s.dtype == KDA_BF16;
  a.stream = stream;
  if (packed) {
    a.cs = (const int*)(w + l.off_cs);
    a.list = (const int*)(w + l.off_list);
    if (kda::launch_lina_offsets(cu, n_seqs, s.T, a.L, s.H * (s.dv / 64), (int*)(w + l.off_cs),
                                 (int*)(w + l.off_list), stream) != hipSuccess)
      return KDA_ERR_HIP;
  }
  if (kda::launch_lina_segments(&a, 1) != hipSuccess) return KDA_ERR_HIP;
  return kda::launch_lina_walk(a) == hipSuccess ? KDA_OK : KDA_ERR_HIP;
}

// Workspace of the backward: segment states of the three walks, kept states
// and per-token parts of the decay gradient, the per-head gradients of shared q and k.
struct BwdLayout {
  Plan plan;
  int64_t groups;
  size_t off_dec, off_seg2, off_dec2, off_seg3, off_dec3, off_cs, off_list, off_snap, off_anchor, off_a, off_b, off_e, off_part, off_share, bytes;
};

BwdLayout bwd_layout(const kda_shape& s, int Hk, int n_seqs) {
  BwdLayout l;
  const int64_t n = n_seqs >= 0 ? n_seqs : s.B, toks = (int64_t)s.B * s.T;
  l.plan = lina_plan(s, n_seqs, std::min(s.dk, s.dv) / 64, 160);
  const size_t seg = (size_t)l.plan.states, ends = (size_t)l.plan.ends, state = (size_t)s.H * s.dk * s.dv * 4;
  const int64_t per = 64 * kda::kLinaGroup;
  l.groups = n_seqs >= 0 ? kda::lina_pieces(s.T, n, kda::kLinaGroup) : n * ((s.T + per - 1) / per);
  const int64_t keep = kda::lina_keep(s.dtype == KDA_BF16);
  const int64_t anchors = n_seqs >= 0 ? kda::lina_pieces(s.T, n, keep) : n * ((s.T + 64 * keep - 1) / (64 * keep));
  const int64_t kept = kda::lina_ends(n_seqs >= 0, s.T, n, keep);  // the start of a sequence is the caller's
  l.off_dec = up(seg * state);
  l.off_seg2 = up(l.off_dec + ends * s.H * 4);
  l.off_dec2 = up(l.off_seg2 + seg * state);
  l.off_seg3 = up(l.off_dec2 + ends * s.H * 4);
  l.off_dec3 = up(l.off_seg3 + seg * state);
  l.off_cs = up(l.off_dec3 + ends * s.H * 4);
  l.off_list = up(l.off_cs + (n_seqs >= 0 ? ((size_t)n_seqs + 2) * 4 : 0));
  l.off_snap = up(l.off_list + (n_seqs >= 0 ? (size_t)l.plan.nseg * 8 : 0));
  l.off_anchor = up(l.off_snap + kept * state);
  l.off_a = up(l.off_anchor + (size_t)anchors * s.H * (s.dk / 64) * 4 * 4);
  const size_t dots = (size_t)toks * s.H * 4;
  l.off_b = up(l.off_a + dots * (s.dk / 64));
  l.off_e = up(l.off_b + dots * (s.dk / 64));
  l.off_part = up(l.off_e + dots * (s.dv / 64));
  l.off_share = up(l.off_part + (size_t)l.groups * s.H * 8);
  l.bytes = up(l.off_share + (s.H > Hk ? (size_t)toks * s.H * s.dk * 4 : 0));
  return l;
}

struct BwdPtrs {
  const void *q, *k, *v;
  const float* g;
  int per_head;
  const float* s0;
  const void* d_o;
  const float* dsT;
  void *dq, *dk, *dv;
  float *dg, *ds0;
  void* ws;
  size_t ws_bytes;
};

int bwd_impl(const kda_shape* shape, int Hk, const int* cu, int n_seqs, const BwdPtrs& p, void* stream) {
  int es = 0;
  int rc = check_lina_shape(shape, Hk, false, n_seqs, &es);
  if (rc) return rc;
  const kda_shape& s = *shape;
  const bool packed = n_seqs >= 0;
  if (packed && !cu) return KDA_ERR_NULL;
  const int64_t n = packed ? n_seqs : s.B, toks = (int64_t)s.B * s.T;
  if (toks > 0 && (!p.q || !p.k || !p.v || !p.g || !p.d_o || !p.dq || !p.dk || !p.dv)) return KDA_ERR_NULL;
  for (const void* x : {p.q, p.k, p.v, p.d_o, (const void*)p.s0, (const void*)p.dsT, (const void*)p.dq,
                        (const void*)p.dk, (const void*)p.dv, (const void*)p.ds0})
    if (x && misaligned(x)) return KDA_ERR_ALIGN;
  if (misaligned(p.g, 4) || misaligned(p.dg, 4) || misaligned(cu, 4)) return KDA_ERR_ALIGN;
  const BwdLayout l = bwd_layout(s, Hk, n_seqs);
  if (!launchable(l.plan, s, Hk, std::max(s.dk, s.dv) / 64) || l.groups > 0xFFFFFFFFll / kda::kLinaDecayThreads)
    return KDA_ERR_SHAPE;
  if (l.bytes > 0 && !p.ws) return KDA_ERR_NULL;
  if (p.ws_bytes < l.bytes) return KDA_ERR_WORKSPACE;
  if (misaligned(p.ws, 256)) return KDA_ERR_ALIGN;
  const int64_t st = n * s.H * s.dk * s.dv * 4, qk = toks * Hk * s.dk * es, vo = toks * s.H * s.dv * es;
  const int64_t gb = (p.per_head ? (int64_t)s.H : toks * s.H) * 4;
  const Range in[] = {range_of(p.q, p.q ? qk : 0),   range_of(p.k, p.k ? qk : 0),     range_of(p.v, p.v ? vo : 0),
                      range_of(p.g, p.g ? gb : 0),   range_of(p.s0, p.s0 ? st : 0),   range_of(p.d_o, p.d_o ? vo : 0),
                      range_of(p.dsT, p.dsT ? st : 0), range_of(cu, packed ? (int64_t)(n_seqs + 1) * 4 : 0)};
  const Range out[] = {range_of(p.dq, p.dq ? qk : 0), range_of(p.dk, p.dk ? qk : 0), range_of(p.dv, p.dv ? vo : 0),
                       range_of(p.dg, p.dg ? gb : 0), range_of(p.ds0, p.ds0 ? st : 0),
                       range_of(p.ws, (int64_t)l.bytes)};
  for (int i = 0; i < 6; ++i) {
    for (const Range& r : in)
      if (overlap(out[i], r)) return KDA_ERR_ALIAS;
    for (int j = i + 1; j < 6; ++j)
      if (overlap(out[i], out[j])) return KDA_ERR_ALIAS;
  }
  char* ws = (char*)p.ws;
  kda::LinaWalk a;
  a.g = p.g;
  a.g_fixed = p.per_head != 0;
  a.n = (int)n;
  a.T = s.T;
  a.H = s.H;
  a.L = l.plan.L;
  a.split = l.plan.split;
  a.seg_state = (float*)ws;
  a.seg_dec = (float*)(ws + l.off_dec);
  a.bf16 = s.dtype == KDA_BF16;
  a.stream = stream;
  if (n == 0 || toks == 0) {
    // no token: the start state's gradient is the final state's, a fixed decay's is zero
    if (p.dg && p.per_head && kda::launch_lina_ddecay(a, nullptr, nullptr, nullptr, 0, 0, nullptr, nullptr, nullptr,
                                                      p.dg) != hipSuccess)
      return KDA_ERR_HIP;
    if (n == 0) return KDA_OK;
  }
  if (packed) {
    a.cs = (const int*)(ws + l.off_cs);
    a.list = (const int*)(ws + l.off_list);
    if (kda::launch_lina_offsets(cu, n_seqs, s.T, a.L, s.H * (std::min(s.dk, s.dv) / 64), (int*)(ws + l.off_cs),
                                 (int*)(ws + l.off_list), stream) != hipSuccess)
      return KDA_ERR_HIP;
  }
  const bool shared = s.H > Hk;
  const int* end = packed ? a.cs + n_seqs : nullptr;
  float* share = (float*)(ws + l.off_share);
  float* anchor = (float*)(ws + l.off_anchor);
  float *da = (float*)(ws + l.off_a), *db = (float*)(ws + l.off_b), *de = (float*)(ws + l.off_e);
  const kda::LinaOp q{p.q, Hk}, k{p.k, Hk}, v{p.v, s.H}, u{p.d_o, s.H};
  kda::LinaWalk walks[3] = {a, a, a};
  kda::LinaWalk &wq = walks[0], &wk = walks[1], &wv = walks[2];
  wq.q = u;
  wq.k = v;
  wq.v = k;
  wq.x = q;
  wq.dk = s.dv;
  wq.dv = s.dk;
  wq.out = shared ? (void*)share : p.dq;
  wq.out_f32 = shared;
  wq.s0 = p.s0;
  wq.s_t = true;
  wq.dot = p.dg ? kda::kDotRow : kda::kDotNone;
  wq.dots = da;
  wq.snap = (float*)(ws + l.off_snap);
  wk = wq;
  wk.q = v;
  wk.k = u;
  wk.v = q;
  wk.x = k;
  wk.out = shared ? (void*)share : p.dk;
  wk.s0 = p.dsT;
  wk.rev = true;
  wk.dots = db;
  wk.anchor = anchor;
  wk.snap0 = p.s0;
  wk.seg_state = (float*)(ws + l.off_seg2);
  wk.seg_dec = (float*)(ws + l.off_dec2);
  wv.q = k;  // and the start state's gradient
  wv.k = q;
  wv.v = u;
  wv.x = v;
  wv.dk = s.dk;
  wv.dv = s.dv;
  wv.out = p.dv;
  wv.s0 = p.dsT;
  wv.sT = p.ds0;
  wv.rev = true;
  wv.dot = p.dg && toks > 0 ? kda::kDotCross : kda::kDotNone;
  wv.dots = de;
  wv.seg_state = (float*)(ws + l.off_seg3);
  wv.seg_dec = (float*)(ws + l.off_dec3);
  if (toks == 0) return kda::launch_lina_walk(wv) == hipSuccess ? KDA_OK : KDA_ERR_HIP;
  if (kda::launch_lina_segments(walks, 3) != hipSuccess) return KDA_ERR_HIP;
  auto sum_heads = [&](void* to) {
    return shared ? kda::launch_lina_headsum(share, to, toks, Hk, s.H / Hk, s.dk, a.bf16, end, stream) : hipSuccess;
  };
  // dk after dq, whose kept states it meets; dv with one of them
  const bool fused = a.bf16 && s.dk == s.dv;
  if ((a.bf16 ? kda::launch_lina_walk(wq) : kda::launch_lina_pair(wq, wv)) != hipSuccess || sum_heads(p.dq) != hipSuccess)
    return KDA_ERR_HIP;
  if ((fused ? kda::launch_lina_reverse(wk, wv) : kda::launch_lina_walk(wk)) != hipSuccess ||
      sum_heads(p.dk) != hipSuccess)
    return KDA_ERR_HIP;
  if (a.bf16 && !fused && kda::launch_lina_walk(wv) != hipSuccess) return KDA_ERR_HIP;
  if (p.dg &&
      kda::launch_lina_ddecay(wv, da, db, de, s.dk / 64, s.dv / 64, anchor, p.per_head ? nullptr : p.dg,
                              (double*)(ws + l.off_part), p.per_head ? p.dg : nullptr) != hipSuccess)
    return KDA_ERR_HIP;
  return KDA_OK;
}

int decode_impl(const kda_shape* shape, int Hk, int ntok, const void* q, const void* k, const void* v, const float* g,
                int per_head, float* state, void* o, void* stream) {
  if (!shape) return KDA_ERR_NULL;
  kda_shape s = *shape;
  s.T = ntok;
  int es = 0;
  int rc = check_lina_shape(&s, Hk, true, -1, &es);
  if (rc) return rc;
  if (ntok < 0) return KDA_ERR_SHAPE;
  if ((int64_t)s.B * s.H * (s.dv / 64) > 0xFFFFFFFFll / kda::kLinaDecodeThreads) return KDA_ERR_SHAPE;
  const int64_t toks = (int64_t)s.B * ntok, st = (int64_t)s.B * s.H * s.dk * s.dv * 4;
  if (toks > 0 && (!q || !k || !v || !g || !state || !o)) return KDA_ERR_NULL;
  if (state && misaligned(state)) return KDA_ERR_ALIGN;
  if (misaligned(q, es) || misaligned(k, es) || misaligned(v, es) || misaligned(o, es) || misaligned(g, 4))
    return KDA_ERR_ALIGN;
  const Range in[] = {range_of(q, q ? toks * Hk * s.dk * es : 0), range_of(k, k ? toks * Hk * s.dk * es : 0),
                      range_of(v, v ? toks * s.H * s.dv * es : 0),
                      range_of(g, g ? (per_head ? (int64_t)s.H : toks * s.H) * 4 : 0)};
  const Range ro = range_of(o, o ? toks * s.H * s.dv * es : 0), rs = range_of(state, state ? st : 0);
  for (const Range& r : in)
    if (overlap(ro, r) || overlap(rs, r)) return KDA_ERR_ALIAS;
  if (overlap(ro, rs)) return KDA_ERR_ALIAS;
  if (toks == 0) return KDA_OK;
  const kda::LinaDecodeArgs a{q,    k,    v,  g,    per_head != 0, state, o, (int64_t)s.B * s.H,
                              ntok, s.H, Hk, s.dk, s.dv,          s.dtype == KDA_BF16, stream};
  return kda::launch_lina_decode(a) == hipSuccess ? KDA_OK : KDA_ERR_HIP;
}

}  // namespace

extern "C" {

size_t kda_lina_chunk_fwd_workspace_size(const kda_shape* shape) {
  int es = 0;
  return check_lina_shape(shape, 1, false, -1, &es) == KDA_OK ? fwd_layout(*shape, -1).bytes : 0;
}

int kda_lina_chunk_fwd(const kda_shape* shape, int qk_heads, const void* q, const void* k, const void* v,
                       const float* log_decay, int decay_per_head, const float* initial_state, void* o,
                       float* final_state, void* workspace, size_t workspace_bytes, void* stream) {
  return fwd_impl(shape, qk_heads, nullptr, -1, q, k, v, log_decay, decay_per_head, initial_state, o, final_state,
                  workspace, workspace_bytes, stream);
}

size_t kda_lina_chunk_fwd_varlen_workspace_size(const kda_shape* shape, int n_seqs) {
  int es = 0;
  return n_seqs >= 0 && check_lina_shape(shape, 1, false, n_seqs, &es) == KDA_OK ? fwd_layout(*shape, n_seqs).bytes : 0;
}

int kda_lina_chunk_fwd_varlen(const kda_shape* shape, int qk_heads, const int* cu_seqlens, int n_seqs, const void* q,
                              const void* k, const void* v, const float* log_decay, int decay_per_head,
                              const float* initial_state, void* o, float* final_state, void* workspace,
                              size_t workspace_bytes, void* stream) {
  if (!shape) return KDA_ERR_NULL;
  if (n_seqs < 0) return KDA_ERR_SHAPE;
  return fwd_impl(shape, qk_heads, cu_seqlens, n_seqs, q, k, v, log_decay, decay_per_head, initial_state, o,
                  final_state, workspace, workspace_bytes, stream);
}

size_t kda_lina_chunk_bwd_workspace_size(const kda_shape* shape, int qk_heads) {
  int es = 0;
  return check_lina_shape(shape, qk_heads, false, -1, &es) == KDA_OK ? bwd_layout(*shape, qk_heads, -1).bytes : 0;
}

int kda_lina_chunk_bwd(const kda_shape* shape, int qk_heads, const void* q, const void* k, const void* v,
                       const float* log_decay, int decay_per_head, const float* initial_state, const void* d_o,
                       const float* d_final_state, void* dq, void* dk, void* dv, float* d_log_decay,
                       float* d_initial_state, void* workspace, size_t workspace_bytes, void* stream) {
  const BwdPtrs p{q,  k,  v,  log_decay,   decay_per_head,  initial_state, d_o, d_final_state,
                  dq, dk, dv, d_log_decay, d_initial_state, workspace,     workspace_bytes};
  return bwd_impl(shape, qk_heads, nullptr, -1, p, stream);
}

size_t kda_lina_chunk_bwd_varlen_workspace_size(const kda_shape* shape, int qk_heads, int n_seqs) {
  int es = 0;
  return n_seqs >= 0 && check_lina_shape(shape, qk_heads, false, n_seqs, &es) == KDA_OK
             ? bwd_layout(*shape, qk_heads, n_seqs).bytes
             : 0;
}

int kda_lina_chunk_bwd_varlen(const kda_shape* shape, int qk_heads, const int* cu_seqlens, int n_seqs, const void* q,
                              const void* k, const void* v, const float* log_decay, int decay_per_head,
                              const float* initial_state, const void* d_o, const float* d_final_state, void* dq,
                              void* dk, void* dv, float* d_log_decay, float* d_initial_state, void* workspace,
                              size_t workspace_bytes, void* stream) {
  if (!shape) return KDA_ERR_NULL;
  if (n_seqs < 0) return KDA_ERR_SHAPE;
  const BwdPtrs p{q,  k,  v,  log_decay,   decay_per_head,  initial_state, d_o, d_final_state,
                  dq, dk, dv, d_log_decay, d_initial_state, workspace,     workspace_bytes};
  return bwd_impl(shape, qk_heads, cu_seqlens, n_seqs, p, stream);
}

int kda_lina_decode_step(const kda_shape* shape, int qk_heads, const void* q, const void* k, const void* v,
                         const float* log_decay, int decay_per_head, float* state, void* o, void* stream) {
  return decode_impl(shape, qk_heads, 1, q, k, v, log_decay, decay_per_head, state, o, stream);
}

int kda_lina_decode_tokens(const kda_shape* shape, int qk_heads, const void* q, const void* k, const void* v,
                           const float* log_decay, int decay_per_head, float* state, void* o, void* stream) {
  if (!shape) return KDA_ERR_NULL;
  return decode_impl(shape, qk_heads, shape->T, q, k, v, log_decay, decay_per_head, state, o, stream);
}

}  // extern "C"
