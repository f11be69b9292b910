// kda_gdr.hip -- the gated delta rule with one decay per head, chunk by chunk.
//
//   S_t = e^{g_t} (I - b_t k_t k_t^T) S_{t-1} + b_t k_t v_t^T,   o_t = S_t^T q_t.
//
// With r_t = v_t - e^{g_t} S_{t-1}^T k_t it is linear attention over the values u_t = b_t r_t.  In a chunk
// of 64 tokens with start state S, G the inclusive sum of g, A_ij = e^{G_i - G_j} k_i . k_j (j < i):
//   r = N (V - e^G o K S),          N = (I + A diag(b))^-1,
//   o = e^G o (Q S) + P (b o r),    P_ij = e^{G_i - G_j} q_i . k_j (j <= i),
//   S <- e^{G_C} S + K^T (e^{G_C - G} o b o r).
// The backward's reverse walk is the same form.  With R the gradient of the state behind a chunk, tokens
// in reverse order and the decay of a step that of the token after it,
//   z = N' (e^G' o K R + P' do),    P'_ij = e^{G'_i - G'_j} k_i . q_j,   y = b o z = dv,
//   R <- e^{G'_C} R + Q^T (e^{G'_C - G'} o do) - K^T (e^{G'_C - G'} o y),
// where N' is made from the reversed chunk as N is from the chunk.
//
// N and P do not depend on the state: gdr_prep_kernel makes them for all chunks at once, one wave each;
// gdr_walk_kernel then walks each chain (sequence or segment, head, 64 value columns).  A chain in
// several segments needs the state each starts from: the walk without outputs gives a segment's end
// state B from a zero start and, over the columns of the identity, its transfer M (S -> M S + B);
// gdr_link_kernel goes through the segments with those.
#include <algorithm>
#include <type_traits>

#include "kda_gdr_tile.h"

namespace kda {

namespace {

// Modes of the walk: the forward, the backward's forward, its reverse, and the first pass over segments
// of either direction.
enum GdrMode : int { kFwd, kTrain, kRev, kSegFwd, kSegRev };
__host__ __device__ constexpr bool is_rev(int mode) { return mode == kRev || mode == kSegRev; }
__host__ __device__ constexpr bool is_seg(int mode) { return mode == kSegFwd || mode == kSegRev; }

struct GdrParams {
  GdrWalk a;
  WalkParams p;  // p.w = a.walk
  int64_t chunks;
};

// ---------------------------------------------------------------------------------------
// N and P of every chunk
// ---------------------------------------------------------------------------------------

// rows 16 I + n of a chunk straight from memory: channels 32 s + 8 g ..
template <typename T>
__device__ __forceinline__ void mem_frag(Frag<T>& f, const Rows& b, uint32_t off) {
  const u32x4_t x = b.load16(off);
  if constexpr (sizeof(T) == 2) {
#pragma unroll
    for (int i = 0; i < 4; ++i) f.w[i] = x[i];
  } else {
    const u32x4_t y = b.load16(off + 16);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f.w[i] = __uint_as_float(x[i]);
      f.w[4 + i] = __uint_as_float(y[i]);
    }
  }
}

__device__ __forceinline__ void wave_fence() {  // LDS of one wave: its operations stay in order
#ifndef KDA_HOST_PASS
  asm volatile("" ::: "memory");
#endif
}

struct PrepLds {
  Decays dec;
  float beta[C];
  float blk[4][SUB][SUB + 4];  // one 16 x 16 block of each row group
};

// X = (I - M)^-1 of four strictly lower 16 x 16 blocks at once, M's rows in `blk`: row group r of the wave
// takes block r, lane n its column n, by forward substitution (bounded by X's own size, which the powers
// of M are not: for equal keys they grow like binomials).  X's rows replace M's.
__device__ __forceinline__ void invert_blocks(float (&blk)[4][SUB][SUB + 4], int lane) {
  const int g = lane >> 4, n = lane & 15;
  float t[SUB], x[SUB];
#pragma unroll
  for (int c = 0; c < SUB; c += 4) {
    const float4 w = *(const float4*)&blk[g][n][c];
    t[c] = w.x; t[c + 1] = w.y; t[c + 2] = w.z; t[c + 3] = w.w;
  }
  dpp_sources_ready(t);
#define KDA_SUBST(i)                                                                    \
  {                                                                                     \
    float acc = n == i ? 1.f : 0.f;                                                     \
    _Pragma("unroll") for (int c = 0; c < i; ++c) acc = fmac_bcast<i>(acc, t[c], x[c]); \
    x[i] = acc;                                                                         \
  }
  KDA_SUBST(0) KDA_SUBST(1) KDA_SUBST(2) KDA_SUBST(3) KDA_SUBST(4) KDA_SUBST(5) KDA_SUBST(6) KDA_SUBST(7)
  KDA_SUBST(8) KDA_SUBST(9) KDA_SUBST(10) KDA_SUBST(11) KDA_SUBST(12) KDA_SUBST(13) KDA_SUBST(14) KDA_SUBST(15)
#undef KDA_SUBST
  wave_fence();
#pragma unroll
  for (int i = 0; i < SUB; ++i) blk[g][i][n] = x[i];
  wave_fence();
}

// acc += X Y, X's rows and Y's columns of a lane (rows n and columns n, quads 4 g ..): the accumulator holds
// the product's rows 4 g + i of column n (a "column" block).  With the arguments exchanged it is a "row" block,
// columns 4 g + i of row n.
__device__ __forceinline__ void mm16(f32x4_t& acc, const f32x4_t& x, const f32x4_t& y) {
#ifndef KDA_HOST_PASS
#pragma unroll
  for (int s = 0; s < 4; ++s) acc = __builtin_amdgcn_mfma_f32_16x16x4f32(x[s], y[s], acc, 0, 0, 0);
#endif
}

// One wave: N and P of one chunk and head, fp32.  A wave each, without barriers, three workgroups to a compute unit (bf16).
// What bounds it: bytes.  N and P are 20 KB of fp32 written for 32 KB of bf16 q and k read (d = 128): B4 H32 T8K 0.94 GB
// in 170 us, 5.5 TB/s (matrix cores 15% busy), H16 T128K 331.  Scores of shared heads are made for every value head.
template <typename T, int DK, bool REV>
__global__ __launch_bounds__(256, sizeof(T) == 2 ? 3 : 2) void gdr_prep_kernel(const GdrParams gp) {
  constexpr int KS = DK / 32;
  __shared__ PrepLds lds[4];
  const LinaWalk& w = gp.p.w;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, g = lane >> 4, n = lane & 15;
  PrepLds& L = lds[wave];
  const int quads = (w.H + 3) / 4;
  const int64_t chunk = blockIdx.x / quads;
  const int h = (int)uniform64((int64_t)(blockIdx.x % quads) * 4 + wave);
  if (h >= w.H) return;
  Chain ch;  // of the place only what the rows need
  ch.h = h;
  int c;
  if (w.cs) {
    int x = 0, y = w.n;
    while (y - x > 1) {
      const int m = (x + y) >> 1;
      if (w.cs[m] / C + m <= chunk) x = m;
      else y = m;
    }
    ch.lo = uniform64(w.cs[x]);
    ch.hi = uniform64(w.cs[x + 1]);
    c = (int)uniform64(chunk - (ch.lo / C + x));
  } else {
    const int64_t per = gp.chunks / w.n;
    ch.lo = uniform64(chunk / per * w.T);
    ch.hi = ch.lo + w.T;
    c = (int)uniform64(chunk % per);
  }
  const int64_t t0 = ch.lo + (int64_t)c * C;
  if (t0 >= ch.hi) return;
  ch.first = 0;
  ch.last = c + 1;
  const uint32_t have = ch.rows(c);
  const Operand<T> q(w.q, w, h, DK, 0), k(w.k, w, h, DK, 0);
  const Rows kr = k.rows(t0, have), qr = q.rows(t0, have);
  auto row_of = [&](int I, uint32_t step) { return row_off(REV, 16 * I + n, step) + 8 * g * (uint32_t)sizeof(T); };
  Frag<T> fk[4][KS];
#pragma unroll
  for (int I = 0; I < 4; ++I)
#pragma unroll
    for (int s = 0; s < KS; ++s) mem_frag<T>(fk[I][s], kr, row_of(I, k.step) + s * 32 * sizeof(T));
  {
    const int64_t t = t0 + (REV ? C - 1 - lane : lane);
    L.beta[lane] = t < ch.hi ? Elem<T>::load(gp.a.beta, (size_t)t * w.H + h) : 0.f;
    chunk_decays(L.dec, row_decay<REV>(w, ch, c, lane), lane);
  }
  wave_fence();
  const size_t slot = (size_t)chunk * w.H + h;
  float4* inv = (float4*)gp.a.inv + slot * kTriUnits + lane;
  float4* score = (float4*)gp.a.score + slot * kTriUnits + lane;
  auto decay = [&](int I, int J, float (&r)[4]) {
    const float ih = L.dec.hi[16 * I + n], il = L.dec.lo[16 * I + n];
    const float4 jh = *(const float4*)&L.dec.hi[16 * J + 4 * g], jl = *(const float4*)&L.dec.lo[16 * J + 4 * g];
    r[0] = fast_exp2((ih - jh.x) + (il - jl.x));
    r[1] = fast_exp2((ih - jh.y) + (il - jl.y));
    r[2] = fast_exp2((ih - jh.z) + (il - jl.z));
    r[3] = fast_exp2((ih - jh.w) + (il - jl.w));
  };

  {  // what the walk needs of the tokens
    float* tok = gp.a.token + slot * kTokenFloats;
    tok[lane] = L.dec.row[lane];
    tok[C + lane] = L.dec.col[lane];
    tok[2 * C + lane] = L.beta[lane];
    if (lane == 0) tok[3 * C] = L.dec.tot;
  }

  // P: rows of block row I are q's (in reverse k's) against k's (q's)
  f32x4_t M[10];
#pragma unroll
  for (int I = 0; I < 4; ++I) {
    Frag<T> fq[KS];
#pragma unroll
    for (int s = 0; s < KS; ++s) mem_frag<T>(fq[s], qr, row_of(I, q.step) + s * 32 * sizeof(T));
#pragma unroll
    for (int J = 0; J < 4; ++J) {
      if (REV ? J < I : J > I) continue;  // in reverse fq are the columns: block (J, I)
      f32x4_t a = zero4();
#pragma unroll
      for (int s = 0; s < KS; ++s) {
        if constexpr (REV) mma(a, fq[s], fk[J][s]);
        else mma(a, fk[J][s], fq[s]);
      }
      const int bi = REV ? J : I, bj = REV ? I : J;
      float r[4];
      decay(bi, bj, r);
#pragma unroll
      for (int i = 0; i < 4; ++i) a[i] = bi != bj || 4 * g + i <= n ? a[i] * r[i] : 0.f;
      *(f32x4_t*)&score[tri(bi, bj) * 64] = a;
    }
  }
  // -A o beta, as row blocks
#pragma unroll
  for (int I = 0; I < 4; ++I)
#pragma unroll
    for (int J = 0; J <= I; ++J) {
      f32x4_t a = zero4();
#pragma unroll
      for (int s = 0; s < KS; ++s) mma(a, fk[J][s], fk[I][s]);
      float r[4];
      decay(I, J, r);
      const float4 b = *(const float4*)&L.beta[16 * J + 4 * g];
      const float bs[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) M[tri(I, J)][i] = I != J || 4 * g + i < n ? -(a[i] * r[i]) * bs[i] : 0.f;
    }
#pragma unroll
  for (int I = 0; I < 4; ++I) *(f32x4_t*)&L.blk[I][n][4 * g] = M[tri(I, I)];
  wave_fence();
  invert_blocks(L.blk, lane);
  f32x4_t Dr[4], Dc[4];  // the diagonal blocks' inverses as row and as column blocks
#pragma unroll
  for (int I = 0; I < 4; ++I) {
    Dr[I] = *(const f32x4_t*)&L.blk[I][n][4 * g];
#pragma unroll
    for (int i = 0; i < 4; ++i) Dc[I][i] = L.blk[I][4 * g + i][n];
    *(f32x4_t*)&inv[tri(I, I) * 64] = Dr[I];
  }
  // below the diagonal, column by column: X_IJ = D_I sum_m -M_Im X_mJ
#pragma unroll
  for (int J = 0; J < 3; ++J) {
    f32x4_t Xc[4];
    Xc[J] = Dc[J];
#pragma unroll
    for (int I = J + 1; I < 4; ++I) {
      f32x4_t W = zero4(), X = zero4();
#pragma unroll
      for (int m = J; m < I; ++m) mm16(W, M[tri(I, m)], Xc[m]);
      mm16(X, W, Dr[I]);
      *(f32x4_t*)&inv[tri(I, J) * 64] = X;
      if (I < 3) {
        Xc[I] = zero4();
        mm16(Xc[I], Dr[I], W);
      }
    }
  }
}

// ---------------------------------------------------------------------------------------
// the walk
// ---------------------------------------------------------------------------------------

template <typename T, int DK, int MODE>
struct WalkLds {
  static constexpr int NP = MODE == kFwd ? kMost<T> : kAll<T>;  // terms of P
  static constexpr int K = 0, V = K + RowTile<T, DK>::BYTES, N = V + RowTile<T, VT>::BYTES, Q = N + kTriBytes<T, kAll<T>>;
  static constexpr int P = Q + (MODE == kSegFwd ? 0 : RowTile<T, DK>::BYTES);
  static constexpr int SIZE = P + (MODE == kSegFwd ? 0 : kTriBytes<T, NP>);
  static constexpr int NBUF = 2 * SIZE <= 152 * 1024 ? 2 : 1;
  static constexpr int BYTES = NBUF * SIZE;
};

// fn(ct, i, element) over a thread's entries of a [dk, dv] state: row channel(ct, 4 g + i), column 16 wave + n
template <int DK, typename F>
__device__ __forceinline__ void each_entry(const LinaWalk& w, const Chain& ch, int wave, int lane, F fn) {
  const int g = lane >> 4, vc = ch.vt * VT + 16 * wave + (lane & 15);
  const size_t b0 = ((size_t)ch.sq * w.H + ch.h) * (size_t)DK * w.dv + vc;
#pragma unroll
  for (int ct = 0; ct < DK / 16; ++ct)
#pragma unroll
    for (int i = 0; i < 4; ++i) fn(ct, i, b0 + (size_t)(channel(ct, 4 * g) + i) * w.dv);
}

// Where a walk's segment slots lie: [piece][H][value tiles].
__device__ __forceinline__ size_t seg_at(const LinaWalk& w, const Chain& ch, int64_t piece, int vt) {
  return ((size_t)piece * w.H + ch.h) * (w.dv / VT) + vt;
}

// The state a chain starts from: the caller's, or what gdr_link_kernel left for its segment.
template <int DK>
__device__ __forceinline__ void first_state(const GdrParams& gp, const Chain& ch, bool rev, int tid,
                                            f32x4_t (&S)[DK / 16]) {
  const LinaWalk& w = gp.p.w;
#pragma unroll
  for (int ct = 0; ct < DK / 16; ++ct) S[ct] = zero4();
  if (w.split && ch.nsg > 1) {
    const int64_t piece = ch.head ? ch.start(gp.p) : ch.end(rev, rev ? ch.sg + 1 : ch.sg - 1);
    const f32x4_t* from = (const f32x4_t*)(w.seg_state + seg_at(w, ch, piece, ch.vt) * (DK * VT));
#pragma unroll
    for (int ct = 0; ct < DK / 16; ++ct) S[ct] = from[ct * NT + tid];
  } else if (w.s0) {
    each_entry<DK>(w, ch, tid >> 6, tid & 63, [&](int ct, int i, size_t at) { S[ct][i] = w.s0[at]; });
  }
}

// <kept state, S> of a wave at the first token of chunk c, with that token's decay: its gradient
template <int DK>
__device__ __forceinline__ void gdr_anchor(const WalkParams& p, const Chain& ch, int c, int tid,
                                           const f32x4_t (&S)[DK / 16]) {
  const LinaWalk& w = p.w;
  float d = 0.f;
  if (c > 0) {
    const f32x4_t* from = (const f32x4_t*)(w.snap + ch.at(p, ch.kept(p, c)) * (DK * VT)) + tid;
#pragma unroll
    for (int ct = 0; ct < DK / 16; ++ct) {
      const f32x4_t x = from[ct * NT];
#pragma unroll
      for (int i = 0; i < 4; ++i) d = fmaf(x[i], S[ct][i], d);
    }
  } else if (w.snap0) {
    each_entry<DK>(w, ch, tid >> 6, tid & 63, [&](int ct, int i, size_t at) { d = fmaf(w.snap0[at], S[ct][i], d); });
  }
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) d += __shfl_xor(d, off);
  if ((tid & 63) == 0) w.anchor[ch.at(p, ch.anchor(p, c)) * 4 + (tid >> 6)] = expf(ch.decay_log(w, ch.lo + (int64_t)c * C)) * d;
}

// What a chunk's tokens need besides the tiles, as gdr_prep_kernel leaves it.
struct TokenLds {
  float row[C];   // decay from the chunk's start to the token
  float col[C];   // from the token to the chunk's end
  float beta[C];
  float tot;      // the whole chunk
  float pad[3];
};
static_assert(sizeof(TokenLds) == kTokenFloats * 4, "as in memory");

// One chain: four waves keep the state (16 value columns each, fp32 accumulators that serve as operands), four
// fetch the next chunk's tiles.  Products run as [token][value] where the next product takes them along the
// tokens (K S, N ., P .), so that no value leaves its lane between them, and transposed where they are
// stored (four neighbouring columns of one token to a lane).  A state wave has its matrix unit to itself, and its products
// wait for each other: operands are read a group of products ahead, and what the state does not wait for (P u, the
// outputs) stands between what it does.
//
// Precision (bf16 inputs): what ends in the state or in an fp32 output goes through the matrix cores in
// three bf16 terms (all 24 bits): S against k, N and what it multiplies, b o r against k.  The forward's
// outputs, which are rounded to bf16 themselves, take S, P and b o r in two (16 bits).
//
// What bounds it: the chain from S through K S, r and b o r back to S.  A step of the forward (d = 128, bf16) has 182 products
// a wave and takes about 6,900 cycles, matrix cores 42% busy; tiles of fewer LDS conflicts, another order and other ways to
// split changed it by a few percent.  B4 H32 T8K: 409 to 419 us for 128 steps in a row; in training 634 forward (36% busy), 811
// in reverse (26%), where states and r are written too and the products of Q and d_o come on top.  Of 131,072 tokens, 16 heads
// (32 chains): end states and transfers of segments 1,075 us, links 63, outputs 780.  Two workgroups to a compute unit in the first
// pass (128 registers) spill: 4,260 us for the whole call instead of 2,227.
// Registers: all 256 are in use in training, and some do not fit: bf16, d = 128 in reverse 51 (208 bytes of scratch a
// lane); fp32, d = 128 5 in the forward, 31 in training, 192 in reverse (772 bytes) and 60 in its first pass; d = 64 11 in reverse.
template <typename T, int DK, int MODE>
__global__ __launch_bounds__(2 * NT, 2) void gdr_walk_kernel(const GdrParams gp) {
  typedef WalkLds<T, DK, MODE> Lds;
  constexpr bool REV = is_rev(MODE), SEG = is_seg(MODE);
  constexpr bool HAS_Q = MODE != kSegFwd, HAS_P = HAS_Q, OUT = MODE == kFwd || MODE == kTrain, DOTS = MODE == kTrain || MODE == kRev;
  constexpr int A3 = kAll<T>, CT = DK / 16, KS = DK / 32, NBUF = Lds::NBUF;
  extern __shared__ __align__(16) char smem[];
  __shared__ __align__(16) TokenLds tok[2];
  __shared__ float sdot[DOTS ? 2 : 1][4][C], sdot2[MODE == kRev ? 2 : 1][4][C];
  const WalkParams& p = gp.p;
  const LinaWalk& w = p.w;
  const int tid = threadIdx.x & (NT - 1), lane = tid & 63, wave = tid >> 6, g = lane >> 4, n = lane & 15;
  Chain ch;
  if (!ch.place(p, REV, blockIdx.x)) return;
  if (SEG && ch.tail) return;  // nobody starts from a tail's end
  const int nv = w.dv / VT;
  const bool ident = SEG && ch.vt >= nv;  // columns of the identity, no values
  const int steps = ch.last - ch.first;
  auto chunk = [&](int it) { return REV ? ch.last - 1 - it : ch.first + it; };
  auto buf = [&](int it) { return smem + (NBUF == 2 ? (it & 1) * Lds::SIZE : 0); };
  // the first of this sequence's chunks in the tables of N and P
  const int64_t base = w.cs ? ch.lo / C + ch.sq : (int64_t)ch.sq * ch.nch;
  auto slot = [&](int it) { return (size_t)(base + chunk(it)) * w.H + ch.h; };
  const Residual res;

  if (threadIdx.x >= NT) {
    if (steps == 0) return;
    const Operand<T> q(w.q, w, ch.h, DK, 0), k(w.k, w, ch.h, DK, 0), v(w.v, w, ch.h, w.dv, (ident ? 0 : ch.vt) * VT);
    struct Tiles {
      StageRows<T, DK> k, q;
      StageRows<T, VT> v;
      StageTri<T, A3> n;
      StageTri<T, Lds::NP> p;
      u32x4_t t;  // the last wave's
    };
    // bf16: two chunks are on their way, because from memory under load a tile takes longer than a step; fp32's tiles are
    // twice as large and their steps longer.
    constexpr int SETS = sizeof(T) == 2 ? 2 : 1;
    Tiles ra, rb;
    auto fetch = [&](Tiles& r, int it) {
      const int c = chunk(it);
      const int64_t t = ch.lo + (int64_t)c * C;
      const uint32_t have = ch.rows(c);
      if (wave == 3) r.t = Rows(gp.a.token + slot(it) * kTokenFloats, kTokenFloats * 4).load16(lane * 16);
      r.k.load(k.rows(t, have), k.step, REV, tid);
      r.v.load(v.rows(t, ident ? 0 : have), v.step, REV, tid);
      r.n.load(gp.a.inv, slot(it), tid);
      if constexpr (HAS_Q) r.q.load(q.rows(t, have), q.step, REV, tid);
      if constexpr (HAS_P) r.p.load(gp.a.score, slot(it), tid);
    };
    auto put = [&](const Tiles& r, int it) {
      char* b = buf(it);
      if (wave == 3 && lane < kTokenFloats / 4) *(u32x4_t*)((char*)&tok[it & 1] + lane * 16) = r.t;
      r.k.store(b + Lds::K, tid);
      r.v.store(b + Lds::V, tid);
      r.n.store(res, b + Lds::N, tid);
      if constexpr (HAS_Q) r.q.store(b + Lds::Q, tid);
      if constexpr (HAS_P) r.p.store(res, b + Lds::P, tid);
    };
    auto dots = [&](int it) {  // a step's, once its waves are done
      if constexpr (DOTS) {
        if (wave == 1) store_dots<kDotRow, REV>(p, ch, chunk(it), sdot[it & 1], sdot[0][0], lane);
        if constexpr (MODE == kRev) {
          if (wave == 2) {
            const float(&s)[4][C] = sdot2[it & 1];
            const float d = (s[0][lane] + s[1][lane]) + (s[2][lane] + s[3][lane]);
            const int64_t t = ch.lo + (int64_t)chunk(it) * C + C - 1 - lane;
            if (t < ch.hi) gp.a.dots2[((size_t)ch.vt * w.H + ch.h) * p.rows + t] = d;
          }
        }
      }
    };
    fetch(ra, 0);
    if (SETS == 2 && steps > 1) fetch(rb, 1);
#pragma unroll
    for (int x = 0; x < NBUF; ++x) {
      tri_clear<T, A3>(smem + x * Lds::SIZE + Lds::N, tid);
      if constexpr (HAS_P) tri_clear<T, Lds::NP>(smem + x * Lds::SIZE + Lds::P, tid);
    }
    put(ra, 0);
    if (steps > SETS) fetch(ra, SETS);
    lds_barrier();
    auto step = [&](Tiles& r, int it) {  // r: chunk it + 1
      if constexpr (NBUF == 1) {
        lds_barrier();
        dots(it);
      }
      if (it + 1 < steps) put(r, it + 1);
      if (it + 1 + SETS < steps) fetch(r, it + 1 + SETS);
      if (NBUF == 2 && it > 0) dots(it - 1);
      lds_barrier();
    };
    for (int it = 0; it < steps; it += 2) {
      if constexpr (SETS == 2) step(rb, it);
      else step(ra, it);
      if (it + 1 < steps) step(ra, it + 1);
    }
    if constexpr (NBUF == 2) dots(steps - 1);
    return;
  }

  f32x4_t S[CT];
  if constexpr (SEG) {
#pragma unroll
    for (int ct = 0; ct < CT; ++ct)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        S[ct][i] = ident && channel(ct, 4 * g) + i == (ch.vt - nv) * VT + 16 * wave + n ? 1.f : 0.f;
  } else {
    first_state<DK>(gp, ch, REV, tid, S);
  }
  DotRows<T> xd, rd;  // rows of d_o (forward), of v and of r (reverse), a chunk ahead
  const Operand<T> x(w.x, w, ch.h, w.dv, (ident ? 0 : ch.vt) * VT), xr(gp.a.r, w, ch.h, w.dv, (ident ? 0 : ch.vt) * VT);
  auto fetch_dots = [&](int it) {
    const int c = chunk(it);
    const int64_t t = ch.lo + (int64_t)c * C;
    if constexpr (DOTS) xd.load(x.rows(t, ch.rows(c)), x.step, REV, wave, lane);
    if constexpr (MODE == kRev) rd.load(xr.rows(t, ch.rows(c)), xr.step, REV, wave, lane);
  };
  const RowAt<T, DK> rows(lane);
  const ColAt<T, DK, true> cols(lane);
  const ColAt<T, VT, false> vals(lane);
  // The state's operands, 32 channels each, made as soon as the update before is through with them.
  Terms<T, A3> fs[KS];
#pragma unroll
  for (int s = 0; s < KS; ++s) split(res, S[2 * s], S[2 * s + 1], fs[s]);
  if (steps > 0) {
    fetch_dots(0);
    lds_barrier();
  }
  for (int it = 0; it < steps; ++it) {
    const int c = chunk(it);
    const char* b = buf(it);
    const TokenLds& tl = tok[it & 1];
    const char *sK = b + Lds::K, *sQ = b + Lds::Q, *sV = b + Lds::V, *sN = b + Lds::N, *sP = b + Lds::P;
    // operands a group of products ahead
    Frag<T> fk[2][KS], fq[2][KS], fv[2];
    auto load_rows = [&](int t) {
#pragma unroll
      for (int s = 0; s < KS; ++s) rows.load(fk[t & 1][s], sK, 16 * t, s);
      if constexpr (OUT)
#pragma unroll
        for (int s = 0; s < KS; ++s) rows.load(fq[t & 1][s], sQ, 16 * t, s);
    };
    load_rows(0);
    f32x4_t rw[4], bt[4], cw[4];
    float rn[4];
#pragma unroll
    for (int y = 0; y < 2; ++y) vals.load(fv[y], sV, wave, y, lane);
#pragma unroll
    for (int t = 0; t < 4; ++t) rw[t] = *(const f32x4_t*)&tl.row[16 * t + 4 * g];
    if constexpr (DOTS) {
      // the state this chunk meets, as rows of value columns
      T* to = (T*)gp.a.kept + (((size_t)(base + c) * w.H + ch.h) * nv + ch.vt) * (size_t)(VT * DK) + (16 * wave + n) * DK + 8 * g;
#pragma unroll
      for (int c2 = 0; c2 < KS; ++c2) {
        const float s8[8] = {S[2 * c2][0],     S[2 * c2][1],     S[2 * c2][2],     S[2 * c2][3],
                             S[2 * c2 + 1][0], S[2 * c2 + 1][1], S[2 * c2 + 1][2], S[2 * c2 + 1][3]};
        st_row8<T>((char*)(to + 32 * c2), s8);
      }
      if (MODE == kTrain && c > 0 && c % lina_keep(w.bf16) == 0) store_snap<DK>(p, ch, c, tid, S);
    }
    // x0 = V - e^G o K S as [token][value] (in reverse e^G' o K R + P' d_o); Q S as [value][token]
    f32x4_t kS[4], o[4], x0[4];
    Terms<T, A3> fx[2], fn[4];
    Terms<T, Lds::NP> fp[4];
    auto from_values = [&](int t) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float y = rw[t][i] * kS[t][i];
        x0[t][i] = REV ? y : fv[t >> 1].get((t & 1) * 4 + i) - y;
      }
      if constexpr (REV)
#pragma unroll
        for (int s = 0; s <= t / 2; ++s) {
          tri_frag(fp[0], sP, t, s, lane);
#pragma unroll
          for (int m = Lds::NP - 1; m >= 0; --m) mma(x0[t], fp[0].f[m], fv[s]);
        }
    };
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      if (t < 3) {
        load_rows(t + 1);
      } else {
#pragma unroll
        for (int y = 0; y < 4; ++y) tri_frag(fn[y], sN, y, 0, lane);
      }
      if (t == 2) from_values(0);
      if (t == 3) {
        from_values(1);
        split(res, x0[0], x0[1], fx[0]);
      }
      kS[t] = o[t] = zero4();
#pragma unroll
      for (int s = 0; s < KS; ++s)
#pragma unroll
        for (int m = 0; m < A3; ++m) mma(kS[t], fk[t & 1][s], fs[s].f[m]);
      if constexpr (OUT)
#pragma unroll
        for (int s = 0; s < KS; ++s)
#pragma unroll
          for (int m = 0; m < (MODE == kTrain ? A3 : kMost<T>); ++m) mma(o[t], fs[s].f[m], fq[t & 1][s]);
      if (t == 3) made(fx[0]);
      in_turn();
    }
    // r = N x0 (z in reverse): the first 32 columns of N, then the last; rt: [value][token], to store it
    f32x4_t r[4], rt[4];
    Terms<T, A3> fn2[2];
#pragma unroll
    for (int t = 0; t < 2; ++t) tri_frag(fn2[t], sN, 2 + t, 1, lane);
#pragma unroll
    for (int t = 0; t < 4; ++t) bt[t] = *(const f32x4_t*)&tl.beta[16 * t + 4 * g];
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      r[t] = rt[t] = zero4();
      mma_terms(r[t], fn[t], fx[0]);
      if constexpr (DOTS) mma_terms(rt[t], fx[0], fn[t]);
    }
    from_values(2);
    from_values(3);
    split(res, x0[2], x0[3], fx[1]);
    made(fx[1]);
    in_turn();
    // u = b o r (y in reverse), and what enters the state
    constexpr int NU = MODE == kTrain ? A3 : kMost<T>;
    f32x4_t u[4];
    Terms<T, A3> fy[2], fz[2];
    Terms<T, NU> fu[2];
    const float tot = tl.tot;
    auto weigh = [&](int s) {
      f32x4_t y[2], z[2];
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          u[2 * s + j][i] = bt[2 * s + j][i] * r[2 * s + j][i];
          y[j][i] = (REV ? -cw[2 * s + j][i] : cw[2 * s + j][i]) * u[2 * s + j][i];
          if constexpr (REV) z[j][i] = cw[2 * s + j][i] * fv[s].get(4 * j + i);
        }
      split(res, y[0], y[1], fy[s]);
      made(fy[s]);
      if constexpr (OUT) {
        split(res, u[2 * s], u[2 * s + 1], fu[s]);
        made(fu[s]);
      }
      if constexpr (REV) {
        split(res, z[0], z[1], fz[s]);
        made(fz[s]);
      }
    };
#pragma unroll
    for (int t = 0; t < 4; ++t) cw[t] = *(const f32x4_t*)&tl.col[16 * t + 4 * g];
    if constexpr (OUT) {
#pragma unroll
      for (int t = 0; t < 4; ++t) tri_frag(fp[t], sP, t, 0, lane);
#pragma unroll
      for (int t = 0; t < 4; ++t) rn[t] = tl.row[16 * t + n];
    }
#pragma unroll
    for (int t = 2; t < 4; ++t) {
      mma_terms(r[t], fn2[t - 2], fx[1]);
      if constexpr (DOTS) mma_terms(rt[t], fx[1], fn2[t - 2]);
    }
    weigh(0);
    if constexpr (OUT)
#pragma unroll
      for (int t = 0; t < 4; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) o[t][i] *= rn[t];
    in_turn();
    // o += P u, the first 32 columns of P, while the second half of what enters the state is made
    Frag<T> fc[2][2], fd[2][2];
    auto load_cols = [&](int ct) {
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        cols.load(fc[ct & 1][s], sK, ct, s, lane);
        if constexpr (REV) cols.load(fd[ct & 1][s], sQ, ct, s, lane);
      }
    };
    load_cols(0);
    if constexpr (OUT)
#pragma unroll
      for (int t = 0; t < 4; ++t) mma_terms(o[t], fu[0], fp[t]);
    weigh(1);
    in_turn();
    // S <- e^{G_C} S + K^T y (in reverse + Q^T z)
#pragma unroll
    for (int ct = 0; ct < CT; ++ct) {
      if (ct + 1 < CT) {
        load_cols(ct + 1);
      } else {
        if constexpr (OUT)
#pragma unroll
          for (int t = 2; t < 4; ++t) tri_frag(fp[t], sP, t, 1, lane);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) S[ct][i] *= tot;
#pragma unroll
      for (int s = 0; s < 2; ++s)
#pragma unroll
        for (int m = 0; m < A3; ++m) mma(S[ct], fc[ct & 1][s], fy[s].f[m]);
      if constexpr (REV)
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
          for (int m = 0; m < A3; ++m) mma(S[ct], fd[ct & 1][s], fz[s].f[m]);
      if (ct >= 2 && ct % 2 == 0) {
        split(res, S[ct - 2], S[ct - 1], fs[ct / 2 - 1]);
        made(fs[ct / 2 - 1]);
      }
      in_turn();
    }
    if constexpr (OUT)
#pragma unroll
      for (int t = 2; t < 4; ++t) mma_terms(o[t], fu[1], fp[t]);
    split(res, S[CT - 2], S[CT - 1], fs[KS - 1]);
    made(fs[KS - 1]);
    if constexpr (MODE == kFwd) store_out<T, false>(o, w, ch, c, wave, lane);
    if constexpr (MODE == kTrain) {
      xd.dot(o, sdot[it & 1][wave], lane);
      store_out<T, false>(rt, w, ch, c, wave, lane);
    }
    if constexpr (MODE == kRev) {
      rd.dot(rt, sdot2[it & 1][wave], lane);
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        const float bn = tl.beta[16 * t + n];
#pragma unroll
        for (int i = 0; i < 4; ++i) rt[t][i] *= bn;
      }
      xd.dot(rt, sdot[it & 1][wave], lane);
      store_out<T, true>(rt, w, ch, c, wave, lane);
    }
    if constexpr (DOTS)
      if (it + 1 < steps) fetch_dots(it + 1);
    if constexpr (MODE == kRev)
      if (w.anchor && c % lina_keep(w.bf16) == 0) gdr_anchor<DK>(p, ch, c, tid, S);
    lds_barrier();
    if constexpr (NBUF == 1) lds_barrier();
  }
  if constexpr (SEG) {
    const int64_t piece = ch.end(REV, ch.sg);
    float* at = ident ? gp.a.transfer + (((size_t)piece * w.H + ch.h) * (DK / VT) + ch.vt - nv) * (DK * VT)
                      : w.seg_state + seg_at(w, ch, piece, ch.vt) * (DK * VT);
#pragma unroll
    for (int ct = 0; ct < CT; ++ct) ((f32x4_t*)at)[ct * NT + tid] = S[ct];
  } else if (w.sT && ch.tail) {  // a reverse walk's state is the gradient after the first token's decay
    const float d = REV && ch.nch > 0 ? expf(ch.decay_log(w, ch.lo)) : 1.f;
    each_entry<DK>(w, ch, wave, lane, [&](int ct, int i, size_t at) { w.sT[at] = S[ct][i] * d; });
  }
}

// Start states of a chain's segments, in walk order: S -> M S + B over each one's transfer and end state.  The
// start replaces the end state it came from; the caller's own is copied, because the last segment may
// write its final state over it while others have not begun.  fp32 products: M goes through LDS, S stays in registers.
// One segment after another, a workgroup for each 64 value columns: latency, 63 us for 16 heads over 131,072 tokens (d = 128).
template <int DK>
__global__ __launch_bounds__(NT) void gdr_link_kernel(const GdrParams gp, bool rev) {
  constexpr int CT = DK / 16, LD = DK + 4;
  extern __shared__ __align__(16) char smem[];
  float* sM = (float*)smem;  // [DK][LD]
  const LinaWalk& w = gp.p.w;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, g = lane >> 4, n = lane & 15;
  Chain ch;
  if (!ch.place(gp.p, rev, blockIdx.x)) return;
  if (ch.sg != 0 || ch.nsg == 1) return;  // one workgroup for each chain
  f32x4_t S[CT];
#pragma unroll
  for (int ct = 0; ct < CT; ++ct) S[ct] = zero4();
  if (w.s0) each_entry<DK>(w, ch, wave, lane, [&](int ct, int i, size_t at) { S[ct][i] = w.s0[at]; });
  auto put = [&](int64_t piece) {
    f32x4_t* to = (f32x4_t*)(w.seg_state + seg_at(w, ch, piece, ch.vt) * (DK * VT));
#pragma unroll
    for (int ct = 0; ct < CT; ++ct) to[ct * NT + tid] = S[ct];
  };
  put(ch.start(gp.p));
  for (int j = 0; j < ch.nsg - 1; ++j) {
    const int64_t piece = ch.end(rev, rev ? ch.nsg - 1 - j : j);
    f32x4_t X[CT];
    const f32x4_t* B = (const f32x4_t*)(w.seg_state + seg_at(w, ch, piece, ch.vt) * (DK * VT));
    const f32x4_t* M = (const f32x4_t*)(gp.a.transfer + ((size_t)piece * w.H + ch.h) * (DK * DK));
#pragma unroll
    for (int ct = 0; ct < CT; ++ct) X[ct] = B[ct * NT + tid];
    __syncthreads();
#pragma unroll
    for (int vt = 0; vt < DK / VT; ++vt)
#pragma unroll
      for (int ct = 0; ct < CT; ++ct) {
        const f32x4_t m = M[(vt * CT + ct) * NT + tid];
#pragma unroll
        for (int i = 0; i < 4; ++i) sM[(16 * ct + 4 * g + i) * LD + vt * VT + 16 * wave + n] = m[i];
      }
    __syncthreads();
#pragma unroll
    for (int ct = 0; ct < CT; ++ct)
#pragma unroll
      for (int kt = 0; kt < CT; ++kt) mm16(X[ct], *(const f32x4_t*)&sM[(16 * ct + n) * LD + channel(kt, 4 * g)], S[kt]);
#pragma unroll
    for (int ct = 0; ct < CT; ++ct) S[ct] = X[ct];
    put(piece);
  }
}

template <typename K, typename... P>
hipError_t launch(K kern, unsigned blocks, int threads, int lds, void* stream, const P&... p) {
  if (blocks == 0) return hipSuccess;
  if (lds > 64 * 1024) {
    const hipError_t e = hipFuncSetAttribute((const void*)kern, hipFuncAttributeMaxDynamicSharedMemorySize, lds);
    if (e != hipSuccess) return e;
  }
  hipLaunchKernelGGL(kern, dim3(blocks), dim3(threads), lds, (hipStream_t)stream, p...);
  return hipGetLastError();
}

GdrParams params(const GdrWalk& a) {
  GdrParams gp;
  gp.a = a;
  const LinaWalk& w = a.walk;
  WalkParams& p = gp.p;
  p.w = w;
  p.nv = w.dv / VT;
  p.rows = w.cs ? w.T : (int64_t)w.n * w.T;
  const int64_t nch = ((int64_t)w.T + C - 1) / C;
  p.nseg = w.cs ? lina_pieces(w.T, w.n, w.L) : (int64_t)w.n * (nch > 0 ? (nch + w.L - 1) / w.L : 1);
  p.ends = w.split ? lina_ends(w.cs != nullptr, w.T, w.n, w.L) : 0;
  gp.chunks = gdr_chunks(w.cs != nullptr, w.T, w.n);
  return gp;
}

template <typename T, int DK, bool REV>
hipError_t prep(const GdrParams& gp) {
  const int64_t blocks = gp.chunks * ((gp.p.w.H + 3) / 4);
  if (blocks > 0xFFFFFFFFll / 256) return hipErrorInvalidValue;
  return launch(gdr_prep_kernel<T, DK, REV>, (unsigned)blocks, 256, 0, gp.p.w.stream, gp);
}
template <typename T, int DK>
hipError_t prep(const GdrParams& gp) {
  return gp.p.w.rev ? prep<T, DK, true>(gp) : prep<T, DK, false>(gp);
}

// Slots of a packed batch's list that a sequence's segments but its last can have: they are L chunks long, and the list has
// those first.  (In reverse it is the first one that no other starts from: the last, of any length, is walked too.)
int64_t cut_slots(const WalkParams& p) {
  const LinaWalk& w = p.w;
  return w.cs ? std::min(p.nseg, (int64_t)w.T / ((int64_t)C * (w.L - 1) + 1)) : p.nseg;
}

template <typename T, int DK, int MODE>
hipError_t walk(GdrParams gp) {
  if constexpr (is_seg(MODE)) {
    gp.p.nv += DK / VT;
    if (!is_rev(MODE)) gp.p.nseg = cut_slots(gp.p);
  }
  return launch(gdr_walk_kernel<T, DK, MODE>, walk_blocks(gp.p), 2 * NT, WalkLds<T, DK, MODE>::BYTES, gp.p.w.stream, gp);
}
template <typename T, int DK>
hipError_t walk(const GdrParams& gp) {
  return gp.p.w.rev ? walk<T, DK, kRev>(gp) : gp.a.train ? walk<T, DK, kTrain>(gp) : walk<T, DK, kFwd>(gp);
}

template <typename T, int DK>
hipError_t segments(const GdrParams& gp) {
  const hipError_t e = gp.p.w.rev ? walk<T, DK, kSegRev>(gp) : walk<T, DK, kSegFwd>(gp);
  if (e != hipSuccess) return e;
  GdrParams link = gp;
  link.p.nseg = cut_slots(gp.p);
  return launch(gdr_link_kernel<DK>, walk_blocks(link.p), NT, DK * (DK + 4) * 4, gp.p.w.stream, link, gp.p.w.rev);
}

template <typename F>
hipError_t by_type(const LinaWalk& w, F f) {
  if (w.bf16) return w.dk == 128 ? f(bf16_t{}, std::integral_constant<int, 128>{}) : f(bf16_t{}, std::integral_constant<int, 64>{});
  return w.dk == 128 ? f(float{}, std::integral_constant<int, 128>{}) : f(float{}, std::integral_constant<int, 64>{});
}

}  // namespace

hipError_t launch_gdr_prep(const GdrWalk& a) {
  return by_type(a.walk, [&](auto t, auto dk) { return prep<decltype(t), decltype(dk)::value>(params(a)); });
}
hipError_t launch_gdr_segments(const GdrWalk& a) {
  if (!a.walk.split) return hipSuccess;
  return by_type(a.walk, [&](auto t, auto dk) { return segments<decltype(t), decltype(dk)::value>(params(a)); });
}
hipError_t launch_gdr_walk(const GdrWalk& a) {
  return by_type(a.walk, [&](auto t, auto dk) { return walk<decltype(t), decltype(dk)::value>(params(a)); });
}

}  // namespace kda
