// kda_lina.hip -- chunked linear attention with a decay for each head: one walk kernel for
// the forward and the three products of its backward.
//
//   S_t = e^{g_t} S_{t-1} + k_t v_t^T,   o_t = S_t^T q_t.
//
// With G the inclusive sum of g inside a chunk of C = 64 tokens,
//   o_i = e^{G_i} S^T q_i + sum_{j <= i} r_ij (q_i . k_j) v_j,     r_ij = e^{G_i - G_j},
//   S  <- e^{G_C} S + sum_j e^{G_C - G_j} k_j v_j^T.
// The gradients are the same walk over other operands (d_o = u):
//   dq = walk(Q = u, K = v, V = k) in order, from S_0^T;
//   dk = walk(Q = v, K = u, V = q) and dv = walk(Q = k, K = q, V = u) in reverse token
//   order, from dS_T (transposed for dk); in reverse order the decay of a step is the one
//   of the token after it.  The walk of dv ends in e^{-g_1} dS_0.
// The gradient of g_t sums r_ij (q_i . k_j)(u_i . v_j) over all pairs j < t <= i; the walks
// leave its parts per token (a, b, e below) and lina_ddecay_kernel adds them up:
//   a_i = q_i . (dq_i's part from the chunk's start state)     b_j = k_j . (dk_j's from R)
//   e_t = sum over the chunk of M_tj - M_jt, M_ij = r_ij (q_i . k_j)(u_i . v_j), i > j
//   dg_t = sum_{i >= t} e_i + sum_{j < t} b_j - sum_{i < t} a_i + D,  D = <S, R> e^{g} at the
//   chunk's first token; D moves from chunk to chunk by sum b - sum a, and every
//   lina_keep() chunks it is taken afresh from the two states, so that no rounding error
//   travels further than that.
//
// Four waves walk one chain (sequence or segment, head, 64 value columns) or keep its state beside
// others that feed them; wave w keeps columns 16 w .. 16 w + 15 of the state in fp32 accumulators,
// which serve as matrix-core operands without leaving the registers.  Products run transposed (rows are
// value columns, columns are tokens), so that a lane holds four neighbouring columns of one
// token and stores them at once; K and V are read along the token axis with the LDS
// transpose loads.
//
// Precision (bf16 inputs): sums, decays and the state are fp32, and what enters the state,
// e^{G_C - G_j} v_j, goes through the matrix cores as three bf16 terms, all of its 24 bits (two
// terms left the state 2.4e-6 of its norm off, three 2e-7, as fp32 sums do; a sixth more matrix
// work).  Rounded to bf16 (off by at most 2^-8 relative, as the output itself is) are P = r o QK^T
// and the state where it is multiplied by q: outputs are off by 2.3e-3 of their norm, 1.66e-3 of which is their own
// rounding, 1.35e-3 the state's and 0.96e-3 P's.  Two terms of the state cost a forward 299 -> 322 us (B4 H32 T8K), two of
// both 335 (H16 T128K 880 -> 952).  In the walks that a and b are taken from, the state
// meets its rows as three terms too: D is a small difference of long sums of a and b, and with
// two-term operands its error was 1e-5 of the gradient's norm, with three at most 7e-7.
#include <algorithm>
#include <type_traits>

#include "kda_lina_tile.h"

namespace kda {

namespace {

// bf16: eight waves, two to a SIMD, one barrier per chunk.  Waves 0-3 keep the state and make
// the outputs of chunk c; waves 4-7 meanwhile write the tiles of chunk c + 2 to LDS (fetched two
// steps before, into the one of two register sets that is free), compute its decays, and make P of
// chunk c + 1, so that neither the fetch nor Q K^T lies on the state's path.  Tiles are triple-, P
// double-buffered.  B4 H32 T8K, d = 128 (256 chains, one to a compute unit): 290 us, 3.8 TB/s of the
// bytes that have to move (copies: 5.15).  Loads and stores of the same pattern with no arithmetic take
// 234 us; a step is 4,800 cycles, matrix cores busy 27% and vector units 44% of them, at the 1.75 GHz
// that the clock settles at.  With all work in four waves it took 450 us, with twelve waves (fetch and
// P apart) 300.
template <int DK, int DOT>
struct PipeLds {
  static constexpr int TILES = 2 * Tile<bf16_t, DK>::BYTES + Tile<bf16_t, VT>::BYTES;
  static constexpr int P = 3 * TILES;
  static constexpr int X = P + 2 * Tile<bf16_t, 64>::BYTES;
  static constexpr int BYTES = X + (DOT == kDotCross ? 2 * Tile<bf16_t, VT>::BYTES : 0);
};

template <int DK, bool REV, int DOT>
__global__ __launch_bounds__(2 * NT) void lina_walk_bf16_kernel(const WalkParams p) {
  typedef bf16_t T;
  typedef PipeLds<DK, DOT> Lds;
  extern __shared__ __align__(16) char smem[];
  __shared__ Decays dec[3];
  __shared__ float sdot[DOT == kDotNone ? 1 : 2][4][C], sdot2[DOT == kDotCross ? 2 : 1][C];
  auto tK = [&](int it) { return smem + it % 3 * Lds::TILES; };
  auto tV = [&](int it) { return tK(it) + Tile<T, DK>::BYTES; };
  auto tQ = [&](int it) { return tV(it) + Tile<T, VT>::BYTES; };
  auto tP = [&](int it) { return smem + Lds::P + (it & 1) * Tile<T, 64>::BYTES; };
  auto tX = [&](int it) { return smem + Lds::X + (it & 1) * Tile<T, VT>::BYTES; };

  const LinaWalk& w = p.w;
  const int tid = threadIdx.x & (NT - 1), lane = tid & 63, wave = tid >> 6;
  Chain ch;
  if (!ch.place(p, REV, blockIdx.x)) return;
  const int steps = ch.last - ch.first;
  auto chunk = [&](int it) { return REV ? ch.last - 1 - it : ch.first + it; };
  const Operand<T> x(w.x, w, ch.h, w.dv, ch.vt * VT);

  if (threadIdx.x >= NT) {
    if (steps == 0) return;
    const Operand<T> q(w.q, w, ch.h, DK, 0), k(w.k, w, ch.h, DK, 0), v(w.v, w, ch.h, w.dv, ch.vt * VT);
    struct Tiles {
      Stage<T, DK> q, k;
      Stage<T, VT> v, x;
    } ra, rb;
    auto fetch_to = [&](Tiles& r, int it) {
      const int c = chunk(it);
      const int64_t t = ch.lo + (int64_t)c * C;
      const uint32_t n = ch.rows(c);
      r.k.load(k.rows(t, n), k.step, REV, tid);
      r.q.load(q.rows(t, n), q.step, REV, tid);
      r.v.load(v.rows(t, n), v.step, REV, tid);
      if constexpr (DOT == kDotCross) r.x.load(x.rows(t, n), x.step, REV, tid);
    };
    auto put_from = [&](const Tiles& r, int it) {
      r.k.store(tK(it), tid);
      r.q.store(tQ(it), tid);
      r.v.store(tV(it), tid);
      if constexpr (DOT == kDotCross) r.x.store(tX(it), tid);
    };
    // wave 0's logarithms of the decays come with the tiles of their chunk, a step before these
    // are written and two before they are used
    float ga = 0.f, gb = 0.f;
    auto fetch_decay = [&](float& g, int it) {
      if (wave == 0) g = it < steps ? row_decay<REV>(w, ch, chunk(it), lane) : 0.f;
    };
    auto decays = [&](float g, int it) {
      if (wave == 0 && it < steps) chunk_decays(dec[it % 3], g, lane);
    };
    auto scores = [&](int it) {
      make_p<T, DK, DOT>(tQ(it), tK(it), tV(it), tX(it), tP(it), dec[it % 3], sdot[DOT == kDotNone ? 0 : it & 1][wave],
                         sdot2[DOT == kDotCross ? it & 1 : 0], wave, lane);
    };
    fetch_decay(ga, 0);
    fetch_to(ra, 0);
    fetch_decay(gb, 1);
    if (steps > 1) fetch_to(rb, 1);
    decays(ga, 0);
    put_from(ra, 0);
    fetch_decay(ga, 2);
    if (steps > 2) fetch_to(ra, 2);
    decays(gb, 1);
    lds_barrier();
    if (steps > 1) put_from(rb, 1);
    fetch_decay(gb, 3);
    if (steps > 3) fetch_to(rb, 3);
    if (ch.skip == 0) scores(0);
    lds_barrier();
    auto step = [&](Tiles& r, float& g, int it) {
      if (it + 2 < steps) put_from(r, it + 2);
      decays(g, it + 2);
      fetch_decay(g, it + 4);
      if (it + 4 < steps) fetch_to(r, it + 4);
      if (it + 1 < steps && it + 1 >= ch.skip) scores(it + 1);
      if constexpr (DOT == kDotRow)
        if (wave == 0 && it > 0) store_dots<DOT, REV>(p, ch, chunk(it - 1), sdot[(it - 1) & 1], sdot2[0], lane);
      lds_barrier();
    };
    for (int it = 0; it < steps; it += 2) {
      step(ra, ga, it);
      if (it + 1 < steps) step(rb, gb, it + 1);
    }
    if constexpr (DOT == kDotRow)
      if (wave == 0) store_dots<DOT, REV>(p, ch, chunk(steps - 1), sdot[(steps - 1) & 1], sdot2[0], lane);
  } else {
    f32x4_t S[DK / 16];
    start_state<DK>(p, ch, REV, tid, S);
    DotRows<T> rd, xd;
    auto fetch = [&](int it) {
      const int c = chunk(it);
      if constexpr (DOT == kDotRow) rd.load(x.rows(ch.lo + (int64_t)c * C, ch.rows(c)), x.step, REV, wave, lane);
    };
    if (steps > 0) {
      fetch(0);
      lds_barrier();
      lds_barrier();
    }
    auto values = [&](Frag<T> (&fv)[2], int it) {
      tok_frag<T, VT>(fv[0], tV(it), tok_base<T, VT, false>(lane), 16 * wave, 0, lane);
      tok_frag<T, VT>(fv[1], tV(it), tok_base<T, VT, false>(lane), 16 * wave, 1, lane);
    };
    for (int it = 0; it < ch.skip; ++it) {
      Frag<T> fv[2];
      values(fv, it);
      add_chunk<T, DK>(S, fv, tK(it), dec[it % 3], lane);
      lds_barrier();
    }
    for (int it = ch.skip; it < steps; ++it) {
      const int c = chunk(it);
      const Decays& dc = dec[it % 3];
      if constexpr (DOT == kDotRow) {
        xd = rd;
        if (it + 1 < steps) fetch(it + 1);
        if (!REV && c > 0 && c % lina_keep(true) == 0) store_snap<DK>(p, ch, c, tid, S);
      }
      f32x4_t acc[4];
      from_state<T, DK, DOT == kDotRow>(S, tQ(it), lane, acc);
      scale_rows(acc, dc, lane);
      if constexpr (DOT == kDotRow) xd.dot(acc, sdot[it & 1][wave], lane);
      if constexpr (DOT == kDotCross)
        if (wave == 0) store_dots<DOT, REV>(p, ch, c, sdot[it & 1], sdot2[it & 1], lane);
      Frag<T> fv[2];
      values(fv, it);
      add_intra<T, VT>(acc, fv, tP(it), tV(it), 16 * wave, lane);
      store_out<T, REV>(acc, w, ch, c, wave, lane);
      add_chunk<T, DK>(S, fv, tK(it), dc, lane);
      if constexpr (DOT == kDotRow && REV)
        if (c % lina_keep(true) == 0) store_anchor<DK>(p, ch, c, tid, S);
      lds_barrier();
    }
    store_state<DK, REV>(p, ch, tid, S);
  }
}

// The two reverse walks of the backward in one, for d_k = d_v = D (bf16): dk = walk(Q = v, K = u,
// V = q) and dv = walk(Q = k, K = q, V = u) meet the same four tiles, so these are fetched and
// written to LDS once, and the pair sums M = r o (q k^T) o (u v^T) come from the two score
// matrices the walks need anyway.  Twelve waves, three to a SIMD: four keep 64 columns of the
// transposed state and make dk, four 64 columns of the state and make dv, four fetch, write and
// make the scores of the next chunk.  A step has two halves: from the states (meanwhile the next
// tiles and this chunk's P go to LDS), then P V and the states' update (meanwhile the next scores,
// kept in registers).  B4 H32 T8K, d = 128: 650 to 700 us (with the clock), 11,900 cycles a step, of
// which the vector units are busy 46% and the matrix cores 26%: the two chains of dependent products
// between two barriers, not memory (1.75 GB).  Two separate walks took 870.
template <int D>
struct RevLds {
  static constexpr int Q = 0, K = Tile<bf16_t, D>::BYTES, V = 2 * K, U = 3 * K, TILES = 4 * K;
  static constexpr int PK = 2 * TILES, PV = PK + Tile<bf16_t, 64>::BYTES;
  static constexpr int BYTES = PV + Tile<bf16_t, 64>::BYTES;
};

struct RevParams {
  WalkParams k, v;  // the walks of dk and dv
};

template <int D, bool WANT>
__global__ __launch_bounds__(3 * NT) void lina_reverse_kernel(const RevParams p) {
  typedef bf16_t T;
  typedef RevLds<D> Lds;
  constexpr int KS = D / 32;
  extern __shared__ __align__(16) char smem[];
  __shared__ Decays dec[2];
  __shared__ __align__(16) float srow[WANT ? 4 : 1][C], scol[WANT ? 4 : 1][C];
  __shared__ float sown[WANT ? C : 1];
  auto tile = [&](int it, int at) { return smem + (it & 1) * Lds::TILES + at; };

  const int tid = threadIdx.x & (NT - 1), lane = tid & 63, wave = tid >> 6, g = lane >> 4, n = lane & 15;
  Chain ch;
  if (!ch.place(p.k, true, blockIdx.x)) return;
  const int steps = ch.last - ch.first;
  auto chunk = [&](int it) { return ch.last - 1 - it; };
  const int role = threadIdx.x / NT;

  if (role == 2) {
    if (steps == 0) return;
    const LinaWalk& w = p.v.w;
    const Operand<T> v(w.x, w, ch.h, D, 0), u(w.v, w, ch.h, D, 0);
    Stage<T, D, true> rv, ru;
    float lg = 0.f;
    auto fetch = [&](int it) {
      const int c = chunk(it);
      const int64_t t = ch.lo + (int64_t)c * C;
      const uint32_t have = ch.rows(c);
      if (wave == 1) lg = row_decay<true>(w, ch, c, lane);
      ru.load(u.rows(t, have), u.step, true, tid);
      rv.load(v.rows(t, have), v.step, true, tid);
    };
    auto put = [&](int it) {
      if (wave == 1) chunk_decays(dec[it & 1], lg, lane);
      ru.store(tile(it, Lds::U), tid);
      rv.store(tile(it, Lds::V), tid);
    };
    uint2 pk[4], pv[4];  // the wave's rows of both P, on their way to LDS
    auto scores = [&](int it) {
      const Decays& dc = dec[it & 1];
      const int row = 16 * wave + n;
      Frag<T> fv[KS], fk[KS];
      const uint32_t rb = row_base<T, D, true>(lane);
      auto at = [&](int t, int r0) { return rows_at<T, D, true>(rb + t, r0); };
      const uint32_t ov = at(Lds::V, 16 * wave), ok = at(Lds::K, 16 * wave);
      const char* const t0 = tile(it, 0);
#pragma unroll
      for (int s = 0; s < KS; ++s) {
        row_frag<T>(fv[s], t0, ov, s);
        row_frag<T>(fk[s], t0, ok, s);
      }
      const float ih = dc.hi[row], il = dc.lo[row];
      float own = 0.f;
#pragma unroll
      for (int J = 0; J < 4; ++J) {
        float x[4] = {0.f, 0.f, 0.f, 0.f}, y[4] = {0.f, 0.f, 0.f, 0.f};
        if (J <= wave) {
          f32x4_t a = zero4(), b = zero4();
          const uint32_t ru = at(Lds::U, 16 * J), rq = at(Lds::Q, 16 * J);
#pragma unroll
          for (int s = 0; s < KS; ++s) {
            Frag<T> f;
            row_frag<T>(f, t0, ru, s);
            mma(a, f, fv[s]);
            row_frag<T>(f, t0, rq, s);
            mma(b, f, fk[s]);
          }
          const float4 jh = *(const float4*)&dc.hi[16 * J + 4 * g], jl = *(const float4*)&dc.lo[16 * J + 4 * g];
          const float jhs[4] = {jh.x, jh.y, jh.z, jh.w}, jls[4] = {jl.x, jl.y, jl.z, jl.w};
          float m[4], cols = 0.f;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int j = 16 * J + 4 * g + i;
            const float r = fast_exp2((ih - jhs[i]) + (il - jls[i]));
            x[i] = j <= row ? a[i] * r : 0.f;
            y[i] = j <= row ? b[i] * r : 0.f;
            m[i] = j < row ? (a[i] * r) * b[i] : 0.f;
          }
          if (WANT && (p.k.nv == 1 || ((wave + J) & 1) == ch.vt)) {  // M is whole: half of its tiles here
#pragma unroll
            for (int i = 0; i < 4; ++i) own += m[i];
            cols = row16_sums(m, n);
          }
          if constexpr (WANT)
            if (n < 4) scol[wave][16 * J + 4 * g + n] = cols;
        }
        pk[J] = make_uint2(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]));
        pv[J] = make_uint2(pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]));
      }
      if constexpr (WANT) {
        own += __shfl_xor(own, 16);
        own += __shfl_xor(own, 32);
        if (g == 0) sown[row] = own;
      }
    };
    fetch(0);
    put(0);
    if (steps > 1) fetch(1);
    lds_barrier();
    scores(0);
    lds_barrier();
    for (int it = 0; it < steps; ++it) {
      const uint32_t pb = row_base<T, 64, true>(lane);
#pragma unroll
      for (int J = 0; J < 4; ++J)
        if (J <= (wave | 1)) {
          const uint32_t at = 16 * wave * Tile<T, 64>::RB + (pb ^ (J * 32));
          *(uint2*)(smem + Lds::PK + at) = pk[J];
          *(uint2*)(smem + Lds::PV + at) = pv[J];
        }
      if constexpr (WANT)
        if (wave == 0) store_dots<kDotCross, true>(p.v, ch, chunk(it), scol, sown, lane);
      if (it + 1 < steps) put(it + 1);
      if (it + 2 < steps) fetch(it + 2);
      lds_barrier();
      if constexpr (WANT)
        if (wave == 0) store_dots<kDotRow, true>(p.k, ch, chunk(it), srow, sown, lane);
      if (it + 1 < steps) scores(it + 1);
      lds_barrier();
    }
    return;
  }

  // dk: rows of v and u against q; dv: rows of k and q against u
  auto walk = [&](const WalkParams& wp, int tq, int tk, int tv, int tx, int tp, auto exact, auto fetch, auto put) {
    constexpr bool EXACT = decltype(exact)::value;
    const int c0 = ch.vt * VT + 16 * wave;
    f32x4_t S[D / 16];
    if (steps > 0) fetch(0);
    start_state<D>(wp, ch, true, tid, S);
    if (steps > 0) {
      put(0);
      if (steps > 1) fetch(1);
      lds_barrier();
      lds_barrier();
    }
    for (int it = 0; it < steps; ++it) {
      const int c = chunk(it);
      const Decays& dc = dec[it & 1];
      if (it + 1 < steps) put(it + 1);
      if (it + 2 < steps) fetch(it + 2);
      f32x4_t acc[4];
      from_state<T, D, EXACT, true>(S, tile(it, tq), lane, acc);
      scale_rows(acc, dc, lane);
      if constexpr (EXACT) {  // with the rows of k: b
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          float x[4];
          ld_quad<T>(tile(it, tx) + Tile<T, D>::quad(16 * t + n, c0 / 4 + g), 0, x);
          float d = acc[t][0] * x[0] + acc[t][1] * x[1] + acc[t][2] * x[2] + acc[t][3] * x[3];
          d += __shfl_xor(d, 16);
          d += __shfl_xor(d, 32);
          if (g == 0) srow[wave][16 * t + n] = d;
        }
      }
      Frag<T> fv[2];
      tok_frag<T, D>(fv[0], tile(it, tv), tok_base<T, D, true>(lane), c0, 0, lane);
      tok_frag<T, D>(fv[1], tile(it, tv), tok_base<T, D, true>(lane), c0, 1, lane);
      lds_barrier();
      add_intra<T, D, true>(acc, fv, smem + tp, tile(it, tv), c0, lane);
      store_out<T, true, true>(acc, wp.w, ch, c, wave, lane);
      add_chunk<T, D, true>(S, fv, tile(it, tk), dc, lane);
      if constexpr (EXACT)
        if (c % lina_keep(true) == 0) store_anchor<D>(wp, ch, c, tid, S);
      lds_barrier();
    }
    store_state<D, true>(wp, ch, tid, S);
  };
  if (role == 0) {
    walk(p.k, Lds::V, Lds::U, Lds::Q, Lds::K, Lds::PK, std::integral_constant<bool, WANT>{}, [](int) {}, [](int) {});
  } else {  // with the fewer products, these waves fetch q and k as well
    const LinaWalk& w = p.v.w;
    const Operand<T> q(w.k, w, ch.h, D, 0), k(w.q, w, ch.h, D, 0);
    Stage<T, D, true> rq, rk;
    walk(
        p.v, Lds::K, Lds::Q, Lds::U, Lds::V, Lds::PV, std::false_type{},
        [&](int it) {
          const int c = chunk(it);
          const int64_t t = ch.lo + (int64_t)c * C;
          rq.load(q.rows(t, ch.rows(c)), q.step, true, tid);
          rk.load(k.rows(t, ch.rows(c)), k.step, true, tid);
        },
        [&](int it) {
          rq.store(tile(it, Lds::Q), tid);
          rk.store(tile(it, Lds::K), tid);
        });
  }
}

// fp32: one workgroup of four waves, one tile buffer, chunk after chunk; products of 16 x 16 x 4 at
// 32 cycles each.  d = 64: 11 us for a chain's first chunk (latency of its loads and products), 6.5 for
// each further one, 2.6 where only its state is needed; chains are therefore cut to single chunks
// while there are compute units to spare.
template <int DK, bool REV, int DOT>
__device__ __forceinline__ void walk_f32_body(const WalkParams& p, unsigned block) {
  typedef float T;
  typedef Tile<T, DK> KT;
  typedef Tile<T, VT> VTl;
  extern __shared__ __align__(16) char smem[];
  char* sK = smem;
  char* sV = sK + KT::BYTES;
  char* sQ = sV + VTl::BYTES;
  char* sP = sQ + KT::BYTES;
  char* sX = sP + Tile<T, 64>::BYTES;  // kDotCross only
  __shared__ Decays dec[2];
  __shared__ float sdot[4][C], sdot2[C];

  const LinaWalk& w = p.w;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  Chain ch;
  if (!ch.place(p, REV, block)) return;
  const Operand<T> q(w.q, w, ch.h, DK, 0), k(w.k, w, ch.h, DK, 0), v(w.v, w, ch.h, w.dv, ch.vt * VT),
      x(w.x, w, ch.h, w.dv, ch.vt * VT);
  Stage<T, DK> rq, rk;
  Stage<T, VT> rv, rx;
  DotRows<T> rd, xd;
  auto fetch = [&](int c) {
    const int64_t t = ch.lo + (int64_t)c * C;
    const uint32_t n = ch.rows(c);
    rk.load(k.rows(t, n), k.step, REV, tid);
    rv.load(v.rows(t, n), v.step, REV, tid);
    rq.load(q.rows(t, n), q.step, REV, tid);
    if constexpr (DOT == kDotCross) rx.load(x.rows(t, n), x.step, REV, tid);
    if constexpr (DOT == kDotRow) rd.load(x.rows(t, n), x.step, REV, wave, lane);
  };
  float rg = 0.f;
  auto fetch_decay = [&](int c) {
    if (wave == 0) rg = row_decay<REV>(w, ch, c, lane);
  };
  f32x4_t S[DK / 16];
  start_state<DK>(p, ch, REV, tid, S);
  const int steps = ch.last - ch.first;
  auto chunk = [&](int it) { return REV ? ch.last - 1 - it : ch.first + it; };
  if (steps > 0) {
    fetch_decay(chunk(0));
    if (wave == 0) chunk_decays(dec[0], rg, lane);
    fetch_decay(chunk(1));
    fetch(chunk(0));
  }
  for (int it = 0; it < steps; ++it) {
    const int c = chunk(it);
    const Decays& dc = dec[it & 1];
    lds_barrier();  // the previous chunk's tiles are consumed
    rq.store(sQ, tid);
    rk.store(sK, tid);
    rv.store(sV, tid);
    if constexpr (DOT == kDotCross) rx.store(sX, tid);
    if constexpr (DOT == kDotRow) xd = rd;
    // the next chunk's decays; their logarithms run a chunk ahead of the tiles, because loads
    // return in order and waiting for one behind the tiles would wait for these
    if (wave == 0 && it + 1 < steps) chunk_decays(dec[(it + 1) & 1], rg, lane);
    if (it + 2 < steps) fetch_decay(chunk(it + 2));
    if (it + 1 < steps) fetch(chunk(it + 1));
    lds_barrier();
    Frag<T> fv[2];
    auto values = [&] {
      tok_frag<T, VT>(fv[0], sV, tok_base<T, VT, false>(lane), 16 * wave, 0, lane);
      tok_frag<T, VT>(fv[1], sV, tok_base<T, VT, false>(lane), 16 * wave, 1, lane);
    };
    if (it < ch.skip) {
      values();
      add_chunk<T, DK>(S, fv, sK, dc, lane);
      continue;
    }
    if constexpr (DOT == kDotRow && !REV)
      if (c > 0 && c % lina_keep(false) == 0) store_snap<DK>(p, ch, c, tid, S);
    make_p<T, DK, DOT>(sQ, sK, sV, sX, sP, dc, sdot[wave], sdot2, wave, lane);
    f32x4_t acc[4];
    from_state<T, DK, false>(S, sQ, lane, acc);
    scale_rows(acc, dc, lane);
    if constexpr (DOT == kDotRow) xd.dot(acc, sdot[wave], lane);
    lds_barrier();
    if constexpr (DOT != kDotNone)
      if (wave == 1) store_dots<DOT, REV>(p, ch, c, sdot, sdot2, lane);
    values();
    add_intra<T, VT>(acc, fv, sP, sV, 16 * wave, lane);
    store_out<T, REV>(acc, w, ch, c, wave, lane);
    add_chunk<T, DK>(S, fv, sK, dc, lane);
    if constexpr (DOT == kDotRow && REV)
      if (c % lina_keep(false) == 0) store_anchor<DK>(p, ch, c, tid, S);
  }
  store_state<DK, REV>(p, ch, tid, S);
}

template <int DK, bool REV, int DOT>
__global__ __launch_bounds__(NT) void lina_walk_f32_kernel(const WalkParams p) {
  walk_f32_body<DK, REV, DOT>(p, blockIdx.x);
}

// The walks of dq and dv side by side: they need nothing of each other, and fp32 calls are seldom
// large enough to fill the machine with one (2 x 1,001 tokens, H4, d = 64: 19 us for both, 17 for
// one).
struct PairParams {
  WalkParams q, v;
  unsigned blocks_q;
};

template <int DKQ, int DKV, bool WANT>
__global__ __launch_bounds__(NT) void lina_pair_f32_kernel(const PairParams p) {
  if (blockIdx.x < p.blocks_q) walk_f32_body<DKQ, false, WANT ? kDotRow : kDotNone>(p.q, blockIdx.x);
  else walk_f32_body<DKV, true, WANT ? kDotCross : kDotNone>(p.v, blockIdx.x - p.blocks_q);
}

// End states of the segments from a zero start: the walk without its outputs.  Two tile
// buffers, one barrier per chunk; small enough for three workgroups on a compute unit.  Walks of one
// call that have d_k in common (the backward's three) go in one launch.  H16 T128K, d = 128: 270 us
// for 1.07 GB of k and v (4.0 TB/s; matrix cores busy 33%, vector units 42%); with a step's decays made in that step by one wave it took 310 (all others
// waited for its prefix sums).  Held to 168 registers for the third workgroup: with 188 a backward of
// H4 T32K took 223 us instead of 215.
struct SegParams {
  WalkParams p[3];
  unsigned end[3];  // their workgroups, running sums
};

template <typename T, int DK>
__global__ __launch_bounds__(NT, sizeof(T) == 2 ? 3 : 1) void lina_segment_kernel(const SegParams all) {
  const int which = (blockIdx.x >= all.end[0]) + (blockIdx.x >= all.end[1]);
  const WalkParams& p = all.p[which];
  const unsigned block = blockIdx.x - (which ? all.end[which - 1] : 0);
  const bool rev = p.w.rev;
  constexpr int TILES = Tile<T, DK>::BYTES + Tile<T, VT>::BYTES;
  extern __shared__ __align__(16) char smem[];
  __shared__ ColDecays dec[8];
  const LinaWalk& w = p.w;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  Chain ch;
  if (!ch.place(p, rev, block)) return;
  if (ch.tail) return keep_start<DK>(p, ch, tid);  // nobody starts from a tail's end
  const Operand<T> k(w.k, w, ch.h, DK, 0), v(w.v, w, ch.h, w.dv, ch.vt * VT);
  Stage<T, DK> rk;
  Stage<T, VT> rv;
  float rg = 0.f;
  const int steps = ch.last - ch.first;
  auto chunk = [&](int it) { return rev ? ch.last - 1 - it : ch.first + it; };
  auto fetch = [&](int it) {
    if (it >= steps) return;
    const int c = chunk(it);
    const int64_t t = ch.lo + (int64_t)c * C;
    const uint32_t n = ch.rows(c);
    rk.load(k.rows(t, n), k.step, rev, tid);
    rv.load(v.rows(t, n), v.step, rev, tid);
  };
  // four chunks' decays at a time, a wave each: their prefix sums would hold up every step
  auto fetch_decays = [&](int it) {
    it += wave;
    if (it < steps) rg = rev ? row_decay<true>(w, ch, chunk(it), lane) : row_decay<false>(w, ch, chunk(it), lane);
  };
  auto decays = [&](int it) {
    it += wave;
    if (it < steps) chunk_decays(dec[it & 7], rg, lane);
  };
  auto put = [&](int it) {
    if (it >= steps) return;
    char* t = smem + (it & 1) * TILES;
    rk.store(t, tid);
    rv.store(t + Tile<T, DK>::BYTES, tid);
  };
  f32x4_t S[DK / 16];
#pragma unroll
  for (int ct = 0; ct < DK / 16; ++ct) S[ct] = zero4();
  float total = 1.f;
  fetch_decays(0);
  fetch(0);
  decays(0);
  fetch_decays(4);
  put(0);
  fetch(1);
  lds_barrier();
  for (int it = 0; it < steps; ++it) {
    put(it + 1);
    if (it % 4 == 0) {
      decays(it + 4);
      fetch_decays(it + 8);
    }
    fetch(it + 2);
    const ColDecays& dc = dec[it & 7];
    const char* t = smem + (it & 1) * TILES;
    Frag<T> fv[2];
    tok_frag<T, VT>(fv[0], t + Tile<T, DK>::BYTES, tok_base<T, VT, false>(lane), 16 * wave, 0, lane);
    tok_frag<T, VT>(fv[1], t + Tile<T, DK>::BYTES, tok_base<T, VT, false>(lane), 16 * wave, 1, lane);
    total *= dc.tot;
    add_chunk<T, DK>(S, fv, t, dc, lane);
    lds_barrier();
  }
  f32x4_t* to = (f32x4_t*)(w.seg_state + ch.at(p, ch.end(rev, ch.sg)) * (DK * VT));
#pragma unroll
  for (int ct = 0; ct < DK / 16; ++ct) to[ct * NT + tid] = S[ct];
  if (tid == 0 && ch.vt == 0) w.seg_dec[(size_t)ch.end(rev, ch.sg) * w.H + ch.h] = total;
}

template <typename K, typename P>
hipError_t launch(K kern, const P& p, unsigned blocks, int threads, int lds, void* stream) {
  if (blocks == 0) return hipSuccess;
  if (lds > 64 * 1024) {
    const hipError_t e = hipFuncSetAttribute((const void*)kern, hipFuncAttributeMaxDynamicSharedMemorySize, lds);
    if (e != hipSuccess) return e;
  }
  hipLaunchKernelGGL(kern, dim3(blocks), dim3(threads), lds, (hipStream_t)stream, p);
  return hipGetLastError();
}

template <int DK, bool REV, int DOT>
hipError_t walk_bf16(const WalkParams& p) {
  return launch(lina_walk_bf16_kernel<DK, REV, DOT>, p, walk_blocks(p), 2 * NT, PipeLds<DK, DOT>::BYTES, p.w.stream);
}

template <int DK>
hipError_t walk_bf16(const WalkParams& p) {
  const LinaWalk& w = p.w;
  if (w.dot == kDotCross) return w.rev ? walk_bf16<DK, true, kDotCross>(p) : hipErrorInvalidValue;
  if (w.dot == kDotRow) return w.rev ? walk_bf16<DK, true, kDotRow>(p) : walk_bf16<DK, false, kDotRow>(p);
  return w.rev ? walk_bf16<DK, true, kDotNone>(p) : walk_bf16<DK, false, kDotNone>(p);
}

template <int DK, int DOT>
constexpr int kF32Lds = 2 * Tile<float, DK>::BYTES + (DOT == kDotCross ? 3 : 2) * Tile<float, 64>::BYTES;

template <int DK, bool REV, int DOT>
hipError_t walk_f32(const WalkParams& p) {
  return launch(lina_walk_f32_kernel<DK, REV, DOT>, p, walk_blocks(p), NT, kF32Lds<DK, DOT>, p.w.stream);
}

template <int DK>
hipError_t walk_f32(const WalkParams& p) {  // the others go in pairs
  const LinaWalk& w = p.w;
  if (!w.rev) return w.dot == kDotNone ? walk_f32<DK, false, kDotNone>(p) : hipErrorInvalidValue;
  if (w.dot == kDotCross) return hipErrorInvalidValue;
  return w.dot == kDotRow ? walk_f32<DK, true, kDotRow>(p) : walk_f32<DK, true, kDotNone>(p);
}

template <int DKQ, int DKV, bool WANT>
hipError_t pair_f32(const PairParams& p) {
  constexpr int a = kF32Lds<DKQ, kDotNone>, b = kF32Lds<DKV, WANT ? kDotCross : kDotNone>;
  return launch(lina_pair_f32_kernel<DKQ, DKV, WANT>, p, p.blocks_q + walk_blocks(p.v), NT, a > b ? a : b,
                p.q.w.stream);
}

template <int DKQ, int DKV>
hipError_t pair_f32(const PairParams& p) {
  return p.q.w.dot == kDotNone ? pair_f32<DKQ, DKV, false>(p) : pair_f32<DKQ, DKV, true>(p);
}

template <typename T, int DK>
hipError_t segments(const SegParams& p) {
  return launch(lina_segment_kernel<T, DK>, p, p.end[2], NT, 2 * (Tile<T, DK>::BYTES + Tile<T, VT>::BYTES),
                p.p[0].w.stream);
}

WalkParams walk_params(const LinaWalk& w) {
  WalkParams p;
  p.w = w;
  p.nv = w.dv / VT;
  p.rows = w.cs ? w.T : (int64_t)w.n * w.T;
  const int64_t nch = ((int64_t)w.T + C - 1) / C;
  p.nseg = w.cs ? lina_pieces(w.T, w.n, w.L) : (int64_t)w.n * (nch > 0 ? (nch + w.L - 1) / w.L : 1);
  p.ends = lina_ends(w.cs != nullptr, w.T, w.n, w.L);
  return p;
}

// Packed offsets clamped to [0, T] and made non-decreasing (a running maximum), cs[0] = 0; the
// chunks of a segment, cs[n + 1]; and the list of segments (sequence, segment), the longest first
// (in 64 classes): workgroups are dealt in that order, so that no long chain starts last.  Order
// within a class is left to chance; no result depends on it.  Slots that no segment needs hold -1.
//
// Only here are the lengths known.  Whole chains take the longest one's steps or a compute unit's
// share of all steps, whichever is more; segments of `least` chunks that share and half of it again
// (their end states come first).  Prompts of 20,011 tokens, H = 32, d = 128, one of them 0.44 of all
// (1.7 shares): 308 us whole, 273 cut; 0.6 of all (2.2 shares): 369 and 283; 24 like ones: 218 whole.
constexpr int NTB = 1024;
__global__ __launch_bounds__(NTB) void lina_offsets_kernel(const int* __restrict__ cu, int nseq, int T, int least,
                                                           int chains, int cut, int link,
                                                           int64_t slots, int* __restrict__ cs,
                                                           int* __restrict__ list) {
  __shared__ int part[NTB / 64], from[64], total, longest, used;
  const int tid = threadIdx.x, lane = tid & 63, per = (nseq + NTB - 1) / NTB;
  const int s0 = min(nseq, tid * per), s1 = min(nseq, s0 + per);
  int mx = 0;
  for (int i = s0; i < s1; ++i) mx = max(mx, min(max(cu[i + 1], 0), T));
  for (int off = 1; off < 64; off <<= 1) {
    const int v = __shfl_up(mx, off);
    if (lane >= off) mx = max(mx, v);
  }
  if (lane == 63) part[tid >> 6] = mx;
  if (tid < 64) from[tid] = 0;
  if (tid == 0) cs[0] = total = longest = 0;
  __syncthreads();
  int run0 = __shfl_up(mx, 1);
  if (lane == 0) run0 = 0;
  for (int i = 0; i < tid >> 6; ++i) run0 = max(run0, part[i]);
  int L = 1;
  auto each = [&](auto fn) {  // this thread's sequences
    int run = run0;
    for (int i = s0; i < s1; ++i) {
      const int end = max(run, min(max(cu[i + 1], 0), T));
      const int nch = (end - run + C - 1) / C, nsg = nch > 0 ? (nch + L - 1) / L : 1;
      fn(i, end, nch, nsg);
      run = end;
    }
  };
  int sum = 0, top = 0;
  each([&](int, int, int nch, int) {
    sum += nch;
    top = max(top, nch);
  });
  if (top > 0) {
    atomicAdd(&total, sum);
    atomicMax(&longest, top);
  }
  __syncthreads();
  // Links: a chain of n chunks in segments of L takes 1.7 L steps of both walks and (n - 1) / L links, which L = sqrt(link n)
  // balances; with the second walk's start, twice L and the links have to be less than n.  16 chunks, d = 128: 64 us
  // whole, 69 cut; 20: 76 and 77; 24: 86 and 76.
  const int seg = max(least, (int)ceilf(sqrtf(0.1f * (float)link * (float)longest)));
  const bool segs = (int64_t)longest * cut > (int64_t)total * chains &&  // cut 160: 1.6 shares of 256
                    (link == 0 || 2.f * ((float)seg + 0.1f * (float)(link * ((longest - 1) / seg))) < (float)longest);
  L = segs ? seg : max(least, longest);
  if (tid == 0) cs[nseq + 1] = L;
  auto cls = [&](int len) { return 63 - (int)((int64_t)len * 63 / L); };
  each([&](int i, int end, int nch, int nsg) {
    cs[i + 1] = end;
    if (nsg > 1) atomicAdd(&from[0], nsg - 1);
    atomicAdd(&from[cls(nch - (nsg - 1) * L)], 1);
  });
  __syncthreads();
  if (tid < 64) {
    const int n = from[lane];
    int x = n;
    for (int off = 1; off < 64; off <<= 1) {
      const int v = __shfl_up(x, off);
      if (lane >= off) x += v;
    }
    from[lane] = x - n;
    if (lane == 63) used = x;
  }
  __syncthreads();
  each([&](int i, int, int nch, int nsg) {
    if (nsg > 1) {
      const int at = atomicAdd(&from[0], nsg - 1);
      for (int x = 0; x < nsg - 1; ++x) {
        list[2 * (at + x)] = i;
        list[2 * (at + x) + 1] = x;
      }
    }
    const int at = atomicAdd(&from[cls(nch - (nsg - 1) * L)], 1);
    list[2 * at] = i;
    list[2 * at + 1] = nsg - 1;
  });
  for (int64_t x = used + tid; x < slots; x += NTB) list[2 * x] = -1;
}

// dq, dk of heads that share them: [rows, H, d] fp32 -> [rows, heads, d], summed in order; rows
// behind a packed batch's last offset (*end) are left as they are
template <typename T>
__global__ __launch_bounds__(256) void lina_headsum_kernel(const float* __restrict__ part, void* __restrict__ out,
                                                           int64_t quads, int heads, int group, int qd,
                                                           const int* __restrict__ end) {
  if (end) quads = min(quads, (int64_t)*end * heads * qd);
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < quads; i += (int64_t)gridDim.x * 256) {
    const int64_t row = i / qd;  // (token, shared head)
    const int c = (int)(i % qd);
    const float4* src = (const float4*)part + (row * group) * qd + c;
    float4 s = src[0];
    for (int x = 1; x < group; ++x) {
      const float4 y = src[(int64_t)x * qd];
      s.x += y.x; s.y += y.y; s.z += y.z; s.w += y.w;
    }
    const float v[4] = {s.x, s.y, s.z, s.w};
    st_quad<T>((char*)out + (size_t)i * 4 * sizeof(T), v);
  }
}

// dg from the walks' parts: one workgroup of 16 waves per group of 16 chunks and head,
// wave = chunk, lane = token.  B4 H32 T8K: 20 us; sums in fp64, so that none of its roundings counts.
__global__ __launch_bounds__(kLinaDecayThreads) void lina_ddecay_kernel(const int* __restrict__ cs, int nseq, int T, int H,
                                                           int64_t rows, const float* __restrict__ a,
                                                           const float* __restrict__ b, const float* __restrict__ e,
                                                           int na, int ne, const float* __restrict__ anchor, int keep,
                                                           const float* __restrict__ g, bool g_fixed,
                                                           float* __restrict__ dg, double* __restrict__ part) {
  __shared__ double chunk_sum[kLinaGroup];
  const int64_t grp = blockIdx.x;
  const int h = blockIdx.y, lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int per = C * kLinaGroup;
  int64_t lo, hi, kept;  // kept: the sequence's first anchor
  int gi;
  if (cs) {
    int x = 0, y = nseq;
    while (y - x > 1) {
      const int m = (x + y) >> 1;
      if (cs[m] / per + m <= grp) x = m; else y = m;
    }
    lo = cs[x];
    hi = cs[x + 1];
    gi = (int)(grp - (lo / per + x));
    kept = lo / (C * keep) + x;
  } else {
    const int groups = max(1, (T + per - 1) / per);
    lo = grp / groups * T;
    hi = lo + T;
    gi = (int)(grp % groups);
    kept = grp / groups * ((T + C * keep - 1) / (C * keep));
  }
  const int64_t t = lo + (int64_t)gi * per + wave * C + lane;
  const bool in = t < hi;
  double av = 0., bv = 0., ev = 0.;
  if (in) {
    for (int x = 0; x < na; ++x) {
      av += a[((size_t)x * H + h) * rows + t];
      bv += b[((size_t)x * H + h) * rows + t];
    }
    for (int x = 0; x < ne; ++x) ev += e[((size_t)x * H + h) * rows + t];
  }
  double pre = bv - av;  // inclusive prefix of b - a, suffix of e
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) {
    const double x = __shfl_up(pre, off), y = __shfl_down(ev, off);
    if (lane >= off) pre += x;
    if (lane + off < 64) ev += y;
  }
  if (lane == 63) chunk_sum[wave] = pre;
  __syncthreads();
  double D = 0.;
  if (in) {
    const int from = wave / keep * keep;  // the last chunk with an anchor
    const int64_t at = kept + (gi * kLinaGroup + from) / keep;
    for (int x = 0; x < 4 * na; ++x) D += anchor[((size_t)at * H + h) * 4 * na + x];
    for (int x = from; x < wave; ++x) D += chunk_sum[x];
  }
  double r = in ? ev + (pre - (bv - av)) + D : 0.;
  // e^g under 2^-126 is zero to the walks: such a token passes nothing on, and r is what rounding left of sums
  if (in && (g_fixed ? g[h] : g[(size_t)t * H + h]) * 1.4426950408889634 < -126.) r = 0.;
  if (dg) {
    if (in) dg[(size_t)t * H + h] = (float)r;
  } else {  // one decay for each head: the group's sum
    double s = r;
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) s += __shfl_xor(s, off);
    __syncthreads();
    if (lane == 0) chunk_sum[wave] = s;
    __syncthreads();
    if (threadIdx.x == 0) {
      s = 0.;
      for (int x = 0; x < kLinaGroup; ++x) s += chunk_sum[x];
      part[(size_t)h * gridDim.x + grp] = s;
    }
  }
}

__global__ __launch_bounds__(256) void lina_ddecay_sum_kernel(const double* __restrict__ part, int64_t groups,
                                                              float* __restrict__ dg) {
  __shared__ double s[256];
  double x = 0.;
  for (int64_t i = threadIdx.x; i < groups; i += 256) x += part[(size_t)blockIdx.x * groups + i];
  s[threadIdx.x] = x;
  for (int off = 128; off > 0; off >>= 1) {
    __syncthreads();
    if ((int)threadIdx.x < off) s[threadIdx.x] += s[threadIdx.x + off];
  }
  if (threadIdx.x == 0) dg[blockIdx.x] = (float)s[0];
}

}  // namespace

hipError_t launch_lina_segments(const LinaWalk* w, int n) {
  bool done[3] = {false, false, false};
  for (int i = 0; i < n; ++i) {
    if (done[i] || !w[i].split) continue;
    SegParams p;
    int m = 0;
    unsigned end = 0;
    for (int j = i; j < n; ++j)
      if (w[j].dk == w[i].dk) {
        p.p[m] = walk_params(w[j]);
        p.end[m] = end += walk_blocks(p.p[m]);
        ++m;
        done[j] = true;
      }
    for (; m < 3; ++m) {
      p.p[m] = p.p[0];
      p.end[m] = end;
    }
    const hipError_t e = w[i].bf16 ? (w[i].dk == 128 ? segments<bf16_t, 128>(p) : segments<bf16_t, 64>(p))
                                   : (w[i].dk == 128 ? segments<float, 128>(p) : segments<float, 64>(p));
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

hipError_t launch_lina_walk(const LinaWalk& w) {
  const WalkParams p = walk_params(w);
  if (w.bf16) return w.dk == 128 ? walk_bf16<128>(p) : walk_bf16<64>(p);
  return w.dk == 128 ? walk_f32<128>(p) : walk_f32<64>(p);
}

hipError_t launch_lina_pair(const LinaWalk& wq, const LinaWalk& wv) {
  PairParams p;
  p.q = walk_params(wq);
  p.v = walk_params(wv);
  p.blocks_q = walk_blocks(p.q);
  if (wq.dk == 128) return wv.dk == 128 ? pair_f32<128, 128>(p) : pair_f32<128, 64>(p);
  return wv.dk == 128 ? pair_f32<64, 128>(p) : pair_f32<64, 64>(p);
}

template <int D, bool WANT>
static hipError_t reverse(const RevParams& p) {
  return launch(lina_reverse_kernel<D, WANT>, p, walk_blocks(p.k), 3 * NT, RevLds<D>::BYTES, p.k.w.stream);
}

hipError_t launch_lina_reverse(const LinaWalk& wk, const LinaWalk& wv) {
  RevParams p;
  p.k = walk_params(wk);
  p.v = walk_params(wv);
  const bool want = wk.dot != kDotNone;
  if (wk.dk == 128) return want ? reverse<128, true>(p) : reverse<128, false>(p);
  return want ? reverse<64, true>(p) : reverse<64, false>(p);
}

hipError_t launch_lina_offsets(const int* cu, int n, int T, int L, int chains, int* cs, int* list, void* stream,
                               int cut, int link) {
  hipLaunchKernelGGL(lina_offsets_kernel, dim3(1), dim3(NTB), 0, (hipStream_t)stream, cu, n, T, L, chains, cut, link,
                     lina_pieces(T, n, L), cs, list);
  return hipGetLastError();
}

hipError_t launch_lina_headsum(const float* part, void* out, int64_t rows, int heads, int group, int d, bool bf16,
                               const int* end, void* stream) {
  const int64_t quads = rows * heads * (d / 4);
  if (quads == 0) return hipSuccess;
  const int64_t blocks = std::min<int64_t>((quads + 255) / 256, 1 << 20);
  if (bf16)
    hipLaunchKernelGGL(lina_headsum_kernel<bf16_t>, dim3((unsigned)blocks), dim3(256), 0, (hipStream_t)stream, part,
                       out, quads, heads, group, d / 4, end);
  else
    hipLaunchKernelGGL(lina_headsum_kernel<float>, dim3((unsigned)blocks), dim3(256), 0, (hipStream_t)stream, part,
                       out, quads, heads, group, d / 4, end);
  return hipGetLastError();
}

hipError_t launch_lina_ddecay(const LinaWalk& w, const float* a, const float* b, const float* e, int na, int ne,
                              const float* anchor, float* dg, double* part, float* dg_fixed) {
  const int64_t rows = w.cs ? w.T : (int64_t)w.n * w.T;
  const int64_t per = (int64_t)C * kLinaGroup;
  const int64_t groups = w.cs ? lina_pieces(w.T, w.n, kLinaGroup) : (int64_t)w.n * (((int64_t)w.T + per - 1) / per);
  if (rows > 0 && groups > 0) {
    hipLaunchKernelGGL(lina_ddecay_kernel, dim3((unsigned)groups, (unsigned)w.H), dim3(kLinaDecayThreads), 0,
                       (hipStream_t)w.stream, w.cs, w.n, w.T, w.H, rows, a, b, e, na, ne, anchor, lina_keep(w.bf16),
                       w.g, w.g_fixed, dg, part);
    const hipError_t er = hipGetLastError();
    if (er != hipSuccess) return er;
  }
  if (dg_fixed) {
    hipLaunchKernelGGL(lina_ddecay_sum_kernel, dim3((unsigned)w.H), dim3(256), 0, (hipStream_t)w.stream, part,
                       rows > 0 ? groups : (int64_t)0, dg_fixed);
    return hipGetLastError();
  }
  return hipSuccess;
}

}  // namespace kda
