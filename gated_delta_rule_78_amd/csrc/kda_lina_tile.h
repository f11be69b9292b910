// kda_lina_tile.h -- device pieces shared by the linear-attention walks: LDS tiles and their
// fragments, bounded chunk buffers, chunk decays, and the mapping of workgroups to chains.
#pragma once
#include "kda_common.h"
#include "kda_lina.h"
#include "kda_tile.h"

namespace kda {

namespace {

constexpr int VT = 64;  // value columns of a workgroup
constexpr int NT = 256;  // threads that hold a workgroup's state, and threads that fetch its tiles

typedef short v4s_t __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) v4s_t lds_v4s;

// LEAN: x, but not known to be the same each time, so that the addresses made from it stay out of
// the registers that live through a loop.  The kernel with three waves to a SIMD (168 registers)
// spilled without it; the one with two (256) is 3% faster with its addresses kept.
template <bool LEAN>
__device__ __forceinline__ uint32_t fresh(uint32_t x) {
#ifndef KDA_HOST_PASS
  if constexpr (LEAN) asm volatile("" : "+v"(x));
#endif
  return x;
}

// 64-row LDS tile of D elements a row, in quads of four elements.  Units of 16 bytes are
// permuted (exclusive or) by the row so that the three ways of reading it (16 rows at one quad,
// four plus four rows at one 16-column block by the transpose loads, 16 rows at two quads) touch
// all banks evenly: measured at the rate of a linear read.  The permutation depends on the row
// within 16 only, so every address is a lane's base, an exclusive or and a constant.  (Rows
// padded instead, with every address a base and a constant, cost more in conflicts than they
// saved: B4 H32 T8K forward 303 us against 294.)
template <typename T, int D>
struct Tile {
  static constexpr int DIM = D;
  static constexpr int RB = D * (int)sizeof(T);
  static constexpr int BYTES = C * RB;
  static constexpr int QB = 4 * (int)sizeof(T);
  __device__ __forceinline__ static int unit(int row, int u) {
    if constexpr (sizeof(T) == 4) return row * RB + (((u & ~15) | ((u ^ row) & 15)) << 4);
    else if constexpr (D == 128) return row * RB + ((u ^ (((row & 3) << 1) | (row & 8) | ((row >> 2) & 1))) << 4);
    else {
      const int y = row >> 1;
      return row * RB + ((u ^ (((y & 1) << 1) | (y & 4) | ((y >> 1) & 1))) << 4);
    }
  }
  __device__ __forceinline__ static int quad(int row, int q) {
    if constexpr (sizeof(T) == 4) return unit(row, q);
    else return unit(row, q >> 1) + ((q & 1) << 3);
  }
};

// A lane's bases in a tile, by what it reads.
template <typename T, int D, bool LEAN>
__device__ __forceinline__ uint32_t row_base(int lane) {  // row n, quad g
  return fresh<LEAN>(Tile<T, D>::quad(lane & 15, lane >> 4));
}
template <typename T, int D, bool LEAN>
__device__ __forceinline__ uint32_t tok_base(int lane) {  // bf16: row 8 g + n / 4, quad n % 4
  const int g = lane >> 4, n = lane & 15;
  return sizeof(T) == 2 ? fresh<LEAN>(Tile<T, D>::quad(8 * g + (n >> 2), n & 3)) : 0;
}

// A lane's base for the rows from r0 on (a multiple of 16).  Nothing is known of how two of them
// lie to each other: the compiler would make one ds_read2st64_b64 of two reads a constant apart,
// which takes 16 cycles where two ds_read_b64 take 5 (measured).
template <typename T, int D, bool LEAN>
__device__ __forceinline__ uint32_t rows_at(uint32_t base, int r0) {
  uint32_t x = base + r0 * Tile<T, D>::RB;
#ifndef KDA_HOST_PASS
  if constexpr (sizeof(T) == 2) {
    if constexpr (LEAN) asm volatile("" : "+v"(x));
    else asm("" : "+v"(x));
  }
#endif
  return x;
}

// row fragment of 32 columns: slots 0-3 columns 32 s + 4 g.., slots 4-7 columns 32 s + 16 + 4 g.. of
// row r0 + n, base = rows_at(.., r0): the order in which two 16-row accumulator tiles of the state
// hold their rows
template <typename T>
__device__ __forceinline__ void row_frag(Frag<T>& f, const char* t, uint32_t base, int s) {
  f.load4x2(t + (base ^ (s * 32 * sizeof(T))), t + (base ^ ((s * 32 + 16) * sizeof(T))));
}

// token fragment: slots hold tokens 32 s + 8 g + e of column c0 + n (c0 a multiple of 16)
template <typename T, int D>
__device__ __forceinline__ void tok_frag(Frag<T>& f, const char* t, uint32_t base, int c0, int s, int lane) {
  if constexpr (sizeof(T) == 2) {
#ifndef KDA_HOST_PASS
    // 16 lanes read four rows of 16 columns and get four rows of their own column; four rows
    // further the permutation differs in its lowest bit
    const char* p = t + 32 * s * Tile<T, D>::RB;
    const uint32_t o = base ^ (c0 * 2);
    const v4s_t a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s*)(p + o));
    const v4s_t b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s*)(p + (o ^ 16) + 4 * Tile<T, D>::RB));
    const uint2 x = __builtin_bit_cast(uint2, a), y = __builtin_bit_cast(uint2, b);
    f.w[0] = x.x; f.w[1] = x.y; f.w[2] = y.x; f.w[3] = y.y;
#endif
  } else {
    const int g = lane >> 4, c = c0 + (lane & 15);
#pragma unroll
    for (int e = 0; e < 8; ++e) f.w[e] = *(const float*)(t + Tile<T, D>::quad(32 * s + 8 * g + e, c >> 2) + (c & 3) * 4);
  }
}

// slots hold columns 32 s + 8 g + e of row r0 + n (r0 a multiple of 16) of a 64-column tile;
// base: row n, quad 2 g
template <typename T, bool LEAN>
__device__ __forceinline__ uint32_t col_base(int lane) {
  return fresh<LEAN>(Tile<T, 64>::quad(lane & 15, 2 * (lane >> 4)));
}
template <typename T>
__device__ __forceinline__ void col_frag(Frag<T>& f, const char* t, uint32_t base, int r0, int s) {
  const char* p = t + r0 * Tile<T, 64>::RB;
  const uint32_t o = base ^ (s * 32 * sizeof(T));
  if constexpr (sizeof(T) == 2) f.load8(p + o);
  else f.load4x2(p + o, p + (o ^ 16));
}

template <typename T>
__device__ __forceinline__ void st_quad(char* p, const float (&x)[4]);
template <>
__device__ __forceinline__ void st_quad<bf16_t>(char* p, const float (&x)[4]) {
  *(uint2*)p = make_uint2(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]));
}
template <>
__device__ __forceinline__ void st_quad<float>(char* p, const float (&x)[4]) {
  *(float4*)p = make_float4(x[0], x[1], x[2], x[3]);
}

template <typename T>
__device__ __forceinline__ void ld_quad(const void* p, size_t i, float (&x)[4]);
template <>
__device__ __forceinline__ void ld_quad<bf16_t>(const void* p, size_t i, float (&x)[4]) {
  const uint2 w = *(const uint2*)((const uint16_t*)p + i);
  x[0] = __uint_as_float(w.x << 16); x[1] = __uint_as_float(w.x & 0xFFFF0000u);
  x[2] = __uint_as_float(w.y << 16); x[3] = __uint_as_float(w.y & 0xFFFF0000u);
}
template <>
__device__ __forceinline__ void ld_quad<float>(const void* p, size_t i, float (&x)[4]) {
  const float4 w = *(const float4*)((const float*)p + i);
  x[0] = w.x; x[1] = w.y; x[2] = w.z; x[3] = w.w;
}

typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));

// One chunk's rows of an operand as a buffer of the rows that exist: what lies behind them
// reads as zeros and is not written, without a branch.
struct Rows {
#ifndef KDA_HOST_PASS
  __amdgpu_buffer_rsrc_t r;
  __device__ __forceinline__ Rows(const void* p, uint32_t bytes)
      : r(__builtin_amdgcn_make_buffer_rsrc((void*)p, 0, bytes, 0x00020000)) {}
  __device__ __forceinline__ u32x4_t load16(uint32_t off) const {
    return __builtin_bit_cast(u32x4_t, __builtin_amdgcn_raw_buffer_load_b128(r, off, 0, 0));
  }
  __device__ __forceinline__ u32x2_t load8(uint32_t off) const {
    return __builtin_bit_cast(u32x2_t, __builtin_amdgcn_raw_buffer_load_b64(r, off, 0, 0));
  }
  __device__ __forceinline__ void store16(uint32_t off, u32x4_t x) const {
    __builtin_amdgcn_raw_buffer_store_b128(x, r, off, 0, 0);
  }
  __device__ __forceinline__ void store8(uint32_t off, u32x2_t x) const {
    __builtin_amdgcn_raw_buffer_store_b64(x, r, off, 0, 0);
  }
#else
  __device__ Rows(const void*, uint32_t) {}
  __device__ u32x4_t load16(uint32_t) const { return u32x4_t{}; }
  __device__ u32x2_t load8(uint32_t) const { return u32x2_t{}; }
  __device__ void store16(uint32_t, u32x4_t) const {}
  __device__ void store8(uint32_t, u32x2_t) const {}
#endif
};

__device__ __forceinline__ float fast_exp2(float x) {  // results under 2^-126 are zero
#ifndef KDA_HOST_PASS
  return __builtin_amdgcn_exp2f(x);
#else
  return x;
#endif
}

__device__ __forceinline__ int64_t uniform64(int64_t x) {
#ifndef KDA_HOST_PASS
  const uint32_t a = __builtin_amdgcn_readfirstlane((uint32_t)x), b = __builtin_amdgcn_readfirstlane((uint32_t)(x >> 32));
  return (int64_t)(((uint64_t)b << 32) | a);
#else
  return x;
#endif
}

// Sums of four values over the 16 lanes of a DPP row: lane n gets that of value n % 4.  Two values
// share each step until one is left, then the row's quads are added: eleven operations for four.
__device__ __forceinline__ float row16_sums(const float (&v)[4], int n) {
#define KDA_DPP(x, ctrl) __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, x), ctrl, 0xF, 0xF, true))
  const bool odd = n & 1, up = n & 2;
  const float a0 = odd ? v[1] : v[0], b0 = odd ? v[0] : v[1];
  const float a1 = odd ? v[3] : v[2], b1 = odd ? v[2] : v[3];
  const float x = a0 + KDA_DPP(b0, 0xB1), y = a1 + KDA_DPP(b1, 0xB1);  // with lane n ^ 1
  const float a = up ? y : x, b = up ? x : y;
  float s = a + KDA_DPP(b, 0x4E);                                      // with lane n ^ 2
  s += KDA_DPP(s, 0x124);                                              // the row's quads, rotated
  s += KDA_DPP(s, 0x128);
#undef KDA_DPP
  return s;
}

// three bf16 terms: all 24 bits
__device__ __forceinline__ void split_triple(const float (&x)[8], Frag<bf16_t>& hi, Frag<bf16_t>& mid,
                                             Frag<bf16_t>& lo) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float a = x[2 * i], b = x[2 * i + 1];
    uint32_t h = pack_bf16x2(a, b);
    hi.w[i] = h;
    a -= __uint_as_float(h << 16);
    b -= __uint_as_float(h & 0xFFFF0000u);
    h = pack_bf16x2(a, b);
    mid.w[i] = h;
    lo.w[i] = pack_bf16x2(a - __uint_as_float(h << 16), b - __uint_as_float(h & 0xFFFF0000u));
  }
}

// e^x below this (in powers of two) is zero next to anything fp32 holds: steps are cut there,
// so that -inf (a reset) leaves the sums finite and 64 of them keep 1/8 exact in fp32
constexpr float kLeast = -512.f;

// Decays of one chunk in LDS.  The exponent of r_ij is (hi_i - hi_j) + (lo_i - lo_j): hi a
// multiple of 1/8, whose difference is exact, so a long or steep chunk costs no digits.
struct Decays {
  float hi[C], lo[C];  // log2 of the decay from the chunk's start to the token
  float row[C];        // 2^(hi + lo)
  float col[C];        // token to the chunk's end
  float tot;           // the whole chunk
  float pad[3];
};

// one wave: lane r holds the log decay of row r (natural logarithm, 0 for rows past the end);
// returns its running sum in powers of two, and the whole chunk's
__device__ __forceinline__ double decay_sums(float gr, int lane, double& tot) {
  const double x = (double)gr * 1.4426950408889634;
  double s = x < (double)kLeast ? (double)kLeast : x;  // NaN stays
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) {
    const double y = __shfl_up(s, off);
    if (lane >= off) s += y;
  }
  tot = __shfl(s, 63);
  return s;
}

__device__ __forceinline__ void chunk_decays(Decays& d, float gr, int lane) {
  double tot;
  const double s = decay_sums(gr, lane, tot);
  const float hi = rintf((float)s * 8.f) * 0.125f;
  d.hi[lane] = hi;
  d.lo[lane] = (float)(s - (double)hi);
  d.row[lane] = fast_exp2((float)s);
  d.col[lane] = fast_exp2((float)(tot - s));
  if (lane == 0) d.tot = fast_exp2((float)tot);
}

// What a state alone needs of them.
struct ColDecays {
  float col[C];
  float tot;
  float pad[3];
};

__device__ __forceinline__ void chunk_decays(ColDecays& d, float gr, int lane) {
  double tot;
  const double s = decay_sums(gr, lane, tot);
  d.col[lane] = fast_exp2((float)(tot - s));
  if (lane == 0) d.tot = fast_exp2((float)tot);
}

struct WalkParams {
  LinaWalk w;
  int nv;        // value tiles
  int64_t rows;  // tokens in all
  int64_t nseg;  // segment slots
  int64_t ends;  // end states
};

// A workgroup's place: its segment of a sequence, its head and its 64 value columns.
struct Chain {
  int64_t lo, hi;       // the sequence's tokens [lo, hi)
  int64_t base;         // its first end state
  int h, vt, sq;        // head, value tile, sequence
  int sg, nsg;          // segment of the sequence, its segments
  int nch;              // the sequence's chunks
  int first, last;      // the segment's chunks [first, last); replayed ones before it included
  int skip;             // replayed chunks
  bool head, tail;      // first and last of its sequence in walk order

  // Heads that share q and k, and the value tiles of a head, go to one XCD (workgroups are
  // dealt to the eight in turn), next to each other.  False: nothing to do here.
  __device__ __forceinline__ bool place(const WalkParams& p, bool rev, unsigned block) {
    const LinaWalk& w = p.w;
    const int L = (int)uniform64(w.cs ? w.cs[w.n + 1] : w.L);
    const int qk = w.q.heads < w.k.heads ? w.q.heads : w.k.heads;
    const int hk = qk < w.v.heads ? qk : w.v.heads;
    const int share = w.H / hk * p.nv;
    const int64_t slot = block >> 3;
    const int64_t unit = slot / share * 8 + (block & 7);
    const int in = (int)(slot % share);
    int64_t seg = unit / hk;
    if (seg >= p.nseg) return false;
    h = (int)(unit % hk) * (w.H / hk) + in / p.nv;
    vt = in % p.nv;
    if (w.cs) {
      sq = w.list[2 * seg];
      if (sq < 0) return false;
      sg = w.list[2 * seg + 1];
      lo = w.cs[sq];
      hi = w.cs[sq + 1];
      base = lo / ((int64_t)C * L);
    } else {
      const int64_t per = p.nseg / w.n;
      sq = (int)(seg / per);
      sg = (int)(seg % per);
      lo = (int64_t)sq * w.T;
      hi = lo + w.T;
      base = sq * (per - 1);
    }
    base = uniform64(base);  // scalar from here on: buffer descriptors are made from them
    lo = uniform64(lo);
    hi = uniform64(hi);
    sq = (int)uniform64(sq);
    sg = (int)uniform64(sg);
    nch = (int)((hi - lo + C - 1) / C);
    nsg = nch > 0 ? (nch + L - 1) / L : 1;
    if (sg >= nsg) return false;
    first = sg * L;
    last = min(nch, first + L);
    skip = w.replay ? first : 0;
    first -= skip;
    head = rev ? sg == nsg - 1 : sg == 0;
    tail = rev ? sg == 0 : sg == nsg - 1;
    return true;
  }
  // slot of this chain in [end states or kept states][H][value tiles]
  __device__ __forceinline__ size_t at(const WalkParams& p, int64_t piece) const {
    return ((size_t)piece * p.w.H + h) * p.nv + vt;
  }
  // end state of segment s, in walk order the next one's start: all but the last have one
  __device__ __forceinline__ int64_t end(bool rev, int s) const { return base + s - (rev ? 1 : 0); }
  // where a cut sequence's start state is kept, after the end states
  __device__ __forceinline__ int64_t start(const WalkParams& p) const { return p.ends + (p.ends < p.w.n ? base : sq); }
  // anchor at the start of chunk c, a multiple of lina_keep()
  __device__ __forceinline__ int64_t anchor(const WalkParams& p, int c) const {
    const int keep = lina_keep(p.w.bf16);
    return p.w.cs ? lo / (C * keep) + sq + c / keep : (int64_t)sq * ((nch + keep - 1) / keep) + c / keep;
  }
  // kept state there, c > 0: laid out as the end states are
  __device__ __forceinline__ int64_t kept(const WalkParams& p, int c) const {
    const int keep = lina_keep(p.w.bf16);
    return (p.w.cs ? lo / (C * keep) : (int64_t)sq * ((nch + keep - 1) / keep - 1)) + c / keep - 1;
  }
  __device__ __forceinline__ uint32_t rows(int c) const {  // tokens of chunk c
    return (uint32_t)min((int64_t)C, hi - lo - (int64_t)c * C);
  }
  __device__ __forceinline__ float decay_log(const LinaWalk& w, int64_t t) const {
    return w.g_fixed ? w.g[h] : w.g[(size_t)t * w.H + h];
  }
};

// An operand at a chain's head: bytes between tokens, and its rows from token t on.
template <typename T>
struct Operand {
  const char* p;
  uint32_t step;
  __device__ __forceinline__ Operand(const LinaOp& o, const LinaWalk& w, int h, int dim, int col) {
    step = o.heads * dim * (uint32_t)sizeof(T);
    p = (const char*)o.p + ((size_t)(o.heads ? h / (w.H / o.heads) : 0) * dim + col) * sizeof(T);
  }
  __device__ __forceinline__ Rows rows(int64_t t, uint32_t have) const { return Rows(p + (size_t)t * step, have * step); }
};

// fn(ct, i, element) over a thread's state entries: row 16 ct + 4 g + i, column 16 wave + n
template <int DK, typename F>
__device__ __forceinline__ void each_state(const LinaWalk& w, const Chain& ch, int wave, int lane, F fn) {
  const int g = lane >> 4, vc = ch.vt * VT + 16 * wave + (lane & 15);
  const size_t b0 = ((size_t)ch.sq * w.H + ch.h) * (size_t)DK * w.dv;
#pragma unroll
  for (int ct = 0; ct < DK / 16; ++ct)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int kc = 16 * ct + 4 * g + i;
      fn(ct, i, b0 + (w.s_t ? (size_t)vc * DK + kc : (size_t)kc * w.dv + vc));
    }
}

// The state a walk starts from: the caller's, carried over the segments before this one.  Of a chain
// in several segments it comes from a copy (keep_start), because the last one may write
// its final state over the caller's while others have not begun.
template <int DK>
__device__ __forceinline__ void start_state(const WalkParams& p, const Chain& ch, bool rev, int tid,
                                            f32x4_t (&S)[DK / 16]) {
  const LinaWalk& w = p.w;
  const bool kept = w.split && ch.nsg > 1;
#pragma unroll
  for (int ct = 0; ct < DK / 16; ++ct) S[ct] = zero4();
  if (w.s0) {
    if (kept) {
      const f32x4_t* from = (const f32x4_t*)(w.seg_state + ch.at(p, ch.start(p)) * (DK * VT));
#pragma unroll
      for (int ct = 0; ct < DK / 16; ++ct) S[ct] = from[ct * NT + tid];
    } else {
      each_state<DK>(w, ch, tid >> 6, tid & 63, [&](int ct, int i, size_t at) { S[ct][i] = w.s0[at]; });
    }
  }
  if (!w.split || ch.head) return;
  const int cnt = rev ? ch.nsg - 1 - ch.sg : ch.sg;
#pragma unroll 2
  for (int j = 0; j < cnt; ++j) {
    const int64_t s = ch.end(rev, rev ? ch.nsg - 1 - j : j);
    const float d = w.seg_dec[(size_t)s * w.H + ch.h];
    const f32x4_t* B = (const f32x4_t*)(w.seg_state + ch.at(p, s) * (DK * VT));
#pragma unroll
    for (int ct = 0; ct < DK / 16; ++ct) {
      const f32x4_t x = B[ct * NT + tid];
#pragma unroll
      for (int i = 0; i < 4; ++i) S[ct][i] = fmaf(S[ct][i], d, x[i]);
    }
  }
}

// The caller's start state of a chain in several segments, copied by its last one, from whose end nobody starts.
template <int DK>
__device__ __forceinline__ void keep_start(const WalkParams& p, const Chain& ch, int tid) {
  const LinaWalk& w = p.w;
  if (!w.s0 || ch.nsg == 1) return;
  f32x4_t* to = (f32x4_t*)(w.seg_state + ch.at(p, ch.start(p)) * (DK * VT));
  f32x4_t S[DK / 16];
  each_state<DK>(w, ch, tid >> 6, tid & 63, [&](int ct, int i, size_t at) { S[ct][i] = w.s0[at]; });
#pragma unroll
  for (int ct = 0; ct < DK / 16; ++ct) to[ct * NT + tid] = S[ct];
}

// The caller's final state; a reverse walk's state is the gradient after the first token's decay.
template <int DK, bool REV>
__device__ __forceinline__ void store_state(const WalkParams& p, const Chain& ch, int tid,
                                            const f32x4_t (&S)[DK / 16]) {
  const LinaWalk& w = p.w;
  if (!w.sT || !ch.tail) return;
  const float d = REV && ch.nch > 0 ? expf(ch.decay_log(w, ch.lo)) : 1.f;
  each_state<DK>(w, ch, tid >> 6, tid & 63, [&](int ct, int i, size_t at) { w.sT[at] = S[ct][i] * d; });
}

// byte offset of row r (rows counted from the end in a reverse walk), and of `rows` rows
__device__ __forceinline__ uint32_t row_off(bool rev, int r, uint32_t step) { return (rev ? C - 1 - r : r) * step; }
__device__ __forceinline__ uint32_t rows_off(bool rev, int rows, uint32_t step) { return (rev ? -rows : rows) * step; }

// A thread's share of one chunk's tiles, on its way from memory to LDS (NT threads).
template <typename T, int D, bool LEAN = false, typename TILE = Tile<T, D>>
struct Stage {
  static constexpr int RU = TILE::RB / 16;  // 16-byte units of a row
  static constexpr int N = C * RU / NT;
  static constexpr int ROWS = NT / RU;            // rows at a time, a multiple of 16 for bf16
  u32x4_t r[N];
  __device__ __forceinline__ void load(const Rows& b, uint32_t step, bool rev, int tid) {
    const uint32_t o = fresh<LEAN>(row_off(rev, tid / RU, step) + tid % RU * 16);
#pragma unroll
    for (int i = 0; i < N; ++i) r[i] = b.load16(o + rows_off(rev, ROWS * i, step));
  }
  __device__ __forceinline__ void store(char* t, int tid) const {
    const uint32_t o = fresh<LEAN>(TILE::unit(tid / RU, tid % RU));
#pragma unroll
    for (int i = 0; i < N; ++i)
      *(u32x4_t*)(t + (ROWS % 16 == 0 ? o + ROWS * i * TILE::RB
                                      : TILE::unit(tid / RU + ROWS * i, tid % RU))) = r[i];
  }
};

// P = r o (Q K^T) of one chunk: wave w makes rows 16 w .. as the transposed tiles K Q^T.
// kDotCross: also the sums over rows (cols[j]) and over columns (own[i]) of r o (Q K^T) o (X V^T)
// off the diagonal.
template <typename T, int DK, int DOT>
__device__ __forceinline__ void make_p(const char* sQ, const char* sK, const char* sV, const char* sX, char* sP,
                                       const Decays& dc, float* cols, float* own, int wave, int lane) {
  constexpr int KS = DK / 32;
  const int g = lane >> 4, n = lane & 15, row = 16 * wave + n;
  Frag<T> fq[KS], fx[DOT == kDotCross ? 2 : 1];
  const uint32_t rb = row_base<T, DK, false>(lane), vb = row_base<T, VT, false>(lane);
#pragma unroll
  for (int s = 0; s < KS; ++s) row_frag<T>(fq[s], sQ, rows_at<T, DK, false>(rb, 16 * wave), s);
  if constexpr (DOT == kDotCross) {
    row_frag<T>(fx[0], sX, rows_at<T, VT, false>(vb, 16 * wave), 0);
    row_frag<T>(fx[1], sX, rows_at<T, VT, false>(vb, 16 * wave), 1);
  }
  const float ih = dc.hi[row], il = dc.lo[row];
  float own_sum = 0.f;
#pragma unroll
  for (int J = 0; J < 4; ++J) {
    float x[4] = {0.f, 0.f, 0.f, 0.f};
    if (J <= wave) {
      f32x4_t a = zero4(), e = zero4();
#pragma unroll
      for (int s = 0; s < KS; ++s) {
        Frag<T> fk;
        row_frag<T>(fk, sK, rows_at<T, DK, false>(rb, 16 * J), s);
        mma(a, fk, fq[s]);
      }
      if constexpr (DOT == kDotCross) {
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          Frag<T> fv;
          row_frag<T>(fv, sV, rows_at<T, VT, false>(vb, 16 * J), s);
          mma(e, fv, fx[s]);
        }
      }
      const float4 jh = *(const float4*)&dc.hi[16 * J + 4 * g], jl = *(const float4*)&dc.lo[16 * J + 4 * g];
      const float jhs[4] = {jh.x, jh.y, jh.z, jh.w}, jls[4] = {jl.x, jl.y, jl.z, jl.w};
      float m[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int j = 16 * J + 4 * g + i;
        const float r = a[i] * fast_exp2((ih - jhs[i]) + (il - jls[i]));
        x[i] = j <= row ? r : 0.f;
        if constexpr (DOT == kDotCross) {
          m[i] = j < row ? r * e[i] : 0.f;
          own_sum += m[i];
        }
      }
      if constexpr (DOT == kDotCross) {
        const float cs = row16_sums(m, n);
        if (n < 4) cols[16 * J + 4 * g + n] = cs;
      }
    }
    if (J <= (wave | 1)) st_quad<T>(sP + 16 * wave * Tile<T, 64>::RB + (vb ^ (J * 16 * sizeof(T))), x);
  }
  if constexpr (DOT == kDotCross) {
    own_sum += __shfl_xor(own_sum, 16);
    own_sum += __shfl_xor(own_sum, 32);
    if (g == 0) own[row] = own_sum;
  }
}

// The start state's part of the outputs, before the decay to the token: rows of S^T against rows
// of Q.  acc[t] holds columns 4 g + i of token 16 t + n.  EXACT: the state in three bf16 terms.
template <typename T, int DK, bool EXACT, bool LEAN = false>
__device__ __forceinline__ void from_state(const f32x4_t (&S)[DK / 16], const char* sQ, int lane, f32x4_t (&acc)[4]) {
  const uint32_t rb = row_base<T, DK, LEAN>(lane);
  uint32_t rt[4];
#pragma unroll
  for (int t = 0; t < 4; ++t) {
    rt[t] = rows_at<T, DK, LEAN>(rb, 16 * t);
    acc[t] = zero4();
  }
#pragma unroll
  for (int s = 0; s < DK / 32; ++s) {
    Frag<T> fs, fm, fl;
    if constexpr (sizeof(T) == 2 && EXACT) {
      const float x[8] = {S[2 * s][0],     S[2 * s][1],     S[2 * s][2],     S[2 * s][3],
                          S[2 * s + 1][0], S[2 * s + 1][1], S[2 * s + 1][2], S[2 * s + 1][3]};
      split_triple(x, fs, fm, fl);
    } else {
      fs.from_acc(S[2 * s], S[2 * s + 1]);
    }
#pragma unroll
    for (int t2 = 0; t2 < 4; t2 += 2) {
      Frag<T> fq[2];
#pragma unroll
      for (int x = 0; x < 2; ++x) row_frag<T>(fq[x], sQ, rt[t2 + x], s);
#pragma unroll
      for (int x = 0; x < 2; ++x) mma(acc[t2 + x], fs, fq[x]);
      if constexpr (sizeof(T) == 2 && EXACT) {
#pragma unroll
        for (int x = 0; x < 2; ++x) mma(acc[t2 + x], fm, fq[x]);
#pragma unroll
        for (int x = 0; x < 2; ++x) mma(acc[t2 + x], fl, fq[x]);
      }
    }
  }
}

// acc (the start state's part) += P V for 16 columns from c0 on of a V tile VD wide; fv: V along
// the tokens
template <typename T, int VD, bool LEAN = false>
__device__ __forceinline__ void add_intra(f32x4_t (&acc)[4], const Frag<T> (&fv)[2], const char* sP, const char* sV,
                                          int c0, int lane) {
  const int g = lane >> 4, n = lane & 15;
  const uint32_t cb = col_base<T, LEAN>(lane);
  f32x4_t a[4];
#pragma unroll
  for (int t = 0; t < 4; ++t) {
    a[t] = acc[t];
#pragma unroll
    for (int s = 0; s <= t / 2; ++s) {
      Frag<T> fp;
      col_frag<T>(fp, sP, cb, 16 * t, s);
      mma(a[t], fv[s], fp);
    }
  }
  // A value row that is not finite spoils (0 times it) the tokens before it in its tile; the
  // last tile sees every row.  Rare: the chunk is then summed token by token.
  bool bad = false;
#pragma unroll
  for (int i = 0; i < 4; ++i) bad |= !(fabsf(a[3][i]) < __builtin_inff());
  if (__builtin_expect(__any(bad), 0)) {
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      a[t] = acc[t];
      for (int j = 0; j <= 16 * t + n; ++j) {
        const float pj = Elem<T>::load(sP + Tile<T, 64>::quad(16 * t + n, j >> 2), j & 3);
        float x[4];
        ld_quad<T>(sV + Tile<T, VD>::quad(j, c0 / 4 + g), 0, x);
#pragma unroll
        for (int i = 0; i < 4; ++i) a[t][i] = fmaf(pj, x[i], a[t][i]);
      }
    }
  }
#pragma unroll
  for (int t = 0; t < 4; ++t) acc[t] = a[t];
}

// S <- decay S + K^T (col o V), the weighted values in three bf16 terms
template <typename T, int DK, bool LEAN = false, typename DEC>
__device__ __forceinline__ void add_chunk(f32x4_t (&S)[DK / 16], const Frag<T> (&fv)[2], const char* sK,
                                          const DEC& dc, int lane) {
  const int g = lane >> 4;
  const uint32_t tb = tok_base<T, DK, LEAN>(lane);
  const float tot = dc.tot;
#pragma unroll
  for (int ct = 0; ct < DK / 16; ++ct)
#pragma unroll
    for (int i = 0; i < 4; ++i) S[ct][i] *= tot;
#pragma unroll
  for (int s = 0; s < 2; ++s) {
    const float4 c0 = *(const float4*)&dc.col[32 * s + 8 * g], c1 = *(const float4*)&dc.col[32 * s + 8 * g + 4];
    const float cw[8] = {c0.x, c0.y, c0.z, c0.w, c1.x, c1.y, c1.z, c1.w};
    float x[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = fv[s].get(e) * cw[e];
    Frag<T> fh, fm, fl;
    if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int e = 0; e < 8; ++e) fh.w[e] = x[e];
    } else {
      split_triple(x, fh, fm, fl);
    }
#pragma unroll
    for (int c2 = 0; c2 < DK / 16; c2 += 2) {  // two tiles in turn: a product waits for the last on its tile
      Frag<T> fk[2];
#pragma unroll
      for (int x = 0; x < 2; ++x) tok_frag<T, DK>(fk[x], sK, tb, 16 * (c2 + x), s, lane);
#pragma unroll
      for (int x = 0; x < 2; ++x) mma(S[c2 + x], fk[x], fh);
      if constexpr (sizeof(T) == 2) {
#pragma unroll
        for (int x = 0; x < 2; ++x) mma(S[c2 + x], fk[x], fm);
#pragma unroll
        for (int x = 0; x < 2; ++x) mma(S[c2 + x], fk[x], fl);
      }
    }
  }
}

// acc to the outputs of chunk c
template <typename T, bool REV, bool LEAN = false>
__device__ __forceinline__ void store_out(const f32x4_t (&acc)[4], const LinaWalk& w, const Chain& ch, int c, int wave,
                                          int lane) {
  const int g = lane >> 4, n = lane & 15;
  const int64_t t0 = ch.lo + (int64_t)c * C;
  const uint32_t ro = w.H * w.dv, have = ch.rows(c);
  const size_t at = ((size_t)t0 * w.H + ch.h) * w.dv + ch.vt * VT;
  const uint32_t o = fresh<LEAN>(row_off(REV, n, ro) + 16 * wave + 4 * g);
  auto off = [&](int t) { return o + rows_off(REV, 16 * t, ro); };
  if (sizeof(T) == 2 && !w.out_f32) {
    const Rows b((char*)w.out + at * 2, have * ro * 2);
#pragma unroll
    for (int t = 0; t < 4; ++t)
      b.store8(off(t) * 2, u32x2_t{pack_bf16x2(acc[t][0], acc[t][1]), pack_bf16x2(acc[t][2], acc[t][3])});
  } else {
    const Rows b((char*)w.out + at * 4, have * ro * 4);
#pragma unroll
    for (int t = 0; t < 4; ++t) b.store16(off(t) * 4, __builtin_bit_cast(u32x4_t, acc[t]));
  }
}

// kDotRow: a wave's columns of X for its four tokens tiles, loaded a chunk ahead
template <typename T>
struct DotRows {
  u32x4_t r[4];
  __device__ __forceinline__ void load(const Rows& b, uint32_t step, bool rev, int wave, int lane) {
    const uint32_t o = (row_off(rev, lane & 15, step) + (16 * wave + 4 * (lane >> 4)) * (uint32_t)sizeof(T));
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      const uint32_t off = o + rows_off(rev, 16 * t, step);
      if constexpr (sizeof(T) == 2) {
        const u32x2_t x = b.load8(off);
        r[t][0] = x[0];
        r[t][1] = x[1];
      } else {
        r[t] = b.load16(off);
      }
    }
  }
  __device__ __forceinline__ float get(int t, int i) const {
    if constexpr (sizeof(T) == 4) return __uint_as_float(r[t][i]);
    else return __uint_as_float(i & 1 ? r[t][i >> 1] & 0xFFFF0000u : r[t][i >> 1] << 16);
  }
  // x . acc of each token over the wave's columns -> sums[token]
  __device__ __forceinline__ void dot(const f32x4_t (&acc)[4], float* sums, int lane) const {
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      float d = 0.f;
#pragma unroll
      for (int i = 0; i < 4; ++i) d = fmaf(acc[t][i], get(t, i), d);
      d += __shfl_xor(d, 16);
      d += __shfl_xor(d, 32);
      if (lane < 16) sums[16 * t + lane] = d;
    }
  }
};

// <kept state, S> of a wave at the first token of chunk c, with that token's decay
template <int DK>
__device__ __forceinline__ void store_anchor(const WalkParams& p, const Chain& ch, int c, int tid,
                                             const f32x4_t (&S)[DK / 16]) {
  const LinaWalk& w = p.w;
  const f32x4_t* from = (const f32x4_t*)(w.snap + ch.at(p, ch.kept(p, c)) * (DK * VT)) + tid;
  int step = NT;
  if (c == 0) {  // the caller's, its rows this walk's columns (s_t): row 16 ct + 4 g of column 16 wave + n
    const int lane = tid & 63, vc = ch.vt * VT + 16 * (tid >> 6) + (lane & 15);
    from = (const f32x4_t*)(w.snap0 + (((size_t)ch.sq * w.H + ch.h) * w.dv + vc) * DK) + (lane >> 4);
    step = 4;
  }
  float d = 0.f;
  if (c > 0 || w.snap0) {
#pragma unroll
    for (int ct = 0; ct < DK / 16; ++ct) {
      const f32x4_t x = from[ct * step];
#pragma unroll
      for (int i = 0; i < 4; ++i) d = fmaf(x[i], S[ct][i], d);
    }
  }
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) d += __shfl_xor(d, off);
  if ((tid & 63) == 0) w.anchor[ch.at(p, ch.anchor(p, c)) * 4 + (tid >> 6)] = expf(ch.decay_log(w, ch.lo + (int64_t)c * C)) * d;
}

template <int DK>
__device__ __forceinline__ void store_snap(const WalkParams& p, const Chain& ch, int c, int tid,
                                           const f32x4_t (&S)[DK / 16]) {
  f32x4_t* to = (f32x4_t*)(p.w.snap + ch.at(p, ch.kept(p, c)) * (DK * VT));
#pragma unroll
  for (int ct = 0; ct < DK / 16; ++ct) to[ct * NT + tid] = S[ct];
}

// log decay of row `lane` of chunk c (0 behind the sequence); a reverse step decays by the
// token after it
template <bool REV>
__device__ __forceinline__ float row_decay(const LinaWalk& w, const Chain& ch, int c, int lane) {
  if (c < ch.first || c >= ch.last) return 0.f;
  const int64_t t = ch.lo + (int64_t)c * C + (REV ? C - lane : lane);
  return t < ch.hi ? ch.decay_log(w, t) : 0.f;
}

__device__ __forceinline__ void scale_rows(f32x4_t (&acc)[4], const Decays& dc, int lane) {
#pragma unroll
  for (int t = 0; t < 4; ++t) {
    const float r = dc.row[16 * t + (lane & 15)];
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[t][i] *= r;
  }
}

// one wave: the chunk's per-token dots, from the four waves' parts
template <int DOT, bool REV>
__device__ __forceinline__ void store_dots(const WalkParams& p, const Chain& ch, int c, const float (&s)[4][C],
                                           const float* own, int lane) {
  float d;
  if constexpr (DOT == kDotRow) {
    d = (s[0][lane] + s[1][lane]) + (s[2][lane] + s[3][lane]);
  } else {
    d = -own[lane];
    for (int x = lane >> 4; x < 4; ++x) d += s[x][lane];
  }
  const int64_t t = ch.lo + (int64_t)c * C + (REV ? C - 1 - lane : lane);
  if (t < ch.hi) p.w.dots[((size_t)ch.vt * p.w.H + ch.h) * p.rows + t] = d;
}

inline unsigned walk_blocks(const WalkParams& p) {
  const LinaWalk& w = p.w;
  const int qk = w.q.heads < w.k.heads ? w.q.heads : w.k.heads;
  const int hk = qk < w.v.heads ? qk : w.v.heads;
  const int64_t blocks = (p.nseg * hk + 7) / 8 * (w.H / hk * p.nv) * 8;
  return blocks > 0x7FFFFFFF ? 0u : (unsigned)blocks;
}

}  // namespace

}  // namespace kda
