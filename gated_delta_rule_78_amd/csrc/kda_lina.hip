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
//   kLinaGroup chunks it is taken afresh from the two states, so that no rounding error
//   travels further than that.
//
// One workgroup of four waves walks one chain (sequence or segment, head, 64 value columns);
// wave w keeps columns 16 w .. 16 w + 15 of the state in fp32 accumulators, which serve as
// matrix-core operands without leaving the registers.  Products run transposed (rows are
// value columns, columns are tokens), so that a lane holds four neighbouring columns of one
// token and stores them at once; K and V are read along the token axis with the LDS
// transpose loads.
//
// Precision (bf16 inputs): sums, decays and the state are fp32.  Rounded to bf16 (2^-9
// relative, as the output itself is) are P = r o QK^T and the state where it is multiplied
// by q.  What enters the fp32 state, e^{G_C - G_j} v_j, goes through the matrix cores as a
// bf16 pair (value and residual, 2^-18), and so does the state where a, b are taken from it.
#include "kda_common.h"
#include "kda_lina.h"
#include "kda_tile.h"

namespace kda {

namespace {

constexpr int VT = 64;  // value columns of a workgroup
constexpr int NT = 256;

typedef short v4s_t __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) v4s_t lds_v4s;

// 64-row LDS tile of D elements a row, in quads of four elements.  Units of 16 bytes are
// permuted by the row so that the three ways of reading it (16 rows at one quad, four plus
// four rows at one 16-column block by the transpose loads, 16 rows at two quads) touch all
// banks evenly.
template <typename T, int D>
struct Tile {
  static constexpr int RB = D * (int)sizeof(T);
  static constexpr int BYTES = C * RB;
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

// row fragment of 32 channels: slots 0-3 channels 32 s + 4 g.., slots 4-7 channels 32 s + 16 + 4 g..
// of row `row`: the order in which two 16-row accumulator tiles of the state hold their rows
template <typename T, int D>
__device__ __forceinline__ void row_frag(Frag<T>& f, const char* t, int row, int s, int g) {
  f.load4x2(t + Tile<T, D>::quad(row, 8 * s + g), t + Tile<T, D>::quad(row, 8 * s + 4 + g));
}

// token fragment: slots hold tokens 32 s + 8 g + e of column c0 + n
template <typename T, int D>
__device__ __forceinline__ void tok_frag(Frag<T>& f, const char* t, int c0, int s, int lane) {
  const int g = lane >> 4, n = lane & 15;
  if constexpr (sizeof(T) == 2) {
#ifndef KDA_HOST_PASS
    // 16 lanes read four rows of 16 columns and get four rows of their own column
    const int q = c0 / 4 + (n & 3), r = 32 * s + 8 * g + (n >> 2);
    const v4s_t a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s*)(t + Tile<T, D>::quad(r, q)));
    const v4s_t b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s*)(t + Tile<T, D>::quad(r + 4, q)));
    const uint2 x = __builtin_bit_cast(uint2, a), y = __builtin_bit_cast(uint2, b);
    f.w[0] = x.x; f.w[1] = x.y; f.w[2] = y.x; f.w[3] = y.y;
#endif
  } else {
    const int c = c0 + n;
#pragma unroll
    for (int e = 0; e < 8; ++e) f.w[e] = *(const float*)(t + Tile<T, D>::quad(32 * s + 8 * g + e, c >> 2) + (c & 3) * 4);
  }
}

// slots hold columns 32 s + 8 g + e of row `row`
template <typename T>
__device__ __forceinline__ void col_frag(Frag<T>& f, const char* t, int row, int s, int g) {
  f.load4x2(t + Tile<T, 64>::quad(row, 8 * s + 2 * g), t + Tile<T, 64>::quad(row, 8 * s + 2 * g + 1));
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

// sum over the 16 lanes of a DPP row, in every lane
__device__ __forceinline__ float row16_sum(float x) {
#define KDA_ROR(n) x += __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, x), 0x120 + n, 0xF, 0xF, true))
  KDA_ROR(8);
  KDA_ROR(4);
  KDA_ROR(2);
  KDA_ROR(1);
#undef KDA_ROR
  return x;
}

// hi and residual of eight values as bf16 fragments
__device__ __forceinline__ void split_pair(const float (&x)[8], Frag<bf16_t>& hi, Frag<bf16_t>& lo) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float a = x[2 * i], b = x[2 * i + 1];
    const uint32_t h = pack_bf16x2(a, b);
    hi.w[i] = h;
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

// one wave: lane r holds the log decay of row r (natural logarithm, 0 for rows past the end)
__device__ __forceinline__ void chunk_decays(Decays& d, float gr, int lane) {
  const double x = (double)gr * 1.4426950408889634;
  double s = x < (double)kLeast ? (double)kLeast : x;  // NaN stays
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) {
    const double y = __shfl_up(s, off);
    if (lane >= off) s += y;
  }
  const double tot = __shfl(s, 63);
  const float hi = rintf((float)s * 8.f) * 0.125f;
  d.hi[lane] = hi;
  d.lo[lane] = (float)(s - (double)hi);
  d.row[lane] = fast_exp2((float)s);
  d.col[lane] = fast_exp2((float)(tot - s));
  if (lane == 0) d.tot = fast_exp2((float)tot);
}

struct WalkParams {
  LinaWalk w;
  int nv;        // value tiles
  int64_t rows;  // tokens in all
  int64_t nseg;  // segment slots
};

// STATE_ONLY: end states of the segments from a zero start, nothing else
template <typename T, int DK, bool REV, int DOT, bool STATE_ONLY>
__global__ __launch_bounds__(NT, sizeof(T) == 2 && (DOT == kDotNone || DK == 64) ? 2 : 1) void lina_walk_kernel(const WalkParams p) {
  constexpr int KS = DK / 32;   // product steps over the channels
  constexpr int CT = DK / 16;   // state tiles of a wave
  constexpr int QU = C * DK * (int)sizeof(T) / 16 / NT;  // 16-byte units a thread stages of Q or K
  constexpr int VU = C * VT * (int)sizeof(T) / 16 / NT;  // of V or X
  typedef Tile<T, DK> KT;
  typedef Tile<T, VT> VTl;
  typedef Tile<T, 64> PT;
  extern __shared__ __align__(16) char smem[];
  char* sK = smem;
  char* sV = sK + KT::BYTES;
  char* sQ = sV + VTl::BYTES;
  char* sP = sQ + KT::BYTES;
  char* sX = sP + PT::BYTES;  // kDotCross only
  __shared__ Decays dec[2];
  __shared__ float sdot[4][C];
  __shared__ float sdot2[C];

  const LinaWalk& w = p.w;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, g = lane >> 4, n = lane & 15;

  // block -> (segment, head, value tile): heads that share q and k and the value tiles of a
  // head go to one XCD (workgroups are dealt to the eight in turn), next to each other
  int64_t seg;
  int h, vt;
  {
    const int qk = w.q.heads < w.k.heads ? w.q.heads : w.k.heads;
    const int hk = qk < w.v.heads ? qk : w.v.heads;
    const int share = w.H / hk * p.nv;
    const int64_t slot = blockIdx.x >> 3;
    const int64_t unit = slot / share * 8 + (blockIdx.x & 7);
    const int in = (int)(slot % share);
    seg = unit / hk;
    if (seg >= p.nseg) return;
    h = (int)(unit % hk) * (w.H / hk) + in / p.nv;
    vt = in % p.nv;
  }
  // the segment's sequence and tokens
  int64_t lo, hi;
  int sq, sg;
  if (w.cs) {
    const int64_t per = (int64_t)C * w.L;
    int a = 0, b = w.n;  // the last sequence whose first segment is <= seg
    while (b - a > 1) {
      const int m = (a + b) >> 1;
      if (w.cs[m] / per + m <= seg) a = m; else b = m;
    }
    sq = a;
    sg = (int)(seg - (w.cs[a] / per + a));
    lo = w.cs[a];
    hi = w.cs[a + 1];
  } else {
    const int64_t per = p.nseg / w.n;
    sq = (int)(seg / per);
    sg = (int)(seg % per);
    lo = (int64_t)sq * w.T;
    hi = lo + w.T;
  }
  lo = uniform64(lo);
  hi = uniform64(hi);
  const int nch = (int)((hi - lo + C - 1) / C);
  const int nsg = nch > 0 ? (nch + w.L - 1) / w.L : 1;
  if (sg >= nsg) return;
  const int first = sg * w.L, last = min(nch, first + w.L);  // chunks [first, last)
  const bool head_seg = REV ? sg == nsg - 1 : sg == 0;       // the walk's first segment of its sequence
  const bool tail_seg = REV ? sg == 0 : sg == nsg - 1;
  if (STATE_ONLY && tail_seg) return;                        // nobody starts from its end

  const size_t seg_stride = (size_t)w.H * p.nv;
  auto seg_at = [&](int64_t s) { return w.seg_state + ((size_t)s * seg_stride + (size_t)h * p.nv + vt) * (DK * VT); };

  // operands: [rows, heads, dim], at this head
  auto base = [&](const LinaOp& o, int dim) {
    return (const char*)o.p + (size_t)(h / (w.H / o.heads)) * dim * sizeof(T);
  };
  const char* gq = STATE_ONLY ? nullptr : base(w.q, DK);
  const char* gk = base(w.k, DK);
  const char* gv = base(w.v, w.dv) + (size_t)vt * VT * sizeof(T);
  const char* gx = DOT != kDotNone ? base(w.x, w.dv) + (size_t)vt * VT * sizeof(T) : nullptr;
  const uint32_t rq = w.q.heads * DK * (uint32_t)sizeof(T), rk = w.k.heads * DK * (uint32_t)sizeof(T);
  const uint32_t ro = w.H * w.dv;  // elements between two tokens of the output
  const uint32_t rv = w.v.heads * w.dv * (uint32_t)sizeof(T), rx = w.x.heads * w.dv * (uint32_t)sizeof(T);

  // token of row r of chunk c (reverse walks count rows from the chunk's last token)
  auto token = [&](int c, int r) { return lo + (int64_t)c * C + (REV ? C - 1 - r : r); };

  // tiles of the next chunk in registers; off*: a thread's bytes from the chunk's first token
  u32x4_t rgq[STATE_ONLY ? 1 : QU], rgk[QU], rgv[VU], rgx[DOT == kDotCross ? VU : 1];
  u32x4_t rgd[DOT == kDotRow ? 4 : 1];  // kDotRow: four columns of X for each token tile (bf16: in .xy)
  auto tile_row = [&](int r) { return (uint32_t)(REV ? C - 1 - r : r); };
  auto prefetch = [&](int c) {
    const int64_t t0 = lo + (int64_t)c * C;
    const uint32_t have = (uint32_t)min((int64_t)C, hi - t0);
    const Rows bk(gk + (size_t)t0 * rk, have * rk), bv(gv + (size_t)t0 * rv, have * rv);
#pragma unroll
    for (int i = 0; i < QU; ++i) {
      const int u = tid + NT * i;
      rgk[i] = bk.load16(tile_row(u / (KT::RB / 16)) * rk + u % (KT::RB / 16) * 16);
    }
#pragma unroll
    for (int i = 0; i < VU; ++i) {
      const int u = tid + NT * i;
      rgv[i] = bv.load16(tile_row(u / (VTl::RB / 16)) * rv + u % (VTl::RB / 16) * 16);
    }
    if constexpr (!STATE_ONLY) {
      const Rows bq(gq + (size_t)t0 * rq, have * rq);
#pragma unroll
      for (int i = 0; i < QU; ++i) {
        const int u = tid + NT * i;
        rgq[i] = bq.load16(tile_row(u / (KT::RB / 16)) * rq + u % (KT::RB / 16) * 16);
      }
    }
    if constexpr (DOT == kDotCross && !STATE_ONLY) {
      const Rows bx(gx + (size_t)t0 * rx, have * rx);
#pragma unroll
      for (int i = 0; i < VU; ++i) {
        const int u = tid + NT * i;
        rgx[i] = bx.load16(tile_row(u / (VTl::RB / 16)) * rx + u % (VTl::RB / 16) * 16);
      }
    }
    if constexpr (DOT == kDotRow && !STATE_ONLY) {
      const Rows bx(gx + (size_t)t0 * rx, have * rx);
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        const uint32_t off = tile_row(16 * t + n) * rx + (16 * wave + 4 * g) * (uint32_t)sizeof(T);
        if constexpr (sizeof(T) == 2) {
          const u32x2_t x = bx.load8(off);
          rgd[t][0] = x[0];
          rgd[t][1] = x[1];
        } else {
          rgd[t] = bx.load16(off);
        }
      }
    }
  };
  // the decays run one chunk further ahead: loads return in order, and waiting for one issued
  // after the tiles would wait for the tiles
  float rgg = 0.f;
  auto load_decay = [&](int c) {
    if (wave == 0) {
      const int64_t t = token(c, lane) + (REV ? 1 : 0);
      rgg = c >= first && c < last && t < hi ? (w.g_fixed ? w.g[h] : w.g[(size_t)t * w.H + h]) : 0.f;
    }
  };

  // state: S[ct] holds rows 16 ct + 4 g + i of column 16 wave + n
  f32x4_t S[CT];
  auto state_io = [&](auto fn) {  // fn(ct, i, element index)
    const size_t b0 = ((size_t)sq * w.H + h) * (size_t)DK * w.dv;
    const int vc = vt * VT + 16 * wave + n;
#pragma unroll
    for (int ct = 0; ct < CT; ++ct)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int kc = 16 * ct + 4 * g + i;
        fn(ct, i, b0 + (w.s_t ? (size_t)vc * DK + kc : (size_t)kc * w.dv + vc));
      }
  };
#pragma unroll
  for (int ct = 0; ct < CT; ++ct) S[ct] = zero4();
  if (!STATE_ONLY) {
    if (w.s0) state_io([&](int ct, int i, size_t at) { S[ct][i] = w.s0[at]; });
    if (w.split && !head_seg) {  // the segments before this one, in walk order
      const int cnt = REV ? nsg - 1 - sg : sg;
      for (int j = 0; j < cnt; ++j) {
        const int64_t s = seg - sg + (REV ? nsg - 1 - j : j);
        const float d = w.seg_dec[(size_t)s * w.H + h];
        const f32x4_t* B = (const f32x4_t*)seg_at(s);
#pragma unroll
        for (int ct = 0; ct < CT; ++ct) {
          const f32x4_t x = B[ct * NT + tid];
#pragma unroll
          for (int i = 0; i < 4; ++i) S[ct][i] = fmaf(S[ct][i], d, x[i]);
        }
      }
    }
  }
  float seg_dec = 1.f;

  const int steps = last - first;
  if (steps > 0) {
    load_decay(REV ? last - 1 : first);
    if (wave == 0) chunk_decays(dec[0], rgg, lane);
    load_decay(REV ? last - 2 : first + 1);
    prefetch(REV ? last - 1 : first);
  }
  for (int it = 0; it < steps; ++it) {
    const int c = REV ? last - 1 - it : first + it;
    const Decays& dc = dec[it & 1];
    lds_barrier();  // the previous chunk's tiles are consumed
#pragma unroll
    for (int i = 0; i < QU; ++i) {
      const int u = tid + NT * i, r = u / (KT::RB / 16), x = u % (KT::RB / 16);
      if constexpr (!STATE_ONLY) *(u32x4_t*)(sQ + KT::unit(r, x)) = rgq[i];
      *(u32x4_t*)(sK + KT::unit(r, x)) = rgk[i];
    }
#pragma unroll
    for (int i = 0; i < VU; ++i) {
      const int u = tid + NT * i, r = u / (VTl::RB / 16), x = u % (VTl::RB / 16);
      *(u32x4_t*)(sV + VTl::unit(r, x)) = rgv[i];
      if constexpr (DOT == kDotCross && !STATE_ONLY) *(u32x4_t*)(sX + VTl::unit(r, x)) = rgx[i];
    }
    float xd[DOT == kDotRow ? 4 : 1][4];
    if constexpr (DOT == kDotRow && !STATE_ONLY) {
#pragma unroll
      for (int t = 0; t < 4; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          xd[t][i] = __uint_as_float(sizeof(T) == 4 ? rgd[t][i] : i & 1 ? rgd[t][i >> 1] & 0xFFFF0000u : rgd[t][i >> 1] << 16);
    }
    // the next chunk's decays (its logarithms arrived with this chunk's tiles)
    if (wave == 0 && it + 1 < steps) chunk_decays(dec[(it + 1) & 1], rgg, lane);
    load_decay(REV ? c - 2 : c + 2);
    if (it + 1 < steps) prefetch(REV ? c - 1 : c + 1);
    lds_barrier();

    if constexpr (DOT == kDotRow && !REV && !STATE_ONLY) {
      if (c % kLinaGroup == 0) {
        const int64_t grp = w.cs ? lo / (C * kLinaGroup) + sq + c / kLinaGroup
                                 : (int64_t)sq * ((nch + kLinaGroup - 1) / kLinaGroup) + c / kLinaGroup;
        f32x4_t* to = (f32x4_t*)(w.snap + ((size_t)grp * seg_stride + (size_t)h * p.nv + vt) * (DK * VT));
#pragma unroll
        for (int ct = 0; ct < CT; ++ct) to[ct * NT + tid] = S[ct];
      }
    }

    f32x4_t acc[4];
    if constexpr (!STATE_ONLY) {
      // P = r o (Q K^T): wave w makes rows 16 w .., the transposed tiles K Q^T
      {
        Frag<T> fq[KS], fx[DOT == kDotCross ? 2 : 1];
        const int row = 16 * wave + n;
#pragma unroll
        for (int s = 0; s < KS; ++s) row_frag<T, DK>(fq[s], sQ, row, s, g);
        if constexpr (DOT == kDotCross) {
          row_frag<T, VT>(fx[0], sX, row, 0, g);
          row_frag<T, VT>(fx[1], sX, row, 1, g);
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
              row_frag<T, DK>(fk, sK, 16 * J + n, s, g);
              mma(a, fk, fq[s]);
            }
            if constexpr (DOT == kDotCross) {
#pragma unroll
              for (int s = 0; s < 2; ++s) {
                Frag<T> fv;
                row_frag<T, VT>(fv, sV, 16 * J + n, s, g);
                mma(e, fv, fx[s]);
              }
            }
            const float4 jh = *(const float4*)&dc.hi[16 * J + 4 * g], jl = *(const float4*)&dc.lo[16 * J + 4 * g];
            const float jhs[4] = {jh.x, jh.y, jh.z, jh.w}, jls[4] = {jl.x, jl.y, jl.z, jl.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int j = 16 * J + 4 * g + i;
              const float r = a[i] * fast_exp2((ih - jhs[i]) + (il - jls[i]));
              x[i] = j <= row ? r : 0.f;
              if constexpr (DOT == kDotCross) {
                const float m = j < row ? r * e[i] : 0.f;
                own_sum += m;
                const float cs = row16_sum(m);
                if (n == 0) sdot[wave][j] = cs;
              }
            }
          }
          if (J <= (wave | 1)) st_quad<T>(sP + PT::quad(row, 4 * J + g), x);
        }
        if constexpr (DOT == kDotCross) {
          own_sum += __shfl_xor(own_sum, 16);
          own_sum += __shfl_xor(own_sum, 32);
          if (g == 0) sdot2[row] = own_sum;
        }
      }
      // the start state's part: rows of S^T against the rows of Q
#pragma unroll
      for (int t = 0; t < 4; ++t) acc[t] = zero4();
#pragma unroll
      for (int s = 0; s < KS; ++s) {
        Frag<T> fs, fl;
        if constexpr (sizeof(T) == 2 && DOT == kDotRow) {
          const float x[8] = {S[2 * s][0], S[2 * s][1], S[2 * s][2], S[2 * s][3],
                              S[2 * s + 1][0], S[2 * s + 1][1], S[2 * s + 1][2], S[2 * s + 1][3]};
          split_pair(x, fs, fl);
        } else {
          fs.from_acc(S[2 * s], S[2 * s + 1]);
        }
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          Frag<T> fq;
          row_frag<T, DK>(fq, sQ, 16 * t + n, s, g);
          mma(acc[t], fs, fq);
          if constexpr (sizeof(T) == 2 && DOT == kDotRow) mma(acc[t], fl, fq);
        }
      }
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        const float rw = dc.row[16 * t + n];
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[t][i] *= rw;
      }
      if constexpr (DOT == kDotRow) {
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          const float(&x)[4] = xd[t];
          float d = acc[t][0] * x[0] + acc[t][1] * x[1] + acc[t][2] * x[2] + acc[t][3] * x[3];
          d += __shfl_xor(d, 16);
          d += __shfl_xor(d, 32);
          if (g == 0) sdot[wave][16 * t + n] = d;
        }
      }
    }
    if constexpr (!STATE_ONLY) lds_barrier();

    if constexpr (DOT != kDotNone && !STATE_ONLY) {
      if (wave == 1) {
        float d;
        if constexpr (DOT == kDotRow) {
          d = (sdot[0][lane] + sdot[1][lane]) + (sdot[2][lane] + sdot[3][lane]);
        } else {
          d = -sdot2[lane];
          for (int x = lane >> 4; x < 4; ++x) d += sdot[x][lane];
        }
        const int64_t tk = token(c, lane);
        if (tk < hi) w.dots[((size_t)vt * w.H + h) * p.rows + tk] = d;
      }
    }

    // V along the tokens: raw for the outputs, weighted for the state
    Frag<T> fv[2];
    tok_frag<T, VT>(fv[0], sV, 16 * wave, 0, lane);
    tok_frag<T, VT>(fv[1], sV, 16 * wave, 1, lane);
    if constexpr (!STATE_ONLY) {
#pragma unroll
      for (int t = 0; t < 4; ++t) {
#pragma unroll
        for (int s = 0; s <= t / 2; ++s) {
          Frag<T> fp;
          col_frag<T>(fp, sP, 16 * t + n, s, g);
          mma(acc[t], fv[s], fp);
        }
      }
      // A non-finite value row spoils (0 times it) the tokens before it in its tile; the last
      // tile sees every row.  Rare: the outputs of the chunk are then summed row by row.
      bool bad = false;
#pragma unroll
      for (int i = 0; i < 4; ++i) bad |= !(fabsf(acc[3][i]) < __builtin_inff());
      if (__builtin_expect(__any(bad), 0)) {
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          f32x4_t o = zero4();
#pragma unroll
          for (int s = 0; s < KS; ++s) {
            Frag<T> fs, fq;
            fs.from_acc(S[2 * s], S[2 * s + 1]);
            row_frag<T, DK>(fq, sQ, 16 * t + n, s, g);
            mma(o, fs, fq);
          }
          const float rw = dc.row[16 * t + n];
#pragma unroll
          for (int i = 0; i < 4; ++i) o[i] *= rw;
          for (int j = 0; j <= 16 * t + n; ++j) {
            const char* pp = sP + PT::quad(16 * t + n, j >> 2) + (j & 3) * sizeof(T);
            const float pj = Elem<T>::load(pp, 0);
            float x[4];
            ld_quad<T>(sV + VTl::quad(j, 4 * wave + g), 0, x);
#pragma unroll
            for (int i = 0; i < 4; ++i) o[i] = fmaf(pj, x[i], o[i]);
          }
          acc[t] = o;
        }
      }
      const int64_t t0 = lo + (int64_t)c * C;
      const uint32_t have = (uint32_t)min((int64_t)C, hi - t0);
      if (sizeof(T) == 2 && !w.out_f32) {
        const Rows bo((char*)w.out + ((size_t)t0 * w.H + h) * w.dv * 2 + vt * VT * 2, have * ro * 2);
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          const u32x2_t x = {pack_bf16x2(acc[t][0], acc[t][1]), pack_bf16x2(acc[t][2], acc[t][3])};
          bo.store8((tile_row(16 * t + n) * ro + 16 * wave + 4 * g) * 2, x);
        }
      } else {
        const Rows bo((char*)w.out + ((size_t)t0 * w.H + h) * w.dv * 4 + vt * VT * 4, have * ro * 4);
#pragma unroll
        for (int t = 0; t < 4; ++t)
          bo.store16((tile_row(16 * t + n) * ro + 16 * wave + 4 * g) * 4, __builtin_bit_cast(u32x4_t, acc[t]));
      }
    }
    // S <- decay S + K^T (col o V)
    const float tot = dc.tot;
    seg_dec *= tot;
#pragma unroll
    for (int ct = 0; ct < CT; ++ct)
#pragma unroll
      for (int i = 0; i < 4; ++i) S[ct][i] *= tot;
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      const float4 c0 = *(const float4*)&dc.col[32 * s + 8 * g], c1 = *(const float4*)&dc.col[32 * s + 8 * g + 4];
      const float cw[8] = {c0.x, c0.y, c0.z, c0.w, c1.x, c1.y, c1.z, c1.w};
      float x[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] = fv[s].get(e) * cw[e];
      Frag<T> fh, fl;
      if constexpr (sizeof(T) == 2) split_pair(x, fh, fl);
      else {
#pragma unroll
        for (int e = 0; e < 8; ++e) fh.w[e] = x[e];
      }
#pragma unroll
      for (int ct = 0; ct < CT; ++ct) {
        Frag<T> fk;
        tok_frag<T, DK>(fk, sK, 16 * ct, s, lane);
        mma(S[ct], fk, fh);
        if constexpr (sizeof(T) == 2) mma(S[ct], fk, fl);
      }
    }

    if constexpr (DOT == kDotRow && REV && !STATE_ONLY) {
      if (c % kLinaGroup == 0) {  // D at the chunk's first token
        const int64_t grp = w.cs ? lo / (C * kLinaGroup) + sq + c / kLinaGroup
                                 : (int64_t)sq * ((nch + kLinaGroup - 1) / kLinaGroup) + c / kLinaGroup;
        const size_t slot = (size_t)grp * seg_stride + (size_t)h * p.nv + vt;
        const f32x4_t* from = (const f32x4_t*)(w.snap + slot * (DK * VT));
        float d = 0.f;
#pragma unroll
        for (int ct = 0; ct < CT; ++ct) {
          const f32x4_t x = from[ct * NT + tid];
#pragma unroll
          for (int i = 0; i < 4; ++i) d = fmaf(x[i], S[ct][i], d);
        }
#pragma unroll
        for (int off = 1; off < 64; off <<= 1) d += __shfl_xor(d, off);
        lds_barrier();  // sdot is consumed
        if (lane == 0) sdot[wave][0] = d;
        lds_barrier();
        if (tid == 0) {
          const float gl = w.g_fixed ? w.g[h] : w.g[(size_t)(lo + (int64_t)c * C) * w.H + h];
          w.anchor[slot] = expf(gl) * ((sdot[0][0] + sdot[1][0]) + (sdot[2][0] + sdot[3][0]));
        }
      }
    }
  }

  if constexpr (STATE_ONLY) {
    f32x4_t* to = (f32x4_t*)seg_at(seg);
#pragma unroll
    for (int ct = 0; ct < CT; ++ct) to[ct * NT + tid] = S[ct];
    if (tid == 0 && vt == 0) w.seg_dec[(size_t)seg * w.H + h] = seg_dec;
  } else if (w.sT && tail_seg) {
    // the reverse walk's state is the gradient after the first token's decay
    const float d = REV && nch > 0 ? expf(w.g_fixed ? w.g[h] : w.g[(size_t)lo * w.H + h]) : 1.f;
    state_io([&](int ct, int i, size_t at) { w.sT[at] = S[ct][i] * d; });
  }
}

template <typename T, int DK, bool REV, int DOT, bool STATE_ONLY>
hipError_t launch_t(const WalkParams& p) {
  const auto kern = lina_walk_kernel<T, DK, REV, DOT, STATE_ONLY>;
  const int lds = Tile<T, DK>::BYTES * (STATE_ONLY ? 1 : 2) +
                  Tile<T, 64>::BYTES * (STATE_ONLY ? 1 : (DOT == kDotCross ? 3 : 2));
  if (lds > 64 * 1024) {
    const hipError_t e = hipFuncSetAttribute((const void*)kern, hipFuncAttributeMaxDynamicSharedMemorySize, lds);
    if (e != hipSuccess) return e;
  }
  const LinaWalk& w = p.w;
  const int qk = w.q.heads < w.k.heads ? w.q.heads : w.k.heads;
  const int hk = qk < w.v.heads ? qk : w.v.heads;
  const int share = w.H / hk * p.nv;
  const int64_t blocks = (p.nseg * hk + 7) / 8 * share * 8;
  if (blocks > 0x7FFFFFFF) return hipErrorInvalidValue;
  hipLaunchKernelGGL(kern, dim3((unsigned)blocks), dim3(NT), lds, (hipStream_t)w.stream, p);
  return hipGetLastError();
}

template <typename T, int DK>
hipError_t launch_d(const WalkParams& p, bool state_only) {
  const LinaWalk& w = p.w;
  if (state_only) return w.rev ? launch_t<T, DK, true, kDotNone, true>(p) : launch_t<T, DK, false, kDotNone, true>(p);
  if (w.dot == kDotCross) return w.rev ? launch_t<T, DK, true, kDotCross, false>(p) : hipErrorInvalidValue;
  if (w.dot == kDotRow) return w.rev ? launch_t<T, DK, true, kDotRow, false>(p) : launch_t<T, DK, false, kDotRow, false>(p);
  return w.rev ? launch_t<T, DK, true, kDotNone, false>(p) : launch_t<T, DK, false, kDotNone, false>(p);
}

// Packed offsets clamped to [0, T] and made non-decreasing (a running maximum), cs[0] = 0.
constexpr int NTB = 1024;
__global__ __launch_bounds__(NTB) void lina_offsets_kernel(const int* __restrict__ cu, int nseq, int T,
                                                           int* __restrict__ cs) {
  __shared__ int part[NTB];
  const int tid = threadIdx.x, per = (nseq + NTB - 1) / NTB;
  const int s0 = min(nseq, tid * per), s1 = min(nseq, s0 + per);
  int mx = 0;
  for (int i = s0; i < s1; ++i) mx = max(mx, min(max(cu[i + 1], 0), T));
  part[tid] = mx;
  __syncthreads();
  for (int off = 1; off < NTB; off <<= 1) {
    const int v = tid >= off ? part[tid - off] : 0;
    __syncthreads();
    part[tid] = max(part[tid], v);
    __syncthreads();
  }
  int run = tid ? part[tid - 1] : 0;
  if (tid == 0) cs[0] = 0;
  for (int i = s0; i < s1; ++i) {
    run = max(run, min(max(cu[i + 1], 0), T));
    cs[i + 1] = run;
  }
}

// dq, dk of heads that share them: [rows, H, d] fp32 -> [rows, heads, d], summed in order
template <typename T>
__global__ __launch_bounds__(256) void lina_headsum_kernel(const float* __restrict__ part, void* __restrict__ out,
                                                           int64_t quads, int heads, int group, int qd) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= quads) return;
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

// dg from the walks' parts: one workgroup of 16 waves per group of 16 chunks and head,
// wave = chunk, lane = token
__global__ __launch_bounds__(1024) void lina_ddecay_kernel(const int* __restrict__ cs, int nseq, int T, int H,
                                                           int64_t rows, const float* __restrict__ a,
                                                           const float* __restrict__ b, const float* __restrict__ e,
                                                           int na, int ne, const float* __restrict__ anchor,
                                                           const float* __restrict__ g, bool g_fixed,
                                                           float* __restrict__ dg, double* __restrict__ part) {
  __shared__ double chunk_sum[kLinaGroup];
  const int64_t grp = blockIdx.x;
  const int h = blockIdx.y, lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int per = C * kLinaGroup;
  int64_t lo, hi;
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
  } else {
    const int groups = max(1, (T + per - 1) / per);
    lo = grp / groups * T;
    hi = lo + T;
    gi = (int)(grp % groups);
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
    for (int x = 0; x < na; ++x) D += anchor[((size_t)grp * H + h) * na + x];
    for (int x = 0; x < wave; ++x) D += chunk_sum[x];
  }
  double r = in ? ev + (pre - (bv - av)) + D : 0.;
  if (in && (g_fixed ? g[h] : g[(size_t)t * H + h]) < kLeast) r = 0.;  // a reset passes nothing on
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

hipError_t launch_lina_walk(const LinaWalk& w) {
  WalkParams p;
  p.w = w;
  p.nv = w.dv / VT;
  p.rows = w.cs ? w.T : (int64_t)w.n * w.T;
  const int64_t nch = ((int64_t)w.T + C - 1) / C;
  p.nseg = w.cs ? lina_pieces(w.T, w.n, w.L) : (int64_t)w.n * (nch > 0 ? (nch + w.L - 1) / w.L : 1);
  if (p.nseg == 0) return hipSuccess;
  for (int pass = w.split ? 0 : 1; pass < 2; ++pass) {
    const bool so = pass == 0;
    const hipError_t e = w.bf16 ? (w.dk == 128 ? launch_d<bf16_t, 128>(p, so) : launch_d<bf16_t, 64>(p, so))
                                : (w.dk == 128 ? launch_d<float, 128>(p, so) : launch_d<float, 64>(p, so));
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

hipError_t launch_lina_offsets(const int* cu, int n, int T, int* cs, void* stream) {
  hipLaunchKernelGGL(lina_offsets_kernel, dim3(1), dim3(NTB), 0, (hipStream_t)stream, cu, n, T, cs);
  return hipGetLastError();
}

hipError_t launch_lina_headsum(const float* part, void* out, int64_t rows, int heads, int group, int d, bool bf16,
                               void* stream) {
  const int64_t quads = rows * heads * (d / 4);
  if (quads == 0) return hipSuccess;
  const int64_t blocks = (quads + 255) / 256;
  if (blocks > 0x7FFFFFFF) return hipErrorInvalidValue;
  if (bf16)
    hipLaunchKernelGGL(lina_headsum_kernel<bf16_t>, dim3((unsigned)blocks), dim3(256), 0, (hipStream_t)stream, part,
                       out, quads, heads, group, d / 4);
  else
    hipLaunchKernelGGL(lina_headsum_kernel<float>, dim3((unsigned)blocks), dim3(256), 0, (hipStream_t)stream, part,
                       out, quads, heads, group, d / 4);
  return hipGetLastError();
}

hipError_t launch_lina_ddecay(const LinaWalk& w, const float* a, const float* b, const float* e, int na, int ne,
                              const float* anchor, float* dg, double* part, float* dg_fixed) {
  const int64_t rows = w.cs ? w.T : (int64_t)w.n * w.T;
  const int64_t per = (int64_t)C * kLinaGroup;
  const int64_t groups = w.cs ? lina_pieces(w.T, w.n, kLinaGroup) : (int64_t)w.n * (((int64_t)w.T + per - 1) / per);
  if (rows > 0 && groups > 0) {
    hipLaunchKernelGGL(lina_ddecay_kernel, dim3((unsigned)groups, (unsigned)w.H), dim3(1024), 0,
                       (hipStream_t)w.stream, w.cs, w.n, w.T, w.H, rows, a, b, e, na, ne, anchor, w.g, w.g_fixed, dg,
                       part);
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
