// kda_gdr_tile.h -- device pieces shared by the kernels of the gated delta rule with one decay per
// head: LDS tiles and their fragments, values in bf16 terms, lower triangles.
#pragma once
#include "kda_gdr.h"
#include "kda_lina_tile.h"

namespace kda {

namespace {

// Between two steps of unrolled code: the compiler moves nothing across, so that a step's loads are issued in the
// step before, where they stand, and no more of them are in flight than that.
__device__ __forceinline__ void in_turn() {
#ifndef KDA_HOST_PASS
  __builtin_amdgcn_sched_barrier(0);
#endif
}

// 64-row LDS tile of D elements a row, read along its rows (16 bytes of bf16 to a lane: row n, unit 4 s + g) and
// along its columns (transpose loads of 8 bytes: 16 lanes take four rows of a row group, four units or two).  A row's
// 16-byte units are permuted by the row so that both go at the rate of a linear read (256 and 128 bytes a clock): a 16-byte
// read serves lanes 0-3, 12-15 and 20-27 together, so rows 0-3 and 12-15 at one unit must not meet rows 4-11 at the next.
template <typename T, int D>
struct RowTile {
  static constexpr int RB = D * (int)sizeof(T);
  static constexpr int BYTES = C * RB;
  __device__ __forceinline__ static int unit(int row, int u) {
    const int low = (((row >> 2) ^ (row >> 3)) & 1) << 1 | ((row >> 3) & 1);
    if constexpr (sizeof(T) == 4) return row * RB + (((u & ~15) | ((u ^ row) & 15)) << 4);
    else if constexpr (D == 128) return row * RB + ((u ^ ((row & 3) << 2 | low)) << 4);
    else return row * RB + ((u ^ ((row & 2) << 1 | low)) << 4);
  }
};

// Channel of row r of state tile ct: two tiles share 32 channels so that a lane's four rows of both, 4 g + i, are eight
// channels in a row, 32 (ct / 2) + 8 g + 4 (ct % 2) + i.
__device__ __forceinline__ constexpr int channel(int ct, int r) { return 32 * (ct >> 1) + 8 * (r >> 2) + 4 * (ct & 1) + (r & 3); }

// A lane's addresses in row-wise tiles of D elements: rows n (fragment of 32 channels: slots hold channels 32 s + 8 g + e).
template <typename T, int D>
struct RowAt {
  uint32_t base;
  __device__ __forceinline__ explicit RowAt(int lane) {
    base = RowTile<T, D>::unit(lane & 15, (sizeof(T) == 2 ? 1 : 2) * (lane >> 4));
  }
  // rows r0 + n (r0 a multiple of 16) of the tile at t
  __device__ __forceinline__ void load(Frag<T>& f, const char* t, int r0, int s) const {
    const char* p = t + (base ^ (s * 32 * sizeof(T))) + r0 * RowTile<T, D>::RB;
    if constexpr (sizeof(T) == 2) f.load8(p);
    else f.load4x2(p, t + (base ^ (s * 32 * sizeof(T)) ^ 16) + r0 * RowTile<T, D>::RB);
  }
};

// Columns along the rows: slots 0-3 hold rows 32 s + 4 g .., slots 4-7 rows 32 s + 16 + 4 g .., the order in which two
// accumulator tiles of 16 rows hold theirs.  CHANNELS: lane n's column is channel(ct, n); else 16 ct + n.
template <typename T, int D, bool CHANNELS>
struct ColAt {
  uint32_t base;
  __device__ __forceinline__ explicit ColAt(int lane) {
    const int g = lane >> 4, n = lane & 15;
    if constexpr (sizeof(T) == 2) {
      const int row = 4 * g + (n >> 2);
      base = CHANNELS ? RowTile<T, D>::unit(row, n & 3) : RowTile<T, D>::unit(row, (n & 3) >> 1) + ((n & 1) << 3);
    } else {
      base = CHANNELS ? channel(0, n) : n;
    }
  }
  __device__ __forceinline__ void load(Frag<T>& f, const char* t, int ct, int s, int lane) const {
    if constexpr (sizeof(T) == 2) {
#ifndef KDA_HOST_PASS
      const char* p = t + (CHANNELS ? (base ^ ((ct >> 1) * 64)) + (ct & 1) * 8 : base ^ (ct * 32)) + 32 * s * RowTile<T, D>::RB;
      const v4s_t a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s*)p);
      const v4s_t b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s*)(p + 16 * RowTile<T, D>::RB));
      const uint2 x = __builtin_bit_cast(uint2, a), y = __builtin_bit_cast(uint2, b);
      f.w[0] = x.x; f.w[1] = x.y; f.w[2] = y.x; f.w[3] = y.y;
#endif
    } else {
      const int g = lane >> 4, c = CHANNELS ? base + channel(ct, 0) : base + 16 * ct;
#pragma unroll
      for (int e = 0; e < 8; ++e)
        f.w[e] = *(const float*)(t + RowTile<T, D>::unit(32 * s + 16 * (e >> 2) + 4 * g + (e & 3), c >> 2) + (c & 3) * 4);
    }
  }
};

// A thread's share of one chunk's rows, on its way from memory to LDS (NT threads).
template <typename T, int D>
using StageRows = Stage<T, D, false, RowTile<T, D>>;

// fp32 values as matrix-core operands: themselves, or in bf16 terms (three hold all 24 bits)
template <typename T, int N>
struct Terms {
  Frag<T> f[N];
};
template <typename T>
constexpr int kAll = sizeof(T) == 2 ? 3 : 1;  // terms that hold a value's 24 bits
template <typename T>
constexpr int kMost = sizeof(T) == 2 ? 2 : 1;  // terms that hold 16 of them

// What a bf16 pair leaves of the values it was rounded from, exactly: a dot product with (-1, 0) or (0, -1) takes one
// instruction where widening and subtracting take two.  The constants go through registers: as an inline operand
// -1.0 is the fp32 pattern, the pair (0, -1).  B4 H32 T8K: forward 584 us, backward 2,727 (widening and subtracting: 594 and
// 2,850); H16 T128K 2,251 (2,387).  The remainders from matrix products with -I: forward 653.
struct Residual {
  uint32_t lo = 0x0000BF80u, hi = 0xBF800000u;
  __device__ __forceinline__ Residual() {
#ifndef KDA_HOST_PASS
    asm("" : "+s"(lo), "+s"(hi));
#endif
  }
  __device__ __forceinline__ void take(uint32_t h, float& a, float& b) const {
#ifndef KDA_HOST_PASS
    const bf16x2_t x = __builtin_bit_cast(bf16x2_t, h);
    a = __builtin_amdgcn_fdot2_f32_bf16(x, __builtin_bit_cast(bf16x2_t, lo), a, false);
    b = __builtin_amdgcn_fdot2_f32_bf16(x, __builtin_bit_cast(bf16x2_t, hi), b, false);
#endif
  }
};

template <typename T, int N>
__device__ __forceinline__ void split(const Residual& res, const f32x4_t& a, const f32x4_t& b, Terms<T, N>& t) {
  if constexpr (sizeof(T) == 4) {
    t.f[0].from_acc(a, b);
  } else {
    float x[8] = {a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
#pragma unroll
    for (int m = 0; m < N; ++m)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        t.f[m].w[i] = pack_bf16x2(x[2 * i], x[2 * i + 1]);
        if (m + 1 < N) res.take(t.f[m].w[i], x[2 * i], x[2 * i + 1]);
      }
  }
}

// Made here: the compiler would put what feeds a later step's products right before them, where they wait for it,
// instead of under the products of this one.
template <typename T, int N>
__device__ __forceinline__ void made(Terms<T, N>& t) {
#ifndef KDA_HOST_PASS
#pragma unroll
  for (int m = 0; m < N; ++m)
#pragma unroll
    for (int i = 0; i < (sizeof(T) == 2 ? 4 : 8); ++i) asm volatile("" : "+v"(t.f[m].w[i]));
#endif
}
// terms of the products of two split operands, as far as the longer one's; the smallest first
template <typename T, int N, int M>
__device__ __forceinline__ void mma_terms(f32x4_t& acc, const Terms<T, N>& a, const Terms<T, M>& b) {
#pragma unroll
  for (int o = (N > M ? N : M) - 1; o >= 0; --o)
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
      for (int j = 0; j < M; ++j)
        if (i + j == o) mma(acc, a.f[i], b.f[j]);
}

// 16 x 16 block (I, J) of a lower triangle.  In memory a lane holds row n, columns 4 g .. 4 g + 3 of a block, lane after
// lane: a transposed accumulator tile is written, and an operand read, without a shuffle.
__host__ __device__ constexpr int tri(int I, int J) { return I * (I + 1) / 2 + J; }
constexpr int kTriUnits = kTriBlocks * 64;  // lane quads of a triangle

// In LDS, pairs of blocks (t, 2 s), (t, 2 s + 1), a lane's eight columns in a row: an operand of 32 columns in one read.
// The blocks above the diagonal, (0, 1) and (2, 3), are zeros that tri_clear writes once.
__host__ __device__ constexpr int tri_pair(int t, int s) { return t < 2 ? t : 2 * (t - 1) + s; }
constexpr int kTriPairs = 6;
template <typename T, int N>
constexpr int kTriBytes = kTriPairs * 64 * 8 * (int)sizeof(T) * (sizeof(T) == 2 ? N : 1);

template <typename T, int N>
__device__ __forceinline__ void tri_clear(char* p, int tid) {  // NT threads
  static_assert(NT == 256, "two blocks of 64 lanes");
  if (tid >= 128) return;
#pragma unroll
  for (int m = 0; m < (sizeof(T) == 2 ? N : 1); ++m) {
    char* at = p + (m * kTriPairs + tri_pair(tid < 64 ? 0 : 2, tid < 64 ? 0 : 1)) * 512 * sizeof(T) + (tid & 63) * 8 * sizeof(T) +
               4 * sizeof(T);
    if constexpr (sizeof(T) == 2) *(uint2*)at = make_uint2(0u, 0u);
    else *(float4*)at = make_float4(0.f, 0.f, 0.f, 0.f);
  }
}

// rows 16 t + n, columns of the block pair s, in the order of ColAt's rows
template <typename T, int N>
__device__ __forceinline__ void tri_frag(Terms<T, N>& f, const char* p, int t, int s, int lane) {
#pragma unroll
  for (int m = 0; m < N; ++m) f.f[m].load8(p + ((m * kTriPairs + tri_pair(t, s)) * 64 + lane) * 8 * sizeof(T));
}

// fp32 quads of a triangle on their way from memory to LDS, in N terms (NT threads)
template <typename T, int N>
struct StageTri {
  static constexpr int R = (kTriUnits + NT - 1) / NT;
  u32x4_t r[R];
  __device__ __forceinline__ void load(const float* base, size_t slot, int tid) {
    const Rows b(base + slot * (kTriUnits * 4), kTriUnits * 16);
#pragma unroll
    for (int i = 0; i < R; ++i) r[i] = b.load16((tid + NT * i) * 16);
  }
  __device__ __forceinline__ void store(const Residual& res, char* t, int tid) const {
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const int u = tid + NT * i;
      if (u >= kTriUnits) break;
      const int b = u >> 6, I = b < 1 ? 0 : b < 3 ? 1 : b < 6 ? 2 : 3, J = b - tri(I, 0);
      char* at = t + ((I < 2 ? I : 2 * (I - 1) + (J >> 1)) * 64 + (u & 63)) * 8 * sizeof(T) + (J & 1) * 4 * sizeof(T);
      if constexpr (sizeof(T) == 4) {
        *(u32x4_t*)at = r[i];
      } else {
        float x[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) x[j] = __uint_as_float(r[i][j]);
#pragma unroll
        for (int m = 0; m < N; ++m) {
          const uint32_t a = pack_bf16x2(x[0], x[1]), c = pack_bf16x2(x[2], x[3]);
          *(uint2*)(at + m * kTriPairs * 1024) = make_uint2(a, c);
          if (m + 1 < N) {
            res.take(a, x[0], x[1]);
            res.take(c, x[2], x[3]);
          }
        }
      }
    }
  }
};

}  // namespace

}  // namespace kda
