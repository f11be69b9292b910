// kda_gdr_bwd.hip -- gradients of q, k and beta of the gated delta rule with one decay per head, chunk by
// chunk, from what the two walks left: S, the state a chunk starts from, R, the gradient of the state behind
// it, r = v - e^g S^T k, y = dv.  With u = b o r (b is taken to the products, fp32) and the chunk's decays e^G (from
// its start), e^G' (to its end, the next token's decay included), D_ij = e^{G_i - G_j},
//   E_ij = D_ij do_i . u_j (j <= i),   F_ij = D_ij y_i . u_j (j < i),
//   dq = E K + e^G o (do S^T),
//   dk = E^T Q - (F + F^T) K - e^G o (y S^T) + e^G' o (u R^T).
// One workgroup makes dq and dk of one chunk and shared head, summed over the heads it serves in registers: wave
// w block w of 16 tokens, in 16 x 16 tiles with rows = channels, columns = tokens, so that a lane stores four
// neighbouring channels.  Operands go through LDS, 64 value columns at a time, the
// two states one after the other through the same tile: 72 KB (bf16), two workgroups to a compute unit, for which 10
// registers do not fit (44 bytes of scratch a lane).  B4 H32 T8K: 727 us (one workgroup to a unit, both states at once: 1,034) for
// 2.5 GB read, 1.07 of them states, and 0.7 written, 4.4 TB/s: loads and products take turns between barriers.  Scores are split in two terms: in one, dk is off by 3.4e-3 of its norm instead of 2.8e-3.
#include "kda_gdr_tile.h"

namespace kda {

namespace {

struct GradParams {
  GdrGrad a;
  int64_t chunks, rows;
};

template <typename T, int DK>
struct GradLds {
  static constexpr int Q = 0, K = Tile<T, DK>::BYTES, S = 2 * K;
  static constexpr int DO = S + Tile<T, DK>::BYTES, Y = DO + Tile<T, VT>::BYTES, U = Y + Tile<T, VT>::BYTES;
  static constexpr int BYTES = U + Tile<T, VT>::BYTES;
};

// slots 0-3 hold rows 32 s + 4 g .., slots 4-7 rows 32 s + 16 + 4 g .. of column c0 + n
template <typename T, int D>
__device__ __forceinline__ void grad_col_frag(Frag<T>& f, const char* t, int c0, int s, int lane) {
  const int g = lane >> 4, n = lane & 15;
  if constexpr (sizeof(T) == 2) {
#ifndef KDA_HOST_PASS
    const char* p = t + 32 * s * Tile<T, D>::RB + ((uint32_t)Tile<T, D>::quad(4 * g + (n >> 2), n & 3) ^ (c0 * 2));
    const v4s_t a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s*)p);
    const v4s_t b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s*)(p + 16 * Tile<T, D>::RB));
    const uint2 x = __builtin_bit_cast(uint2, a), y = __builtin_bit_cast(uint2, b);
    f.w[0] = x.x; f.w[1] = x.y; f.w[2] = y.x; f.w[3] = y.y;
#endif
  } else {
    const int c = c0 + n;
#pragma unroll
    for (int e = 0; e < 8; ++e)
      f.w[e] = *(const float*)(t + Tile<T, D>::quad(32 * s + 16 * (e >> 2) + 4 * g + (e & 3), c >> 2) + (c & 3) * 4);
  }
}

template <typename T, int DK>
__global__ __launch_bounds__(NT, sizeof(T) == 2 ? 2 : 1) void gdr_grad_kernel(const GradParams gp) {
  typedef GradLds<T, DK> Lds;
  constexpr int CT = DK / 16;
  extern __shared__ __align__(16) char smem[];
  __shared__ __align__(16) Decays dec, back;
  __shared__ __align__(16) float beta[C];
  const GdrWalk& f = gp.a.f;
  const LinaWalk& w = f.walk;
  // The wave's number in a scalar: branches on it are jumps.  Under an execution mask, as the compiler may
  // put short ones, matrix instructions would run all the same.
  const int tid = threadIdx.x, lane = tid & 63, g = lane >> 4, n = lane & 15;
  const int wave = (int)uniform64(tid >> 6);
  const int heads = w.q.heads, group = w.H / heads, nv = w.dv / VT;
  const int64_t chunk = blockIdx.x / heads;
  const int hk = (int)uniform64(blockIdx.x % heads);
  Chain ch;
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
  f32x4_t dq[CT], dk[CT];
#pragma unroll
  for (int ct = 0; ct < CT; ++ct) dq[ct] = dk[ct] = zero4();
  {
    const Operand<T> q(w.q, w, hk * group, DK, 0), k(w.k, w, hk * group, DK, 0);
    Stage<T, DK> a, b;
    a.load(q.rows(t0, have), q.step, false, tid);
    b.load(k.rows(t0, have), k.step, false, tid);
    a.store(smem + Lds::Q, tid);
    b.store(smem + Lds::K, tid);
  }
  const uint32_t rb = row_base<T, VT, false>(lane);
  auto rows = [&](Frag<T>& fr, int tile, int block, int s) {
    row_frag<T>(fr, smem + tile, rows_at<T, VT, false>(rb, 16 * block), s);
  };
  auto cols = [&](Frag<T>& fr, int tile, int ct, int s) {
    grad_col_frag<T, DK>(fr, smem + tile, 16 * ct, s, lane);
  };
  for (int x = 0; x < group; ++x) {
    const int h = hk * group + x;
    ch.h = h;
    const size_t at = ((size_t)chunk * w.H + h) * nv * (VT * DK);
    Stage<T, VT> rd, ry, ru;
    Stage<T, DK> rs;
    auto fetch_rows = [&](int vt) {
      const uint32_t col = vt * VT * sizeof(T);
      auto one = [&](Stage<T, VT>& r, const LinaOp& op) {
        const Operand<T> o(op, w, h, w.dv, 0);
        r.load(Rows(o.p + (size_t)t0 * o.step + col, have * o.step - col), o.step, false, tid);
      };
      one(rd, gp.a.d_o);
      one(ry, gp.a.y);
      one(ru, f.r);
    };
    auto fetch_state = [&](const void* p, int vt) {
      rs.load(Rows((const T*)p + at + vt * (VT * DK), VT * DK * sizeof(T)), DK * sizeof(T), false, tid);
    };
    __syncthreads();  // the head before is done with the decays
    {
      if (wave == 0) chunk_decays(dec, row_decay<false>(w, ch, c, lane), lane);
      if (wave == 1) {  // of the reversed chunk: its row is the decay from a token to the chunk's end and over the next
        const int64_t t = t0 + C - lane;
        chunk_decays(back, t < ch.hi ? ch.decay_log(w, t) : 0.f, lane);
      }
      if (wave == 2) {
        const int64_t t = t0 + lane;
        beta[lane] = t < ch.hi ? Elem<T>::load(f.beta, (size_t)t * w.H + h) : 0.f;
      }
      if (wave == 3 && t0 + lane < ch.hi) {
        const int64_t t = t0 + lane;
        float d = 0.f;
        for (int vt = 0; vt < nv; ++vt) d += gp.a.dots2[((size_t)vt * w.H + h) * gp.rows + t];
        Elem<T>::store(gp.a.dbeta, (size_t)t * w.H + h, d);
      }
    }
    __syncthreads();
    const float bn = beta[16 * wave + n], row = dec.row[16 * wave + n], end = back.row[C - 1 - 16 * wave - n] * bn;
    // scores of own tokens (columns) with block B's (rows): E, as dq and dk take it before and behind the own
    // block, and F + F^T; of the own block both halves
    f32x4_t ee[4], ff[4], ed = zero4(), fd = zero4();
#pragma unroll
    for (int B = 0; B < 4; ++B) ee[B] = ff[B] = zero4();
    for (int vt = 0; vt < nv; ++vt) {
      if (vt > 0) __syncthreads();
      fetch_rows(vt);
      fetch_state(f.kept, vt);
      rd.store(smem + Lds::DO, tid);
      ry.store(smem + Lds::Y, tid);
      ru.store(smem + Lds::U, tid);
      rs.store(smem + Lds::S, tid);
      __syncthreads();
      Frag<T> fo[2], fy[2], fu[2];
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        rows(fo[s], Lds::DO, wave, s);
        rows(fy[s], Lds::Y, wave, s);
        rows(fu[s], Lds::U, wave, s);
      }
#pragma unroll
      for (int ct = 0; ct < CT; ++ct) {
        f32x4_t a = zero4(), b = zero4();
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          Frag<T> fs;
          cols(fs, Lds::S, ct, s);
          mma(a, fs, fo[s]);
          mma(b, fs, fy[s]);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          dq[ct][i] = fmaf(row, a[i], dq[ct][i]);
          dk[ct][i] = fmaf(-row, b[i], dk[ct][i]);
        }
        in_turn();
      }
#pragma unroll
      for (int B = 0; B < 4; ++B)
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          Frag<T> a;
          if (B <= wave) {
            rows(a, Lds::U, B, s);
            mma(ee[B], a, fo[s]);
            mma(ff[B], a, fy[s]);
          } else {
            rows(a, Lds::DO, B, s);
            mma(ee[B], a, fu[s]);
            rows(a, Lds::Y, B, s);
            mma(ff[B], a, fu[s]);
          }
          in_turn();
        }
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        mma(ed, fo[s], fu[s]);
        mma(fd, fy[s], fu[s]);
      }
      __syncthreads();
      fetch_state(gp.a.kept_r, vt);
      rs.store(smem + Lds::S, tid);
      __syncthreads();
#pragma unroll
      for (int ct = 0; ct < CT; ++ct) {
        f32x4_t a = zero4();
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          Frag<T> fs;
          cols(fs, Lds::S, ct, s);
          mma(a, fs, fu[s]);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) dk[ct][i] = fmaf(end, a[i], dk[ct][i]);
        in_turn();
      }
    }
    // decays and masks
    const float ih = dec.hi[16 * wave + n], il = dec.lo[16 * wave + n];
    f32x4_t e1[4], e2[4];
#pragma unroll
    for (int B = 0; B < 4; ++B) {
      const float4 jh4 = *(const float4*)&dec.hi[16 * B + 4 * g], jl4 = *(const float4*)&dec.lo[16 * B + 4 * g];
      const float jh[4] = {jh4.x, jh4.y, jh4.z, jh4.w}, jl[4] = {jl4.x, jl4.y, jl4.z, jl4.w};
      const float4 b4 = *(const float4*)&beta[16 * B + 4 * g];
      const float bj[4] = {b4.x, b4.y, b4.z, b4.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float d = (ih - jh[i]) + (il - jl[i]);  // exponent from token 16 B + 4 g + i to the own one
        const int j = 16 * B + 4 * g + i - 16 * wave;
        const float r = fast_exp2(j <= n ? d : -d) * (j <= n ? bj[i] : bn);  // b of the token whose r it is
        e1[B][i] = j <= n ? ee[B][i] * r : 0.f;
        e2[B][i] = j >= n ? (B == wave ? ed[i] : ee[B][i]) * r : 0.f;
        ff[B][i] = j < n ? -ff[B][i] * r : j > n ? -(B == wave ? fd[i] : ff[B][i]) * r : 0.f;
      }
    }
    Terms<T, kMost<T>> f1[2], f2[2], f3[2];
    const Residual res;
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      split(res, e1[2 * s], e1[2 * s + 1], f1[s]);
      split(res, e2[2 * s], e2[2 * s + 1], f2[s]);
      split(res, ff[2 * s], ff[2 * s + 1], f3[s]);
    }
#pragma unroll
    for (int ct = 0; ct < CT; ++ct)
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        Frag<T> a;
        cols(a, Lds::K, ct, s);
#pragma unroll
        for (int m = 0; m < kMost<T>; ++m) {
          mma(dq[ct], a, f1[s].f[m]);
          mma(dk[ct], a, f3[s].f[m]);
        }
        cols(a, Lds::Q, ct, s);
#pragma unroll
        for (int m = 0; m < kMost<T>; ++m) mma(dk[ct], a, f2[s].f[m]);
        in_turn();
      }
  }
  const uint32_t step = heads * DK * sizeof(T);
  const size_t to = ((size_t)t0 * heads + hk) * DK * sizeof(T);
  const Rows bq((char*)gp.a.dq + to, have * step), bk((char*)gp.a.dk + to, have * step);
#pragma unroll
  for (int ct = 0; ct < CT; ++ct) {
    const uint32_t off = (16 * wave + n) * step + (16 * ct + 4 * g) * sizeof(T);
    if constexpr (sizeof(T) == 2) {
      bq.store8(off, u32x2_t{pack_bf16x2(dq[ct][0], dq[ct][1]), pack_bf16x2(dq[ct][2], dq[ct][3])});
      bk.store8(off, u32x2_t{pack_bf16x2(dk[ct][0], dk[ct][1]), pack_bf16x2(dk[ct][2], dk[ct][3])});
    } else {
      bq.store16(off, __builtin_bit_cast(u32x4_t, dq[ct]));
      bk.store16(off, __builtin_bit_cast(u32x4_t, dk[ct]));
    }
  }
}

template <typename T, int DK>
hipError_t grad(const GdrGrad& a) {
  GradParams gp;
  gp.a = a;
  const LinaWalk& w = a.f.walk;
  gp.chunks = gdr_chunks(w.cs != nullptr, w.T, w.n);
  gp.rows = w.cs ? w.T : (int64_t)w.n * w.T;
  const int64_t blocks = gp.chunks * w.q.heads;
  if (blocks == 0) return hipSuccess;
  if (blocks > 0xFFFFFFFFll / NT) return hipErrorInvalidValue;
  constexpr int lds = GradLds<T, DK>::BYTES;
  if (lds > 64 * 1024) {
    const hipError_t e = hipFuncSetAttribute((const void*)gdr_grad_kernel<T, DK>, hipFuncAttributeMaxDynamicSharedMemorySize, lds);
    if (e != hipSuccess) return e;
  }
  hipLaunchKernelGGL((gdr_grad_kernel<T, DK>), dim3((unsigned)blocks), dim3(NT), lds, (hipStream_t)w.stream, gp);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_gdr_grad(const GdrGrad& a) {
  if (a.f.walk.bf16) return a.f.walk.dk == 128 ? grad<bf16_t, 128>(a) : grad<bf16_t, 64>(a);
  return a.f.walk.dk == 128 ? grad<float, 128>(a) : grad<float, 64>(a);
}

}  // namespace kda
