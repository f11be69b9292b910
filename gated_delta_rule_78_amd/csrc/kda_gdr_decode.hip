// kda_gdr_decode.hip -- the recurrent form of the gated delta rule with one decay per head: one token, or a
// few in order, for every (batch, head).
//
//   u = b (v - e^g S^T k),   S <- e^g S + k u^T,   o = S^T q = e^g S_old^T q + (k . q) u.
//
// Bandwidth bound: the fp32 d_k x d_v state is read once and, where it is updated, written once per call.  One
// workgroup owns COLS columns of one (b, h) state, a thread 4 columns of every RG-th row, in registers.  Both
// sums over the rows are of the state before the token, so a token costs one exchange between the waves.
// 256 sequences of 32 heads, d = 128: 194 us, 5.6 TB/s of states in place (a copy: 5.2).  Threads, at 16, 64 and 256
// sequences: 256 take 15.4, 50 and 196 us, 512 take 16.2, 52 and 201, 128 take 16.4, 51 and 199.
#include "kda_common.h"
#include "kda_gdr.h"

namespace kda {

namespace {

constexpr int kThreads = 256;

template <typename T, int DK>
__global__ __launch_bounds__(kThreads) void gdr_decode_kernel(const GdrDecodeArgs a) {
  constexpr int COLS = 64, NT = kThreads, NW = NT / 64;
  constexpr int TPR = COLS / 4;   // threads of a row
  constexpr int RG = NT / TPR;    // rows at a time
  constexpr int RPT = DK / RG;    // rows of a thread
  constexpr int NTK = 8;          // tokens staged at a time
  static_assert(RPT * RG == DK && RPT >= 1, "tile split");
  __shared__ __align__(16) float s_q[NTK][DK], s_k[NTK][DK], s_v[NTK][COLS];
  __shared__ float s_a[NTK], s_b[NTK], s_qk[NTK];
  __shared__ __align__(16) float s_red[2][2][NW][COLS];

  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int tiles = a.dv / COLS;
  const int64_t bh = blockIdx.x / tiles;
  const int c0 = (int)(blockIdx.x % tiles) * COLS;
  const int64_t b = bh / a.H;
  const int h = (int)(bh % a.H), hk = h / (a.H / a.Hk);
  const int cq = tid % TPR, rg = tid / TPR;
  const int ntok = a.counts ? min(max(a.counts[b], 0), a.ntok) : a.ntok;
  if (ntok == 0) return;

  f32x4_t* S = (f32x4_t*)(a.state + (size_t)bh * DK * a.dv + c0);
  const int rs = a.dv / 4;
  f32x4_t s[RPT];
#pragma unroll
  for (int i = 0; i < RPT; ++i) s[i] = __builtin_nontemporal_load(&S[(size_t)(rg + RG * i) * rs + cq]);

  for (int t0 = 0; t0 < ntok; t0 += NTK) {
    const int nb = min(NTK, ntok - t0);
    if (t0 > 0) __syncthreads();  // the previous tokens' inputs are consumed
    for (int x = tid; x < nb * DK; x += NT) {
      const int j = x / DK, c = x % DK;
      const size_t row = ((size_t)b * a.ntok + t0 + j) * a.Hk + hk;
      s_q[j][c] = a.q ? Elem<T>::load(a.q, row * DK + c) : 0.f;
      s_k[j][c] = Elem<T>::load(a.k, row * DK + c);
    }
    for (int x = tid; x < nb * COLS; x += NT) {
      const int j = x / COLS, c = x % COLS;
      s_v[j][c] = Elem<T>::load(a.v, (((size_t)b * a.ntok + t0 + j) * a.H + h) * a.dv + c0 + c);
    }
    if (tid < nb) {
      const size_t at = ((size_t)b * a.ntok + t0 + tid) * a.H + h;
      s_a[tid] = expf(a.g[at]);
      s_b[tid] = Elem<T>::load(a.beta, at);
    }
    __syncthreads();
    for (int j = wave; j < nb; j += NW) {  // k . q
      float d = 0.f;
      for (int c = lane; c < DK; c += 64) d = fmaf(s_q[j][c], s_k[j][c], d);
#pragma unroll
      for (int off = 1; off < 64; off <<= 1) d += __shfl_xor(d, off);
      if (lane == 0) s_qk[j] = d;
    }

    for (int j = 0; j < nb; ++j) {
      const int par = (t0 + j) & 1;  // two buffers: one barrier a token
      const float dec = s_a[j];
      float pk[4] = {0.f, 0.f, 0.f, 0.f}, pq[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int i = 0; i < RPT; ++i) {
        const float kk = s_k[j][rg + RG * i], qq = s_q[j][rg + RG * i];
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          s[i][x] *= dec;
          pk[x] = fmaf(kk, s[i][x], pk[x]);
          pq[x] = fmaf(qq, s[i][x], pq[x]);
        }
      }
#pragma unroll
      for (int off = TPR; off < 64; off <<= 1)
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          pk[x] += __shfl_xor(pk[x], off);
          pq[x] += __shfl_xor(pq[x], off);
        }
      if (lane < TPR) {
        *(float4*)&s_red[par][0][wave][4 * cq] = make_float4(pk[0], pk[1], pk[2], pk[3]);
        *(float4*)&s_red[par][1][wave][4 * cq] = make_float4(pq[0], pq[1], pq[2], pq[3]);
      }
      __syncthreads();
      const float bt = s_b[j];
      float u[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int w = 0; w < NW; ++w) {
        const float4 x = *(const float4*)&s_red[par][0][w][4 * cq];
        u[0] += x.x; u[1] += x.y; u[2] += x.z; u[3] += x.w;
      }
      const float4 v = *(const float4*)&s_v[j][4 * cq];
      u[0] = bt * (v.x - u[0]); u[1] = bt * (v.y - u[1]); u[2] = bt * (v.z - u[2]); u[3] = bt * (v.w - u[3]);
#pragma unroll
      for (int i = 0; i < RPT; ++i) {
        const float kk = s_k[j][rg + RG * i];
#pragma unroll
        for (int x = 0; x < 4; ++x) s[i][x] = fmaf(kk, u[x], s[i][x]);
      }
      if (a.q && tid < TPR) {
        const float qk = s_qk[j];
        float o[4] = {qk * u[0], qk * u[1], qk * u[2], qk * u[3]};
#pragma unroll
        for (int w = 0; w < NW; ++w) {
          const float4 x = *(const float4*)&s_red[par][1][w][4 * cq];
          o[0] += x.x; o[1] += x.y; o[2] += x.z; o[3] += x.w;
        }
        const size_t at = (((size_t)b * a.ntok + t0 + j) * a.H + h) * a.dv + c0 + 4 * cq;
#pragma unroll
        for (int x = 0; x < 4; ++x) Elem<T>::store(a.o, at + x, o[x]);
      }
    }
  }
  if (!a.update) return;
#pragma unroll
  for (int i = 0; i < RPT; ++i) __builtin_nontemporal_store(s[i], &S[(size_t)(rg + RG * i) * rs + cq]);
}

template <typename T, int DK>
hipError_t launch_d(const GdrDecodeArgs& a) {
  const int64_t blocks = a.BH * (a.dv / 64);
  if (blocks > 0x7FFFFFFF) return hipErrorInvalidValue;
  hipLaunchKernelGGL((gdr_decode_kernel<T, DK>), dim3((unsigned)blocks), dim3(kThreads), 0, (hipStream_t)a.stream, a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_gdr_decode(const GdrDecodeArgs& a) {
  if (a.BH == 0) return hipSuccess;
  if (a.bf16) return a.dk == 128 ? launch_d<bf16_t, 128>(a) : launch_d<bf16_t, 64>(a);
  return a.dk == 128 ? launch_d<float, 128>(a) : launch_d<float, 64>(a);
}

}  // namespace kda
