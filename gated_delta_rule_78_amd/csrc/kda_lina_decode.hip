// kda_lina_decode.hip -- the recurrent form of linear attention with a decay per head: one
// token, or a few in order, for every (batch, head), the state in place.
//
//   S <- e^g S + k v^T,   o = S^T q.
//
// Bandwidth bound: the fp32 d_k x d_v state is read once and written once per call.  One
// workgroup owns COLS columns of one (b, h) state, a thread 4 columns of every RG-th row, in
// registers; the sum over the rows goes through lane shuffles and one LDS exchange per token.
#include "kda_common.h"
#include "kda_lina.h"

namespace kda {

namespace {

template <typename T, int DK, int COLS, int NT>
__global__ __launch_bounds__(NT) void lina_decode_kernel(const LinaDecodeArgs a) {
  constexpr int NW = NT / 64;
  constexpr int TPR = COLS / 4;   // threads of a row
  constexpr int RG = NT / TPR;    // rows at a time
  constexpr int RPT = DK / RG;    // rows of a thread
  constexpr int NTK = 8;          // tokens staged at a time
  static_assert(RPT * RG == DK && RPT >= 1, "tile split");
  __shared__ float s_q[NTK][DK], s_k[NTK][DK], s_v[NTK][COLS], s_a[NTK];
  __shared__ float s_red[2][NW][COLS];

  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int tiles = a.dv / COLS;
  const int64_t bh = blockIdx.x / tiles;
  const int c0 = (int)(blockIdx.x % tiles) * COLS;
  const int64_t b = bh / a.H;
  const int h = (int)(bh % a.H), hk = h / (a.H / a.Hk);
  const int cq = tid % TPR, rg = tid / TPR;

  // streamed once: nontemporal, so that nothing that will be reused is displaced
  f32x4_t* S = (f32x4_t*)(a.state + (size_t)bh * DK * a.dv + c0);
  const int rs = a.dv / 4;
  f32x4_t s[RPT];
#pragma unroll
  for (int i = 0; i < RPT; ++i) s[i] = __builtin_nontemporal_load(&S[(size_t)(rg + RG * i) * rs + cq]);

  for (int t0 = 0; t0 < a.ntok; t0 += NTK) {
    const int nb = min(NTK, a.ntok - t0);
    if (t0 > 0) __syncthreads();  // the previous tokens' inputs are consumed
    for (int x = tid; x < nb * DK; x += NT) {
      const int j = x / DK, c = x % DK;
      const size_t row = ((size_t)b * a.ntok + t0 + j) * a.Hk + hk;
      s_q[j][c] = Elem<T>::load(a.q, row * DK + c);
      s_k[j][c] = Elem<T>::load(a.k, row * DK + c);
    }
    for (int x = tid; x < nb * COLS; x += NT) {
      const int j = x / COLS, c = x % COLS;
      s_v[j][c] = Elem<T>::load(a.v, (((size_t)b * a.ntok + t0 + j) * a.H + h) * a.dv + c0 + c);
    }
    if (tid < nb) s_a[tid] = expf(a.g_fixed ? a.g[h] : a.g[((size_t)b * a.ntok + t0 + tid) * a.H + h]);
    __syncthreads();

    for (int j = 0; j < nb; ++j) {
      const int par = (t0 + j) & 1;  // two buffers: one barrier a token
      const float dec = s_a[j];
      const float4 v = *(const float4*)&s_v[j][4 * cq];
      float p[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int i = 0; i < RPT; ++i) {
        const int r = rg + RG * i;
        const float kk = s_k[j][r], qq = s_q[j][r];
        s[i][0] = fmaf(s[i][0], dec, kk * v.x);
        s[i][1] = fmaf(s[i][1], dec, kk * v.y);
        s[i][2] = fmaf(s[i][2], dec, kk * v.z);
        s[i][3] = fmaf(s[i][3], dec, kk * v.w);
#pragma unroll
        for (int x = 0; x < 4; ++x) p[x] = fmaf(qq, s[i][x], p[x]);
      }
#pragma unroll
      for (int off = TPR; off < 64; off <<= 1)
#pragma unroll
        for (int x = 0; x < 4; ++x) p[x] += __shfl_xor(p[x], off);
      if (lane < TPR) *(float4*)&s_red[par][wave][4 * cq] = make_float4(p[0], p[1], p[2], p[3]);
      __syncthreads();
      if (tid < COLS) {
        float o = 0.f;
#pragma unroll
        for (int w = 0; w < NW; ++w) o += s_red[par][w][tid];
        Elem<T>::store(a.o, (((size_t)b * a.ntok + t0 + j) * a.H + h) * a.dv + c0 + tid, o);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < RPT; ++i) __builtin_nontemporal_store(s[i], &S[(size_t)(rg + RG * i) * rs + cq]);
}

// 64 columns a workgroup; 512 threads where the states come from memory, 256 where they are few
// enough to stay in the caches (H = 32, d = 128, per step: 180 us against 189 at B = 256, 46.7
// against 47.4 at 64, but 12.7 against 10.9 at 16 and 4.7 against 4.5 at 4).  180 us are 6.0 TB/s, the
// rate of one buffer updated in place; with another state each time 194 us, 5.6 TB/s.
template <typename T, int DK>
hipError_t launch_d(const LinaDecodeArgs& a) {
  const int64_t blocks = a.BH * (a.dv / 64);
  if (blocks > 0x7FFFFFFF) return hipErrorInvalidValue;
  if (blocks >= 4096)
    hipLaunchKernelGGL((lina_decode_kernel<T, DK, 64, 512>), dim3((unsigned)blocks), dim3(512), 0,
                       (hipStream_t)a.stream, a);
  else
    hipLaunchKernelGGL((lina_decode_kernel<T, DK, 64, 256>), dim3((unsigned)blocks), dim3(256), 0,
                       (hipStream_t)a.stream, a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_lina_decode(const LinaDecodeArgs& a) {
  if (a.BH == 0) return hipSuccess;
  if (a.bf16) return a.dk == 128 ? launch_d<bf16_t, 128>(a) : launch_d<bf16_t, 64>(a);
  return a.dk == 128 ? launch_d<float, 128>(a) : launch_d<float, 64>(a);
}

}  // namespace kda
