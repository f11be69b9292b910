// kda_qk.hip -- per-head norm of queries and keys and their position rotation in one pass,
// forward and backward.
//
//   y = R(theta) (w + w0) o x r,   r = (mean x^2 + eps)^-1/2 (rms), (sum x^2 + eps)^-1/2 (l2), 1
//   theta_c = pos[axis(c)] inv_freq[c] on the channel pairs (c, c + rotary / 2) or, interleaved,
//   (2c, 2c + 1); channels past `rotary` are not turned.
// Backward, with z = R(-theta) dy and u = (w + w0) o z:
//   dw = sum over rows of z o x r,   dx = r (u - x (x . u) r^2 / d)   (l2: without 1 / d).
//
// Bandwidth bound: each row is read once and written once.  D / 8 lanes hold one row, 8
// channels a lane; a lane group stays at one token and goes through its heads, so that the
// angles (8 fp64 products and sine pairs per lane) are made once for all heads of a token.
// 4 x 8,192 tokens, bf16, d = 128: 151 us for 32 + 8 heads (4.5 TB/s; vector units busy 49%), backward
// of 32 + 32 heads 318 us (5.1 TB/s, the rate of a copy).
// The angle's product is fp64, reduced to a fraction of a turn before it is rounded to fp32: at
// position 10^6 an fp32 product would be off by 0.03 radians.
#include "kda_common.h"
#include "kda_qk.h"

namespace kda {

namespace {

constexpr int NT = 256;
// Rows in flight per lane group: 128 bytes a lane.  bf16, 32 + 8 heads of 32,768 tokens: 162 us with
// two or four rows, 152 with eight; backward, 32 + 32 heads: 334 and 324.
template <typename T>
constexpr int kRows = 16 / (int)sizeof(T);

template <typename T>
struct Row8;  // 8 channels of a lane, as stored
template <>
struct Row8<bf16_t> {
  uint32_t w[4];
  __device__ __forceinline__ void load(const void* p, size_t i) {
    const uint4 v = *(const uint4*)((const uint16_t*)p + i);
    w[0] = v.x; w[1] = v.y; w[2] = v.z; w[3] = v.w;
  }
  __device__ __forceinline__ void get(float (&x)[8]) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  }
  static __device__ __forceinline__ void store(void* p, size_t i, const float (&x)[8]) {
    *(uint4*)((uint16_t*)p + i) = make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]),
                                             pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7]));
  }
  static constexpr int kWords = 4;
};
template <>
struct Row8<float> {
  uint32_t w[8];
  __device__ __forceinline__ void load(const void* p, size_t i) {
    const uint4 a = *(const uint4*)((const float*)p + i), b = *(const uint4*)((const float*)p + i + 4);
    w[0] = a.x; w[1] = a.y; w[2] = a.z; w[3] = a.w;
    w[4] = b.x; w[5] = b.y; w[6] = b.z; w[7] = b.w;
  }
  __device__ __forceinline__ void get(float (&x)[8]) const {
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = __uint_as_float(w[i]);
  }
  static __device__ __forceinline__ void store(void* p, size_t i, const float (&x)[8]) {
    *(float4*)((float*)p + i) = make_float4(x[0], x[1], x[2], x[3]);
    *(float4*)((float*)p + i + 4) = make_float4(x[4], x[5], x[6], x[7]);
  }
  static constexpr int kWords = 8;
};

// sum over the G lanes of a row (G = 8 or 16), in every one of them
template <int G>
__device__ __forceinline__ float group_sum(float x) {
#pragma unroll
  for (int off = 1; off < G; off <<= 1) x += __shfl_xor(x, off);
  return x;
}

// A lane's part of the rotation at one token.
template <bool INTER>
struct Turn {
  static constexpr int N = INTER ? 4 : 8;  // frequencies a lane needs
  float c[N], s[N];  // s carries the sign of the lane's half (INTER: of the pair's first channel)
  int partner;       // lane that holds the other half (INTER: unused)
  bool on;           // the lane's channels are turned

  __device__ __forceinline__ void at(const QkArgs& a, int64_t token, int sub, int lane) {
    const int half = a.rotary / 2, c0 = 8 * sub;
    partner = lane;
    bool upper = false;
    on = c0 < a.rotary;
    int f0 = INTER ? c0 / 2 : c0;
    if (!INTER && c0 >= half) {
      upper = true;
      f0 = c0 - half;
    }
    if (!INTER && on) partner = upper ? lane - half / 8 : lane + half / 8;
#pragma unroll
    for (int e = 0; e < N; ++e) {
      c[e] = 1.f;
      s[e] = 0.f;
      if (on) {
        const int f = f0 + e;
        const int ax = (f >= a.ends[0]) + (f >= a.ends[1]) + (f >= a.ends[2]);
        const size_t i = (size_t)ax * a.tokens + token;
        const double p = a.pos64 ? (double)((const int64_t*)a.pos)[i] : (double)((const int*)a.pos)[i];
        const double t = p * a.inv[f] * 0.15915494309189535;  // turns
        const float fr = (float)(t - rint(t));
        float sn, cs;
        sincospif(2.f * fr, &sn, &cs);
        c[e] = cs;
        s[e] = upper ? sn : -sn;
      }
    }
  }
  // y = R x (sign 1) or R^T x (sign -1); o: the partner lane's values
  __device__ __forceinline__ void apply(const float (&x)[8], const float (&o)[8], float sign, float (&y)[8]) const {
    if (!on) {  // not 0 times the other channel: that may be infinite
#pragma unroll
      for (int e = 0; e < 8; ++e) y[e] = x[e];
    } else if constexpr (INTER) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        y[2 * e] = x[2 * e] * c[e] + sign * s[e] * x[2 * e + 1];
        y[2 * e + 1] = x[2 * e + 1] * c[e] - sign * s[e] * x[2 * e];
      }
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) y[e] = x[e] * c[e] + sign * s[e] * o[e];
    }
  }
};

template <typename T>
__device__ __forceinline__ Row8<T> from_lane(const Row8<T>& r, int lane) {
  Row8<T> o;
#pragma unroll
  for (int i = 0; i < Row8<T>::kWords; ++i) o.w[i] = __shfl((int)r.w[i], lane);
  return o;
}

template <int D>
__device__ __forceinline__ float inv_norm(const QkArgs& a, float ss) {
  if (a.norm == 0) return 1.f;
  return 1.f / sqrtf((a.norm == 1 ? ss * (1.f / D) : ss) + a.eps);
}

__device__ __forceinline__ void weights(const float* w, float off, int c0, float (&x)[8]) {
#pragma unroll
  for (int e = 0; e < 8; ++e) x[e] = w ? w[c0 + e] + off : 1.f;
}

// heads [h0, h1) of one tensor at one token
template <typename T, int D, bool INTER>
__device__ __forceinline__ void heads_fwd(const QkArgs& a, const QkTensor& t, int64_t token, int h0, int h1,
                                          const Turn<INTER>& turn, int sub) {
  constexpr int G = D / 8, HB = kRows<T>;
  if (h0 >= h1) return;
  float w[8], wo[8];
  weights(t.w, a.w_offset, 8 * sub, w);
  if (!INTER) {
    const int ps = turn.partner & (G - 1);
    weights(t.w, a.w_offset, 8 * ps, wo);
  }
  const size_t in = (size_t)token * t.stride + 8 * sub, out = (size_t)token * t.heads * D + 8 * sub;
  for (int h = h0; h < h1; h += HB) {
    Row8<T> r[HB];
#pragma unroll
    for (int j = 0; j < HB; ++j)
      if (h + j < h1) r[j].load(t.x, in + (size_t)(h + j) * D);
#pragma unroll
    for (int j = 0; j < HB; ++j) {
      if (h + j >= h1) break;  // the whole lane group
      float x[8], o[8], y[8];
      r[j].get(x);
      float ss = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) ss = fmaf(x[e], x[e], ss);
      const float rn = inv_norm<D>(a, group_sum<G>(ss));
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] *= rn * w[e];
      if constexpr (!INTER) {
        from_lane(r[j], turn.partner).get(o);
#pragma unroll
        for (int e = 0; e < 8; ++e) o[e] *= rn * wo[e];
      }
      turn.apply(x, o, 1.f, y);
      Row8<T>::store(t.out, out + (size_t)(h + j) * D, y);
    }
  }
}

// grid: (tokens / lane groups, parts of the heads)
template <typename T, int D, bool INTER>
__global__ __launch_bounds__(NT) void qk_kernel(const QkArgs a, int per) {
  constexpr int G = D / 8;
  const int lane = threadIdx.x & 63, sub = threadIdx.x % G;
  const int64_t token = (int64_t)blockIdx.x * (NT / G) + threadIdx.x / G;
  if (token >= a.tokens) return;  // whole lane groups
  const int h0 = blockIdx.y * per, h1 = min(h0 + per, a.q.heads + a.k.heads);
  Turn<INTER> turn;
  turn.at(a, token, sub, lane);
  heads_fwd<T, D, INTER>(a, a.q, token, min(h0, a.q.heads), min(h1, a.q.heads), turn, sub);
  heads_fwd<T, D, INTER>(a, a.k, token, max(h0 - a.q.heads, 0), max(h1 - a.q.heads, 0), turn, sub);
}

template <typename T, int D, bool INTER>
__device__ __forceinline__ void heads_bwd(const QkArgs& a, const QkTensor& t, int64_t token, int h0, int h1,
                                          const Turn<INTER>& turn, int sub, float (&dw)[8]) {
  constexpr int G = D / 8, HB = kRows<T>;
  if (h0 >= h1) return;
  float w[8];
  weights(t.w, a.w_offset, 8 * sub, w);
  const size_t in = (size_t)token * t.stride + 8 * sub, out = (size_t)token * t.heads * D + 8 * sub;
  for (int h = h0; h < h1; h += HB) {
    Row8<T> r[HB], u[HB];
#pragma unroll
    for (int j = 0; j < HB; ++j)
      if (h + j < h1) {
        r[j].load(t.x, in + (size_t)(h + j) * D);
        u[j].load(t.dy, out + (size_t)(h + j) * D);
      }
#pragma unroll
    for (int j = 0; j < HB; ++j) {
      if (h + j >= h1) break;
      float x[8], dy[8], o[8], z[8];
      r[j].get(x);
      u[j].get(dy);
      if constexpr (!INTER) from_lane(u[j], turn.partner).get(o);
      turn.apply(dy, o, -1.f, z);
      float ss = 0.f, xu = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        ss = fmaf(x[e], x[e], ss);
        xu = fmaf(x[e], z[e] * w[e], xu);
      }
      float rn = 1.f, c = 0.f;
      if (a.norm != 0) {
        rn = inv_norm<D>(a, group_sum<G>(ss));
        c = group_sum<G>(xu) * rn * rn;
        if (a.norm == 1) c *= 1.f / D;
      }
      float dx[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        dw[e] = fmaf(z[e], x[e] * rn, dw[e]);
        dx[e] = rn * (z[e] * w[e] - x[e] * c);
      }
      Row8<T>::store(t.out, out + (size_t)(h + j) * D, dx);
    }
  }
}

template <typename T, int D, bool INTER>
__global__ __launch_bounds__(NT) void qk_bwd_kernel(const QkArgs a, int per) {
  constexpr int G = D / 8, GRP = NT / G;
  __shared__ float sum[GRP][D];
  const int lane = threadIdx.x & 63, sub = threadIdx.x % G, grp = threadIdx.x / G;
  const int h0 = blockIdx.y * per, h1 = min(h0 + per, a.q.heads + a.k.heads);
  float dwq[8] = {}, dwk[8] = {};
  for (int64_t t0 = (int64_t)blockIdx.x * GRP; t0 < a.tokens; t0 += (int64_t)gridDim.x * GRP) {
    const int64_t token = t0 + grp;
    if (token < a.tokens) {  // whole lane groups
      Turn<INTER> turn;
      turn.at(a, token, sub, lane);
      heads_bwd<T, D, INTER>(a, a.q, token, min(h0, a.q.heads), min(h1, a.q.heads), turn, sub, dwq);
      heads_bwd<T, D, INTER>(a, a.k, token, max(h0 - a.q.heads, 0), max(h1 - a.q.heads, 0), turn, sub, dwk);
    }
  }
  if (!a.partial) return;
  const size_t block = (size_t)blockIdx.y * gridDim.x + blockIdx.x;
#pragma unroll
  for (int m = 0; m < 2; ++m) {
    __syncthreads();
#pragma unroll
    for (int e = 0; e < 8; ++e) sum[grp][8 * sub + e] = m ? dwk[e] : dwq[e];
    __syncthreads();
    if (threadIdx.x < D) {
      float s = 0.f;
#pragma unroll
      for (int x = 0; x < GRP; ++x) s += sum[x][threadIdx.x];
      a.partial[(block * 2 + m) * D + threadIdx.x] = s;
    }
  }
}

// weight gradients: the blocks' parts in a fixed order, 16 channels by 64 threads each (many
// short columns in flight: with 64 channels by 16 threads this took 57 us at 2,048 blocks)
__global__ __launch_bounds__(1024) void qk_dw_kernel(const float* __restrict__ partial, int blocks, int d,
                                                     float* __restrict__ dwq, float* __restrict__ dwk) {
  __shared__ double s[64][16];
  const int c = threadIdx.x & 15, r = threadIdx.x >> 4;
  const int col = blockIdx.x * 16 + c;  // of 2 d
  double x = 0.;
#pragma unroll 8
  for (int b = r; b < blocks; b += 64) x += partial[(size_t)b * 2 * d + col];
  s[r][c] = x;
  __syncthreads();
  if (r == 0) {
    for (int i = 1; i < 64; ++i) x += s[i][c];
    float* to = col < d ? dwq : dwk;
    if (to) to[col < d ? col : col - d] = (float)x;
  }
}

// Heads of a lane group: all of a token's where there are tokens enough to fill the machine
// (256 compute units, eight workgroups each), fewer where there are not.
int heads_per_group(int64_t token_blocks, int heads) {
  int parts = 1;
  token_blocks = token_blocks < 1 ? 1 : token_blocks;  // parts <= 2,048 = kQkMaxBlocks
  while (token_blocks * parts < 2048 && (heads + parts - 1) / parts > 1) parts *= 2;
  return (heads + parts - 1) / parts;
}

template <typename T, int D, bool INTER>
hipError_t fwd_t(const QkArgs& a) {
  const int64_t tb = (a.tokens + NT / (D / 8) - 1) / (NT / (D / 8));
  if (tb > 0x7FFFFFFF) return hipErrorInvalidValue;
  const int heads = a.q.heads + a.k.heads, per = heads_per_group(tb, heads);
  hipLaunchKernelGGL((qk_kernel<T, D, INTER>), dim3((unsigned)tb, (unsigned)((heads + per - 1) / per)), dim3(NT), 0,
                     (hipStream_t)a.stream, a, per);
  return hipGetLastError();
}

template <typename T, int D, bool INTER>
hipError_t bwd_t(const QkArgs& a) {
  const int64_t tb = (a.tokens + NT / (D / 8) - 1) / (NT / (D / 8));
  const int heads = a.q.heads + a.k.heads;
  const int per = heads_per_group(tb, heads), parts = (heads + per - 1) / per;
  int64_t bx = tb < kQkMaxBlocks / parts ? tb : kQkMaxBlocks / parts;
  if (bx < 1) bx = 1;
  hipLaunchKernelGGL((qk_bwd_kernel<T, D, INTER>), dim3((unsigned)bx, (unsigned)parts), dim3(NT), 0,
                     (hipStream_t)a.stream, a, per);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || !a.partial) return e;
  hipLaunchKernelGGL(qk_dw_kernel, dim3(2 * D / 16), dim3(1024), 0, (hipStream_t)a.stream, a.partial,
                     (int)(bx * parts), D, a.q.dw, a.k.dw);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_qk(const QkArgs& a) {
  if (a.bf16) {
    if (a.d == 128) return a.interleaved ? fwd_t<bf16_t, 128, true>(a) : fwd_t<bf16_t, 128, false>(a);
    return a.interleaved ? fwd_t<bf16_t, 64, true>(a) : fwd_t<bf16_t, 64, false>(a);
  }
  if (a.d == 128) return a.interleaved ? fwd_t<float, 128, true>(a) : fwd_t<float, 128, false>(a);
  return a.interleaved ? fwd_t<float, 64, true>(a) : fwd_t<float, 64, false>(a);
}

hipError_t launch_qk_bwd(const QkArgs& a) {
  if (a.bf16) {
    if (a.d == 128) return a.interleaved ? bwd_t<bf16_t, 128, true>(a) : bwd_t<bf16_t, 128, false>(a);
    return a.interleaved ? bwd_t<bf16_t, 64, true>(a) : bwd_t<bf16_t, 64, false>(a);
  }
  if (a.d == 128) return a.interleaved ? bwd_t<float, 128, true>(a) : bwd_t<float, 128, false>(a);
  return a.interleaved ? bwd_t<float, 64, true>(a) : bwd_t<float, 64, false>(a);
}

}  // namespace kda
