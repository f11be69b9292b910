// kda_verify.hip -- which drafted tokens stand against the target's probabilities, and the token after them,
// from given random numbers.
//
// Draft x_i stands while u_i q_i(x_i) < p_i(x_i).  After n of them the next token is drawn from
// max(p_n - q_n, 0) where a draft was refused, from p_n where none was left: the lowest index whose running
// sum passes u_next times the whole.  All of it in fp64, so that only a u_next within about 1e-13 of a border
// between two indices could tell two orders of summation apart.
//
// Only row n of p and q is read whole, in tiles of 2,048 tokens: the first kernel sums each tile (weights, and p's
// own, for where the weights are all zero), the second finds the tile and the token in it.  What both wait for is one
// access to memory after another: the drafts, their probabilities, the row; so a workgroup of the first goes through several
// tiles of a row once it knows which.  128 sequences over 131,072 tokens, fp32 (105 MB: p of all, q of the 54%
// that had a draft refused): 30 us, 3.5 TB/s, and 9 for the second kernel, 33.7 together; with every one refused (134 MB) 38.7:
// further bytes go at 5.8 TB/s, the rest is those accesses and the second kernel.  Drafts chosen outright (67 MB) 30.0; bf16
// rows (52 MB) 55.6, because a guarded load and its widening stand together, so that a thread's loads wait for each other (36 waits in the
// kernel's code, fp32 has 5).  A single sequence 5 and 9, latency.  Tiles of 4,096 tokens were slower.
#include <math.h>

#include "kda_common.h"
#include "kda_verify.h"

namespace kda {

namespace {

constexpr int NT = 256;
constexpr int PER = kVerifyTile / NT;  // tokens of a thread

// what a probability weighs: nothing where it is negative or not finite
__device__ __forceinline__ double weight(float x) { return x > 0.f && x < __builtin_inff() ? (double)x : 0.; }

// A sequence's row: how many drafts stand, and what its next token is drawn from.
struct Row {
  int n;         // drafts that stand
  int refused;   // the draft that does not, or -1 (no draft there)
  size_t p, q;   // its row's first entries
};

template <typename T>
__device__ __forceinline__ Row find_row(const VerifyArgs& a, int64_t b) {
  // one wave looks at 64 drafts at a time; every wave does the same
  const int lane = threadIdx.x & 63;
  Row r;
  r.n = a.K;
  r.refused = -1;
  for (int i0 = 0; i0 < a.K; i0 += 64) {
    const int i = i0 + lane;
    bool stops = false;
    int x = -1;
    if (i < a.K) {
      x = a.drafts[b * a.K + i];
      const bool real = x >= 0 && x < a.V;
      double p = 0., q = 1.;
      if (real) {
        p = (double)Elem<T>::load(a.p, ((size_t)b * (a.K + 1) + i) * a.V + x);
        if (a.q) q = (double)Elem<T>::load(a.q, ((size_t)b * a.K + i) * a.V + x);
      }
      stops = !(real && (double)a.u[b * a.K + i] * q < p);
      if (!real) x = -1;
    }
    const uint64_t m = __ballot(stops);
    if (m) {
      const int first = __ffsll((unsigned long long)m) - 1;
      r.n = i0 + first;
      r.refused = __shfl(x, first);
      break;
    }
  }
  return r;
}

__device__ __forceinline__ void place_row(const VerifyArgs& a, int64_t b, Row& r) {
  r.p = ((size_t)b * (a.K + 1) + r.n) * a.V;
  r.q = ((size_t)b * a.K + min(r.n, max(a.K - 1, 0))) * a.V;
}

// the two weights of token j with probabilities p and q: after a refusal, and the target's own
__device__ __forceinline__ void weights(const VerifyArgs& a, const Row& r, int j, float p, float q, double& rest, double& own) {
  own = weight(p);
  rest = own;
  if (r.refused >= 0) {
    const double less = a.q ? weight(q) : j == r.refused ? 1. : 0.;
    rest = own > less ? own - less : 0.;
  }
}

template <typename T>
__global__ __launch_bounds__(NT) void verify_sum_kernel(const VerifyArgs a) {
  __shared__ double part[2][2][NT / 64];
  const int tid = threadIdx.x;
  const int64_t b = blockIdx.x / a.groups;
  const int first = (int)(blockIdx.x % a.groups);
  Row r = find_row<T>(a, b);
  place_row(a, b, r);
  if (first == 0 && tid == 0) {
    a.rows[2 * b] = r.n;
    a.rows[2 * b + 1] = r.refused;
  }
  const bool both = a.q && r.refused >= 0;
  float p[PER], q[PER];
  auto fetch = [&](int tile) {
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int64_t j = (int64_t)tile * kVerifyTile + i * NT + tid;
      p[i] = j < a.V ? Elem<T>::load(a.p, r.p + j) : 0.f;
      q[i] = both && j < a.V ? Elem<T>::load(a.q, r.q + j) : 0.f;
    }
  };
  fetch(first);
  int par = 0;
  for (int tile = first; tile < a.tiles; tile += a.groups, par ^= 1) {
    double rest = 0., own = 0.;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      double x, y;
      weights(a, r, tile * kVerifyTile + i * NT + tid, p[i], q[i], x, y);
      rest += x;
      own += y;
    }
    if (tile + a.groups < a.tiles) fetch(tile + a.groups);
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
      rest += __shfl_xor(rest, off);
      own += __shfl_xor(own, off);
    }
    if ((tid & 63) == 0) {
      part[par][0][tid >> 6] = rest;
      part[par][1][tid >> 6] = own;
    }
    __syncthreads();  // two buffers: one barrier a tile
    if (tid < 2) {
      double x = 0.;
      for (int i = 0; i < NT / 64; ++i) x += part[par][tid][i];
      a.sums[((size_t)b * a.tiles + tile) * 2 + tid] = x;
    }
  }
}

template <typename T>
__global__ __launch_bounds__(NT) void verify_pick_kernel(const VerifyArgs a) {
  __shared__ double run[NT / 64];
  __shared__ int found, last;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int64_t b = blockIdx.x;
  Row r;
  r.n = a.rows[2 * b];
  r.refused = a.rows[2 * b + 1];
  place_row(a, b, r);
  const double* sums = a.sums + (size_t)b * a.tiles * 2;
  if (tid == 0) {
    found = 0x7FFFFFFF;
    last = -1;
    a.accepted[b] = r.n;
  }
  // every wave: the whole, then the tile that passes the target (or the last one that weighs anything)
  double total = 0., own = 0.;
  for (int t = lane; t < a.tiles; t += 64) {
    total += sums[2 * t];
    own += sums[2 * t + 1];
  }
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) {
    total += __shfl_xor(total, off);
    own += __shfl_xor(own, off);
  }
  const bool rest = total > 0.;
  if (!rest) total = own;
  const double target = (double)a.u_next[b] * total;
  int tile = -1, some = -1;
  double before = 0., carry = 0., some_before = 0.;
  for (int t0 = 0; t0 < a.tiles && tile < 0; t0 += 64) {
    const int t = t0 + lane;
    const double s = t < a.tiles ? sums[2 * t + (rest ? 0 : 1)] : 0.;
    double x = s;
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
      const double y = __shfl_up(x, off);
      if (lane >= off) x += y;
    }
    const double start = carry + (x - s);
    const uint64_t over = __ballot(s > 0. && carry + x > target), any = __ballot(s > 0.);
    if (over) {
      const int f = __ffsll((unsigned long long)over) - 1;
      tile = t0 + f;
      before = __shfl(start, f);
    }
    if (any) {
      const int f = 63 - __clzll((unsigned long long)any);
      some = t0 + f;
      some_before = __shfl(start, f);
    }
    carry += __shfl(x, 63);
  }
  if (tile < 0) {
    tile = some;
    before = some_before;
  }
  if (tile < 0) {  // nothing to draw from
    if (tid == 0) a.next[b] = -1;
    return;
  }
  double w[PER], sum = 0.;
  const int j0 = tile * kVerifyTile + tid * PER;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    double x = 0., y = 0.;
    if (j0 + i < a.V)
      weights(a, r, j0 + i, Elem<T>::load(a.p, r.p + j0 + i), a.q && r.refused >= 0 ? Elem<T>::load(a.q, r.q + j0 + i) : 0.f, x, y);
    w[i] = rest ? x : y;
    sum += w[i];
  }
  double x = sum;
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) {
    const double y = __shfl_up(x, off);
    if (lane >= off) x += y;
  }
  if (lane == 63) run[wave] = x;
  __syncthreads();
  double at = before + (x - sum);
  for (int i = 0; i < wave; ++i) at += run[i];
  int first = 0x7FFFFFFF, mine = -1;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    at += w[i];
    if (w[i] > 0.) {
      if (at > target && first == 0x7FFFFFFF) first = j0 + i;
      mine = j0 + i;
    }
  }
  if (first != 0x7FFFFFFF) atomicMin(&found, first);
  if (mine >= 0) atomicMax(&last, mine);
  __syncthreads();
  if (tid == 0) a.next[b] = found != 0x7FFFFFFF ? found : last;
}

template <typename T>
hipError_t verify(const VerifyArgs& a) {
  const int64_t blocks = (int64_t)a.B * a.groups;
  if (blocks > 0xFFFFFFFFll / NT) return hipErrorInvalidValue;
  hipLaunchKernelGGL(verify_sum_kernel<T>, dim3((unsigned)blocks), dim3(NT), 0, (hipStream_t)a.stream, a);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(verify_pick_kernel<T>, dim3((unsigned)a.B), dim3(NT), 0, (hipStream_t)a.stream, a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_verify(const VerifyArgs& a) { return a.bf16 ? verify<bf16_t>(a) : verify<float>(a); }

}  // namespace kda
