// kda_gdr.h -- arguments of the kernels of the gated delta rule with one decay per head, shared by
// the C ABI (kda_gdr_api.cpp) and the launchers (kda_gdr.hip, kda_gdr_bwd.hip, kda_gdr_decode.hip).
#pragma once
#include "kda_lina.h"

namespace kda {

// One call's batch and buffers.  walk: batch, operands, widths, segments and states as linear
// attention has them (walk.q, walk.k rows of q and k, walk.v of v or, in reverse, of d_o).
struct GdrWalk {
  LinaWalk walk;
  const void* beta = nullptr;   // [rows, H], element type of q
  float* inv = nullptr;         // [chunks][H][kTriBlocks * 256]: (I + A diag(beta))^-1 of each chunk
  float* score = nullptr;       // the same of P
  float* token = nullptr;       // [chunks][H][kTokenFloats]: decays and strengths of each chunk's tokens
  float* transfer = nullptr;    // segments: [lina_ends][H][dk / 64][dk * 64], laid out as seg_state
  bool train = false;           // the backward's forward: leaves r, the chunks' states and do . o
  void* kept = nullptr;         // [chunks][H][dv / 64][64][dk]: the state each chunk meets, element type of q
  LinaOp r;                     // reverse: what the forward left; its rows meet z
  float* dots2 = nullptr;       // reverse: z . r, [dv / 64][H][rows]
};

constexpr int kTokenFloats = 3 * 64 + 4;
constexpr int kTriBlocks = 10;  // 16 x 16 blocks of a chunk's lower triangle

// chunks of a batch, as lina_pieces(.., 1) counts them
inline int64_t gdr_chunks(bool packed, int64_t T, int64_t n) { return packed ? lina_pieces(T, n, 1) : n * ((T + 63) / 64); }

hipError_t launch_gdr_prep(const GdrWalk& a);
hipError_t launch_gdr_segments(const GdrWalk& a);  // where a.walk.split: end states, transfers, then start states
hipError_t launch_gdr_walk(const GdrWalk& a);

// dq, dk and dbeta of every chunk from what the two walks left
struct GdrGrad {
  GdrWalk f;                   // the forward: q, k, beta, kept, and r in walk.out
  LinaOp d_o, y;               // y: dv
  const void* kept_r = nullptr;
  const float* dots2 = nullptr;
  void *dq = nullptr, *dk = nullptr, *dbeta = nullptr;
};
hipError_t launch_gdr_grad(const GdrGrad& a);

struct GdrDecodeArgs {
  const void *q, *k, *v;       // q NULL: no outputs
  const float* g;
  const void* beta;
  float* state;
  const int* counts;           // [B] tokens of each sequence that count, or NULL for all
  bool update;                 // the state is written back
  void* o;
  int64_t BH;
  int ntok, H, Hk, dk, dv;
  bool bf16;
  void* stream;
};
hipError_t launch_gdr_decode(const GdrDecodeArgs& a);

}  // namespace kda
