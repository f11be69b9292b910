// kda_lina.h -- arguments of the linear-attention kernels (decay per head), shared by the
// C ABI (kda_lina_api.cpp) and the launchers (kda_lina.hip, kda_lina_decode.hip).
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace kda {

// An operand of a walk: [rows, heads, dim] with head h of H mapped to h / (H / heads).
struct LinaOp {
  const void* p = nullptr;
  int heads = 0;
};

enum LinaDot : int { kDotNone = 0, kDotRow = 1, kDotCross = 2 };

// One walk  out_i = sum_{j <= i} r_ij (Q_i . K_j) V_j  (+ the start state's part), tokens in
// order or (rev) in reverse order.
struct LinaWalk {
  LinaOp q, k, v, x;      // x: what the walk's dots are taken with (dot != kDotNone)
  void* out = nullptr;    // [rows, H, dv], element type of q, or fp32 when out_f32
  bool out_f32 = false;
  const float* g = nullptr;
  bool g_fixed = false;   // g is [H] instead of [rows, H]
  const float* s0 = nullptr;  // [n, H, dk, dv] (s_t: [n, H, dv, dk]) or NULL
  float* sT = nullptr;
  bool s_t = false;
  bool rev = false;
  int dot = kDotNone;
  float* dots = nullptr;      // [dv / 64][H][rows] fp32
  float* snap = nullptr;      // states every lina_keep() chunks but the first (forward walk with kDotRow writes them)
  const float* snap0 = nullptr;  // reverse walk with kDotRow: the first, the caller's [n, H, dv, dk], or NULL for zeros
  float* anchor = nullptr;    // [groups][H][dv / 64][4] (reverse walk with kDotRow: <snap, state>)
  float* seg_state = nullptr; // end states [lina_ends][H][dv / 64][dk * 64], then kept start states
  float* seg_dec = nullptr;   // [lina_ends][H]
  // batch
  const int* cs = nullptr;    // clamped offsets of a packed batch [n + 1] and its chunks of a segment, or NULL
  const int* list = nullptr;  // its segments in the order they are dealt, [slots][2]
  int n = 0;                  // sequences
  int T = 0;                  // tokens of each sequence (packed: of the batch)
  int H = 0, dk = 0, dv = 0;  // the walk's own widths: Q, K have dk channels, V, out dv
  int L = 0;                  // chunks of a segment (packed: the least)
  bool split = false;         // segments are walked apart (L < the longest chain)
  bool replay = false;        // forward: a segment's state from all chunks before it, by itself
  bool bf16 = true;
  void* stream = nullptr;
};

constexpr int kLinaGroup = 16;  // chunks whose decay gradients one workgroup adds up
// Chunks between two kept states of the backward (a divisor of kLinaGroup): D's error grows with the tokens
// that it passes by differences.  Decay gradient off by, of its norm: fp32, 1,100 tokens, d = 128: 1.1e-6 at 16
// chunks, 2.8e-7 at 4, 2.6e-7 at 1 (91, 92 and 94 us); bf16, 20 calls of 1,024 to 2,048 tokens, the worst 7.9e-7
// at 16, 6.9e-7 at 8, 5.6e-7 at 4 (B4 H32 T8K: 1069, 1067 and 1104 us).
constexpr int lina_keep(bool bf16) { return bf16 ? 8 : 4; }

// most threads of a workgroup: walks, the decay gradient's sums, decode
constexpr int kLinaThreads = 768, kLinaDecayThreads = 64 * kLinaGroup, kLinaDecodeThreads = 512;

// Segments (or groups of `per` chunks) of a batch: sequence i starts at
// offset / (64 per) + i, so that every sequence has at least one.
inline int64_t lina_pieces(int64_t rows, int64_t n, int64_t per) { return rows / (64 * per) + n; }

// Segments from whose end another one starts.  A packed sequence that starts at `offset` has at most
// (its rows - 1) / (64 L) of them, from slot offset / (64 L) on, so that no sequence reaches the next
// one's and a batch of many short ones needs none.
inline int64_t lina_ends(bool packed, int64_t T, int64_t n, int64_t L) {
  const int64_t nch = T > 0 ? (T + 63) / 64 : 1;
  return packed ? T / (64 * L) : n * ((nch + L - 1) / L - 1);
}
// States that a cut batch keeps in all: those ends, and the start state of each cut sequence (fewer than ends).
inline int64_t lina_seg_states(int64_t ends, int64_t n) { return ends + (ends < n ? ends : n); }

// up to three walks of one call: the end states of their segments, where they are split
hipError_t launch_lina_segments(const LinaWalk* w, int n);
hipError_t launch_lina_walk(const LinaWalk& w);
// dq's and dv's walk in one launch: fp32
hipError_t launch_lina_pair(const LinaWalk& wq, const LinaWalk& wv);
// dk's and dv's walk in one kernel: bf16, widths equal; wv.x: v
hipError_t launch_lina_reverse(const LinaWalk& wk, const LinaWalk& wv);
// chains: of a sequence; a batch is cut where its longest chain is over 256 / cut shares of all steps; link: tenths of what
// both walks of a chunk take that joining two segments does, where they are joined one after another (0: they are not)
hipError_t launch_lina_offsets(const int* cu, int n, int T, int L, int chains, int* cs, int* list, void* stream,
                               int cut = 160, int link = 0);
hipError_t launch_lina_headsum(const float* part, void* out, int64_t rows, int heads, int group, int d, bool bf16,
                               const int* end, void* stream);
hipError_t launch_lina_ddecay(const LinaWalk& w, const float* a, const float* b, const float* e, int na, int ne,
                              const float* anchor, float* dg, double* part, float* dg_fixed);

struct LinaDecodeArgs {
  const void *q, *k, *v;
  const float* g;
  bool g_fixed;
  float* state;
  void* o;
  int64_t BH;
  int ntok, H, Hk, dk, dv;
  bool bf16;
  void* stream;
};
hipError_t launch_lina_decode(const LinaDecodeArgs& a);

}  // namespace kda
