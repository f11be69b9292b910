// kda_verify.h -- arguments of the drafted tokens' verification, shared by its C ABI
// (kda_verify_api.cpp) and its kernels (kda_verify.hip).
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace kda {

constexpr int kVerifyTile = 2048;  // tokens of a tile

struct VerifyArgs {
  int B, K, V, tiles;
  const void *p, *q;     // [B, K + 1, V] and [B, K, V], or NULL
  const int* drafts;     // [B, K]
  const float *u, *u_next;
  int *accepted, *next;  // [B]
  double* sums;          // [B][tiles][2]
  int* rows;             // [B][2]: drafts that stand, and the one that does not
  int groups;            // workgroups of a sequence
  bool bf16;
  void* stream;
};
hipError_t launch_verify(const VerifyArgs& a);

}  // namespace kda
