// kda_qk.h -- arguments of the query / key preparation kernels (per-head norm and rotation).
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace kda {

// Rows of one tensor: `heads` rows of d channels for each token.
struct QkTensor {
  const void* x = nullptr;   // input, tokens `stride` elements apart
  const void* dy = nullptr;  // backward: gradient of the output, dense
  void* out = nullptr;       // output (backward: gradient of x), dense
  const float* w = nullptr;  // [d] or NULL
  float* dw = nullptr;       // backward: [d] or NULL
  int heads = 0;
  int64_t stride = 0;
};

struct QkArgs {
  QkTensor q, k;
  int64_t tokens = 0;
  int d = 0;
  int norm = 0;  // 0 none, 1 rms, 2 l2
  float eps = 0.f, w_offset = 0.f;
  int rotary = 0;  // rotated channels (0: none)
  bool interleaved = false;
  int axes = 0;
  int ends[4] = {0, 0, 0, 0};  // frequency index at which each axis ends
  const double* inv = nullptr;  // [rotary / 2]
  const void* pos = nullptr;    // [axes][tokens], int32 or int64
  bool pos64 = false;
  bool bf16 = true;
  float* partial = nullptr;  // backward: [blocks][2][d] weight gradients
  void* stream = nullptr;
};

constexpr int kQkMaxBlocks = 2048;  // of a backward that sums weight gradients

hipError_t launch_qk(const QkArgs& a);
hipError_t launch_qk_bwd(const QkArgs& a);

}  // namespace kda
