// kda_verify_api.cpp -- C ABI of the drafted tokens' verification (include/kda.h, kda_verify_drafts).
#include <stddef.h>
#include <stdint.h>

#include "../../include/kda.h"
#include "kda_check.h"
#include "kda_verify.h"

namespace {

int check_sizes(int B, int K, int V, int dtype) {
  if (dtype != KDA_BF16 && dtype != KDA_F32) return KDA_ERR_DTYPE;
  // up to 2^30 the kernels' K + 1 and their 64 drafts at a time stay in 32 bits
  if (B < 0 || K < 0 || K > (1 << 30) || V < 1 || V > (1 << 30)) return KDA_ERR_SHAPE;
  const int64_t tiles = (V + (int64_t)kda::kVerifyTile - 1) / kda::kVerifyTile, rows = (int64_t)B * ((int64_t)K + 1);
  // probabilities: up to 2^59 of them, 2^61 bytes
  return (int64_t)B * tiles > 0xFFFFFFFFll / 256 || rows > (int64_t(1) << 31) || rows > (int64_t(1) << 59) / V ? KDA_ERR_SHAPE
                                                                                                            : KDA_OK;
}

}  // namespace

extern "C" {

size_t kda_verify_drafts_workspace_size(int B, int K, int V, int dtype) {
  if (check_sizes(B, K, V, dtype) != KDA_OK) return 0;
  return (size_t)B * (((V + (size_t)kda::kVerifyTile - 1) / kda::kVerifyTile) * 16 + 8);
}

int kda_verify_drafts(int B, int K, int V, int dtype, const void* target_probs, const int* drafts,
                      const void* draft_probs, const float* u, const float* u_next, int* accepted, int* next_token,
                      void* workspace, size_t workspace_bytes, void* stream) {
  const int rc = check_sizes(B, K, V, dtype);
  if (rc) return rc;
  if (B == 0) return KDA_OK;
  if (!target_probs || (K > 0 && (!drafts || !u)) || !u_next || !accepted || !next_token || !workspace) return KDA_ERR_NULL;
  const unsigned es = dtype == KDA_BF16 ? 2 : 4;
  if (misaligned(target_probs, es) || misaligned(draft_probs, es) || misaligned(drafts, 4) || misaligned(u, 4) ||
      misaligned(u_next, 4) || misaligned(accepted, 4) || misaligned(next_token, 4) || misaligned(workspace, 8))
    return KDA_ERR_ALIGN;
  const size_t need = kda_verify_drafts_workspace_size(B, K, V, dtype);
  if (workspace_bytes < need) return KDA_ERR_WORKSPACE;
  const int64_t n = (int64_t)B * K;
  const Range in[] = {range_of(target_probs, (n + B) * V * es), range_of(draft_probs, draft_probs ? n * V * es : 0),
                      range_of(drafts, drafts ? n * 4 : 0), range_of(u, u ? n * 4 : 0), range_of(u_next, (int64_t)B * 4)};
  const Range out[] = {range_of(accepted, (int64_t)B * 4), range_of(next_token, (int64_t)B * 4),
                       range_of(workspace, (int64_t)need)};
  for (int i = 0; i < 3; ++i) {
    for (const Range& r : in)
      if (overlap(out[i], r)) return KDA_ERR_ALIAS;
    for (int j = i + 1; j < 3; ++j)
      if (overlap(out[i], out[j])) return KDA_ERR_ALIAS;
  }
  const int tiles = (int)((V + (int64_t)kda::kVerifyTile - 1) / kda::kVerifyTile);
  double* sums = (double*)workspace;
  // eight workgroups to a compute unit, if there are so many tiles: 128 rows of 131,072 tokens 33.8 us, two to a unit 38.7, one
  // for each tile 36.7; 512 rows of 32,000 35.5, 40.7 and 38.7; a single row 14.1, 15.1 and 15.0
  const int groups = (int)(B >= 2048 ? 1 : tiles < 2048 / B ? tiles : 2048 / B);
  const kda::VerifyArgs a{B,        K,          V,    tiles, target_probs, draft_probs,       drafts, u, u_next,
                          accepted, next_token, sums, (int*)(sums + (size_t)B * tiles * 2), groups, dtype == KDA_BF16, stream};
  return kda::launch_verify(a) == hipSuccess ? KDA_OK : KDA_ERR_HIP;
}

}  // extern "C"
