// tree.h — host side of the verification and commit kernels of a tree of
// drafted tokens (tree_verify.cu, tree_commit.cu).
#pragma once

#include "internal.h"

namespace pkv {

struct VerifyParams {
  int32_t *path, *path_len;   // [B][n], [B]
  int64_t *next_token;        // [B]
  const int64_t *tokens;      // [B][n]
  const uint64_t *mask;       // [B][n], or [n] (mask_stride 0)
  const int32_t *lens;        // [B] nodes, or null: n
  const void *target, *draft; // rows b * n + i of V values; draft null: deterministic drafts
  const float *u;             // [B][n], or null: greedy
  int64_t ld_target, ld_draft;  // elements between rows
  int n, mask_stride, V;
};
cudaError_t launch_tree_verify(const VerifyParams &p, int dtype, int B, int sms, cudaStream_t stream);

struct CommitParams {
  uint8_t *k_cache, *v_cache;
  float *k_scale, *v_scale;         // fp8 caches, else null; written by calibrated calls alone
  const int32_t *path, *path_len;   // [B][n], [B]
  const int32_t *block_table, *context_lens, *tree_lens;
  int32_t *new_lens;                // [B] or null
  int64_t num_blocks;
  int B, n, Hkv, max_blocks, row_bytes;
  int calibrated;                   // fp8: block scales follow the rows moved in
};
cudaError_t launch_tree_commit(const CommitParams &p, cudaStream_t stream);

}  // namespace pkv
