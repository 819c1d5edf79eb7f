// decode_tree_fp8.cu — decode-attention kernel variants for a tree of drafted
// tokens (paged_tree_attention) on fp8-E4M3 caches: the pipeline shapes of
// decode_fp8.cu with the tree's masks: up to 16 rows per kv head on more than a small
// cache (16 x 8192, 32 / 8 heads, 1 / 2 / 4 nodes 74 / 77 / 90 us, out of a cold L2, against the tile
// kernel's 94).  V's scales go into the exponent and bf16 queries are scaled by row (decode.cuh), so that
// neither leaves f16's range: 1 - 4 % of those times, 7 % at head dim 64 (64 x 4096, 4 nodes 122 us).
#include "decode.cuh"

namespace pkv {

constexpr int kFp8Warps = 4;
constexpr int kFp8WideBudget = 24 * 1024;

int register_decode_tree_fp8(DecodeKernel *out) {
  int n = 0;
  out[n++] = decode_entry<DecodeCfg<E4M3, BF16, 128, 8, true, 6, kBudget, 2, true>>();
  out[n++] = decode_entry<DecodeCfg<E4M3, BF16, 64, 8, true, kFp8Warps, kBudget, 2, true>>();
  out[n++] = decode_entry<DecodeCfg<E4M3, F16, 128, 8, true, 6, kBudget, 2, true>>();
  out[n++] = decode_entry<DecodeCfg<E4M3, F16, 64, 8, true, kFp8Warps, kBudget, 2, true>>();
  out[n++] = decode_entry<DecodeCfg<E4M3, BF16, 128, 16, true, kFp8Warps, kFp8WideBudget, 2, true>>();
  out[n++] = decode_entry<DecodeCfg<E4M3, BF16, 64, 16, true, kFp8Warps, kFp8WideBudget, 2, true>>();
  out[n++] = decode_entry<DecodeCfg<E4M3, F16, 128, 16, true, kFp8Warps, kFp8WideBudget, 2, true>>();
  out[n++] = decode_entry<DecodeCfg<E4M3, F16, 64, 16, true, kFp8Warps, kFp8WideBudget, 2, true>>();
  return n;
}

}  // namespace pkv
