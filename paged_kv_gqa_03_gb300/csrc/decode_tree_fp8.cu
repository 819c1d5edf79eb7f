// decode_tree_fp8.cu — decode-attention kernel variants for a tree of drafted
// tokens (paged_tree_attention) on fp8-E4M3 caches: the pipeline shapes of
// decode_fp8.cu with the tree's masks: up to 16 rows per kv head on more than a small
// cache (16 x 8192, 32 / 8 heads, 1 / 2 / 4 nodes 62 / 65 / 81 us against the tile kernel's 93).
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
