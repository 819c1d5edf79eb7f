// decode_tree.cu — decode-attention kernel variants for a tree of drafted
// tokens (paged_tree_attention) on bf16, f16 and fp32 caches: the pipeline
// shapes of decode_bf16.cu / decode_f16.cu / decode_f32.cu with the tree's masks.
// They serve fp32 caches, batches beyond the tile kernels' plan, and few rows on many
// items (tree_route in api.cpp): 64 x 500, 32 heads of 4 rows 122 us as the tile kernel, and at D 64
// 16 x 4096, 8 heads of 8 rows 46 us against its 52.  fp32 caches (the reference precision)
// pass over the cache once per two rows: 16 x 2048, 32 / 8 heads, 16 nodes (32 passes) 1.3 ms, 64
// nodes on 64 / 8 heads (256 passes) 10.1 ms, 6.7 TFLOP/s.
#include "decode.cuh"

namespace pkv {

int register_decode_tree(DecodeKernel *out) {
  int n = 0;
  out[n++] = decode_entry<DecodeCfg<BF16, BF16, 128, 8, true, kWarps, kBudget, 1, true>>();
  out[n++] = decode_entry<DecodeCfg<BF16, BF16, 64, 8, true, kWarps, kBudget, 1, true>>();
  out[n++] = decode_entry<DecodeCfg<F16, F16, 128, 8, true, kWarps, kBudget, 1, true>>();
  out[n++] = decode_entry<DecodeCfg<F16, F16, 64, 8, true, kWarps, kBudget, 1, true>>();
  out[n++] = decode_entry<DecodeCfg<F32, F32, 128, 2, false, kWarps, kBudget, 1, true>>();
  out[n++] = decode_entry<DecodeCfg<F32, F32, 64, 2, false, kWarps, kBudget, 1, true>>();
  out[n++] = decode_entry<DecodeCfg<F32, F32, 128, 1, false, kWarps, kBudget, 1, true>>();
  out[n++] = decode_entry<DecodeCfg<F32, F32, 64, 1, false, kWarps, kBudget, 1, true>>();
  return n;
}

}  // namespace pkv
