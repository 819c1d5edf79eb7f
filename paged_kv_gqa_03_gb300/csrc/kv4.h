// kv4.h — launchers of the 4-bit cache's kernels and of the rotary positions
// (kv4_pages.cu, kv4_decode.cu, rope.cu), called by the C-ABI layer.
#pragma once

#include "internal.h"

namespace pkv {

// A tensor's unit: positive and finite.
inline bool kv4_unit_ok(float u) { return u > 0.f && u <= 3.402823466e38f; }

constexpr int kKv4 = 4;  // DecodeKernel::cache_dtype of the 4-bit variants (no public dtype code)

struct Kv4Params {
  DecodeParams d;  // (k_scale, v_scale unused; scale_log2 holds K's unit)
  const uint8_t *cache;
  float v_unit;
};
int register_decode_kv4(DecodeKernel *out);

// Rows of new tokens, `ld` elements apart.
cudaError_t launch_kv4_append(const void *k_new, int64_t ld_k, const void *v_new, int64_t ld_v, int new_dtype,
                              uint8_t *cache, const int64_t *slots, int T, int Hkv, int D, int64_t num_blocks,
                              float k_unit, float v_unit, cudaStream_t stream);
// 16-bit (or fp32) blocks src of k / v -> 4-bit blocks dst, and back.
cudaError_t launch_kv4_pack(uint8_t *cache, int64_t num_blocks, const void *k, const void *v, int dtype,
                            int64_t num_src, const int32_t *pairs, int n, int Hkv, int D, float k_unit, float v_unit,
                            cudaStream_t stream);
cudaError_t launch_kv4_expand(void *k, void *v, int dtype, int64_t num_dst, const uint8_t *cache, int64_t num_blocks,
                              const int32_t *pairs, int n, int Hkv, int D, float k_unit, float v_unit,
                              cudaStream_t stream);
cudaError_t launch_kv4_copy(uint8_t *cache, const int32_t *pairs, int n, size_t block_bytes, int64_t num_blocks,
                            cudaStream_t stream);

// Rotary positions (rope.cu).
struct RopeParams {
  const void *q, *k, *v;
  void *q_out, *k_out;         // k_out: null when the keys go to a cache
  int64_t ld_q, ld_k, ld_v, ld_q_out, ld_k_out;  // elements from a token to the next
  void *k_cache, *v_cache;     // caches of the rows' type, or null
  uint8_t *kv4;                // a 4-bit cache, or null
  const uint64_t *turns;       // [rot / 2] turns a position, in 2^-64
  const int64_t *positions, *slots;
  int64_t num_blocks;
  int T, Hq, Hkv, D, rot, interleaved;
  float magnitude, k_unit, v_unit;
};
cudaError_t launch_rope(const RopeParams &p, int dtype, cudaStream_t stream);

}  // namespace pkv
