// kv4.h — launchers of the 4-bit cache's kernels and of the rotary positions
// (kv4_pages.cu, kv4_decode.cu, rope.cu), called by the C-ABI layer.
#pragma once

#include "internal.h"

namespace pkv {

// A tensor's unit.  (Within 2^+-64 what is multiplied and divided by it stays within fp32's normal numbers: a
// unit over a softmax's sum of up to 2^46, code * scale * unit.  The scores' factor, k_unit times the softmax scale times a
// query row's power of two, may leave them: the decode kernel bounds it.)
inline bool kv4_unit_ok(float u) { return u >= 0x1p-64f && u <= 0x1p64f; }

constexpr int kKv4PageThreads = 128;  // a CTA of kv4_pages.cu

constexpr int kKv4MaxRanges = 224;  // WsHeader::cta_status

// Batches of fewer sequences are planned inside the decode kernel.
constexpr int kKv4Prefix = 512;

// Units of at most this many blocks (alike in bytes) are not cut between CTAs (kv4_decode.cu): 128 x 385-1409 in a step
// 57.5 us, 59.9 with 64; D = 64, 32 x 512-4096 with a window of 1024 (65 blocks) 33.3 us, 36.2 with 48.
template <int D>
constexpr int kKv4Whole = D == 64 ? 96 : 48;
inline int kv4_whole(int D) { return D == 64 ? kKv4Whole<64> : kKv4Whole<128>; }

struct Kv4Params {
  DecodeParams d;  // P: ranges, one per CTA; scale_log2 holds K's unit; k_scale, v_scale, cta_flags unused
  const uint8_t *cache;
  int hg, hg_log2;  // heads of a unit (d.HU: units of a sequence = Hkv / hg * d.NC)
  int4 *records;   // [P]: the units that a CTA's range cuts (kv4_decode.cu)
  float *first_o;  // [P][warps][GC][D]: a ring's first segment, to be joined in its CTA
  float v_unit;
  int merge_units, merge_rows;  // the merge kernel's CTAs: by unit or by range, and their rows
};
struct Kv4WsLayout {
  size_t hdr, prefix, starts, records, part_o, part_lse, first_o, total;
};
Kv4WsLayout kv4_ws_layout(int B, int P, int D, int GC, int hg, int warps);
// Heads that a unit takes together: neighbours in the cache, read by one copy.
inline int kv4_heads(int Hkv) { return Hkv % 4 == 0 ? 4 : Hkv % 2 == 0 ? 2 : 1; }
// One compiled variant of the decode kernel.
struct Kv4Kernel {
  const void *fn;  // __global__ void (Kv4Params)
  int q_dtype, D, GC;
  int warps;    // consumers
  int threads;  // of a CTA: consumers and producers
  size_t smem_bytes;
};
constexpr int kKv4Kernels = 8;
void register_decode_kv4(Kv4Kernel (&out)[kKv4Kernels]);
// Joins the units cut between CTAs.
cudaError_t launch_kv4_merge(Kv4Params p, cudaStream_t stream, bool pdl);

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
