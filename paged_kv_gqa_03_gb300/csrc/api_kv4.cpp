// api_kv4.cpp — the extern "C" boundary of the 4-bit cache's pages and of the
// rotary positions: argument checks and launches (the attention over 4-bit
// pages is in api.cpp, beside the other decode calls).  As there, every check
// runs before the first launch and nothing allocates device memory.
#include <cuda_runtime.h>

#include <cmath>

#include "internal.h"
#include "kv4.h"
#include "pagedkv.h"

using namespace pkv;

namespace {

int status_of(cudaError_t e) {
  if (e == cudaSuccess) return PKV_OK;
  if (e == cudaErrorNotSupported) return PKV_EUNSUPPORTED;  // a count beyond a grid
  record_cuda_error(e);
  return PKV_ECUDA;
}

int row_bytes(int dtype) { return dtype == PKV_F32 ? 4 : (dtype == PKV_F16 || dtype == PKV_BF16 ? 2 : 0); }

bool aligned(const void *p, int64_t ld, int esize) {  // 16-byte aligned rows
  return (reinterpret_cast<uintptr_t>(p) & 15u) == 0 && (ld * esize) % 16 == 0;
}

// Rows of n_a elements, ld_a apart, and rows of n_b share a byte (rows of one buffer's columns, alike in ld, lie
// between one another and need not).
bool overlap(const void *a, int64_t ld_a, int64_t n_a, const void *b, int64_t ld_b, int64_t n_b, int64_t rows,
             int esize) {
  if (!a || !b || rows <= 0) return false;
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  if (x >= y + (uintptr_t)((rows - 1) * ld_b + n_b) * esize || y >= x + (uintptr_t)((rows - 1) * ld_a + n_a) * esize)
    return false;
  if (ld_a != ld_b || rows == 1) return true;
  // b's row j begins d + (j - i) L bytes behind a's row i, which is r or r - L where they can touch
  const int64_t L = ld_a * esize, d = (int64_t)(y - x), r = (d % L + L) % L, k = (r - d) / L;
  auto there = [&](int64_t steps) { return steps > -rows && steps < rows; };
  return (there(k) && r < n_a * esize) || (there(k - 1) && r - L > -n_b * esize);
}

// What the calls on 4-bit pages check alike.
int check_pages(int dtype, int Hkv, int D, int64_t num_blocks, float k_unit, float v_unit) {
  if (Hkv <= 0 || num_blocks <= 0 || !kv4_unit_ok(k_unit) || !kv4_unit_ok(v_unit)) return PKV_EINVAL;
  if (dtype == PKV_FP8_E4M3) return PKV_EUNSUPPORTED;
  if (row_bytes(dtype) == 0) return PKV_EINVAL;
  if (D != 64 && D != 128) return PKV_EUNSUPPORTED;
  return PKV_OK;
}

constexpr double kGrid = 2147483000.0 * kKv4PageThreads;  // threads of a grid

int check_rope(const RopeParams &p, int dtype) {
  if (p.T < 0 || p.Hq < 0 || p.Hkv < 0 || p.Hq + p.Hkv == 0 || p.rot <= 0) return PKV_EINVAL;
  if (dtype == PKV_FP8_E4M3) return PKV_EUNSUPPORTED;
  if (row_bytes(dtype) == 0 || !std::isfinite(p.magnitude)) return PKV_EINVAL;
  if (p.interleaved != 0 && p.interleaved != 1) return PKV_EINVAL;
  if (p.D != 64 && p.D != 128) return PKV_EUNSUPPORTED;
  if (p.rot > p.D) return PKV_EINVAL;
  if (p.rot % 16 != 0) return PKV_EUNSUPPORTED;
  if ((double)p.T * ((double)p.Hq + 2.0 * p.Hkv) * p.D >= kGrid) return PKV_EUNSUPPORTED;
  return PKV_OK;
}

// Rows of `heads` heads: strides at least a row, 16-byte aligned.
bool rows_ok(const void *p, int64_t ld, int heads, int D, int esize) {
  return heads == 0 || (p && ld >= (int64_t)heads * D && aligned(p, ld, esize));
}

}  // namespace

extern "C" {

int64_t paged_kv4_tile_bytes(int D) { return D == 64 || D == 128 ? 18 * D : 0; }

int paged_kv4_append(const void *k_new, int64_t ld_k, const void *v_new, int64_t ld_v, int new_dtype, void *cache,
                     const int64_t *slot_mapping, int T, int Hkv, int D, int64_t num_blocks, float k_unit,
                     float v_unit, pkv_stream_t stream) {
  if (T < 0) return PKV_EINVAL;
  const int rc = check_pages(new_dtype, Hkv, D, num_blocks, k_unit, v_unit);
  if (rc != PKV_OK) return rc;
  if ((double)T * Hkv * 2 * (D / 16) >= kGrid) return PKV_EUNSUPPORTED;
  if (T == 0) return PKV_OK;
  const int es = row_bytes(new_dtype);
  if (!cache || !slot_mapping || !aligned(cache, 0, 1)) return PKV_EINVAL;
  if (!rows_ok(k_new, ld_k, Hkv, D, es) || !rows_ok(v_new, ld_v, Hkv, D, es)) return PKV_EINVAL;
  return status_of(launch_kv4_append(k_new, ld_k, v_new, ld_v, new_dtype, static_cast<uint8_t *>(cache), slot_mapping,
                                     T, Hkv, D, num_blocks, k_unit, v_unit, reinterpret_cast<cudaStream_t>(stream)));
}

int paged_kv4_pack_blocks(void *cache, int64_t num_blocks, const void *k_cache, const void *v_cache, int dtype,
                          int64_t num_src_blocks, const int32_t *src_dst_pairs, int n_pairs, int Hkv, int D,
                          float k_unit, float v_unit, pkv_stream_t stream) {
  if (n_pairs < 0 || num_src_blocks <= 0) return PKV_EINVAL;
  const int rc = check_pages(dtype, Hkv, D, num_blocks, k_unit, v_unit);
  if (rc != PKV_OK) return rc;
  if ((double)n_pairs * Hkv * 2 * D >= kGrid) return PKV_EUNSUPPORTED;
  if (n_pairs == 0) return PKV_OK;
  if (!cache || !k_cache || !v_cache || !src_dst_pairs) return PKV_EINVAL;
  if (!aligned(cache, 0, 1) || !aligned(k_cache, 0, 1) || !aligned(v_cache, 0, 1)) return PKV_EINVAL;
  return status_of(launch_kv4_pack(static_cast<uint8_t *>(cache), num_blocks, k_cache, v_cache, dtype, num_src_blocks,
                                   src_dst_pairs, n_pairs, Hkv, D, k_unit, v_unit,
                                   reinterpret_cast<cudaStream_t>(stream)));
}

int paged_kv4_expand_blocks(void *k_cache, void *v_cache, int dtype, int64_t num_dst_blocks, const void *cache,
                            int64_t num_blocks, const int32_t *src_dst_pairs, int n_pairs, int Hkv, int D,
                            float k_unit, float v_unit, pkv_stream_t stream) {
  if (n_pairs < 0 || num_dst_blocks <= 0) return PKV_EINVAL;
  const int rc = check_pages(dtype, Hkv, D, num_blocks, k_unit, v_unit);
  if (rc != PKV_OK) return rc;
  if ((double)n_pairs * Hkv * 2 * D >= kGrid) return PKV_EUNSUPPORTED;
  if (n_pairs == 0) return PKV_OK;
  if (!cache || !k_cache || !v_cache || !src_dst_pairs) return PKV_EINVAL;
  if (!aligned(cache, 0, 1) || !aligned(k_cache, 0, 1) || !aligned(v_cache, 0, 1)) return PKV_EINVAL;
  return status_of(launch_kv4_expand(k_cache, v_cache, dtype, num_dst_blocks, static_cast<const uint8_t *>(cache),
                                     num_blocks, src_dst_pairs, n_pairs, Hkv, D, k_unit, v_unit,
                                     reinterpret_cast<cudaStream_t>(stream)));
}

int paged_kv4_copy_blocks(void *cache, const int32_t *src_dst_pairs, int n_pairs, int Hkv, int D, int64_t num_blocks,
                          pkv_stream_t stream) {
  if (n_pairs < 0 || Hkv <= 0 || num_blocks <= 0) return PKV_EINVAL;
  if (D != 64 && D != 128) return PKV_EUNSUPPORTED;
  if (n_pairs == 0) return PKV_OK;
  if (!cache || !src_dst_pairs || !aligned(cache, 0, 1)) return PKV_EINVAL;
  return status_of(launch_kv4_copy(static_cast<uint8_t *>(cache), src_dst_pairs, n_pairs, (size_t)Hkv * 18 * D,
                                   num_blocks, reinterpret_cast<cudaStream_t>(stream)));
}

int pkv_rope_turns(uint64_t *turns, const double *frequencies, int n) {
  if (n <= 0 || !turns || !frequencies) return PKV_EINVAL;
  for (int i = 0; i < n; ++i) {
    const double f = frequencies[i];
    if (!std::isfinite(f) || f < 0) return PKV_EINVAL;
    const double t = std::fmod(f / 6.283185307179586476925, 1.0);  // whole turns a position are none
    turns[i] = (uint64_t)std::ldexp(t, 64);                        // (t < 1: below 2^64)
  }
  return PKV_OK;
}

int paged_rope(void *q_out, int64_t ld_q_out, const void *q, int64_t ld_q, void *k_out, int64_t ld_k_out,
               const void *k, int64_t ld_k, int dtype, const int64_t *positions, const uint64_t *turns, int rot_dim,
               int interleaved, float magnitude, int T, int Hq, int Hkv, int D, pkv_stream_t stream) {
  RopeParams p = {};
  p.q = q; p.k = k; p.q_out = q_out; p.k_out = k_out;
  p.ld_q = ld_q; p.ld_k = ld_k; p.ld_q_out = ld_q_out; p.ld_k_out = ld_k_out;
  p.turns = turns; p.positions = positions;
  p.T = T; p.Hq = Hq; p.Hkv = Hkv; p.D = D; p.rot = rot_dim; p.interleaved = interleaved;
  p.magnitude = magnitude;
  const int rc = check_rope(p, dtype);
  if (rc != PKV_OK) return rc;
  if (T == 0) return PKV_OK;
  const int es = row_bytes(dtype);
  if (!positions || !turns) return PKV_EINVAL;
  if (!rows_ok(q, ld_q, Hq, D, es) || !rows_ok(q_out, ld_q_out, Hq, D, es) || !rows_ok(k, ld_k, Hkv, D, es) ||
      !rows_ok(k_out, ld_k_out, Hkv, D, es))
    return PKV_EINVAL;
  // in place, or apart from everything the call reads and writes
  const int64_t nq = (int64_t)Hq * D, nk = (int64_t)Hkv * D;
  if (Hq > 0) {
    if (q_out == q ? ld_q_out != ld_q : overlap(q_out, ld_q_out, nq, q, ld_q, nq, T, es)) return PKV_EINVAL;
    if (Hkv > 0 && overlap(q_out, ld_q_out, nq, k, ld_k, nk, T, es)) return PKV_EINVAL;
  }
  if (Hkv > 0) {
    if (k_out == k ? ld_k_out != ld_k : overlap(k_out, ld_k_out, nk, k, ld_k, nk, T, es)) return PKV_EINVAL;
    if (Hq > 0 && (overlap(k_out, ld_k_out, nk, q, ld_q, nq, T, es) ||
                   overlap(k_out, ld_k_out, nk, q_out, ld_q_out, nq, T, es)))
      return PKV_EINVAL;
  }
  return status_of(launch_rope(p, dtype, reinterpret_cast<cudaStream_t>(stream)));
}

// The checks that the two appends share, and the launch.
static int rope_append(RopeParams &p, int dtype, cudaStream_t stream) {
  const int rc = check_rope(p, dtype);
  if (rc != PKV_OK) return rc;
  if (p.Hq <= 0 || p.Hkv <= 0 || p.num_blocks <= 0) return PKV_EINVAL;
  if (p.T == 0) return PKV_OK;
  const int es = row_bytes(dtype);
  if (!p.positions || !p.turns || !p.slots) return PKV_EINVAL;
  if (!rows_ok(p.q, p.ld_q, p.Hq, p.D, es) || !rows_ok(p.q_out, p.ld_q_out, p.Hq, p.D, es) ||
      !rows_ok(p.k, p.ld_k, p.Hkv, p.D, es) || !rows_ok(p.v, p.ld_v, p.Hkv, p.D, es))
    return PKV_EINVAL;
  const int64_t nq = (int64_t)p.Hq * p.D, nk = (int64_t)p.Hkv * p.D;
  if (p.q_out == p.q ? p.ld_q_out != p.ld_q : overlap(p.q_out, p.ld_q_out, nq, p.q, p.ld_q, nq, p.T, es))
    return PKV_EINVAL;
  if (overlap(p.q_out, p.ld_q_out, nq, p.k, p.ld_k, nk, p.T, es) ||
      overlap(p.q_out, p.ld_q_out, nq, p.v, p.ld_v, nk, p.T, es))
    return PKV_EINVAL;
  return status_of(launch_rope(p, dtype, stream));
}

int paged_rope_append(void *q_out, int64_t ld_q_out, const void *q, int64_t ld_q, const void *k_new, int64_t ld_k,
                      const void *v_new, int64_t ld_v, int dtype, const int64_t *positions, const uint64_t *turns,
                      int rot_dim, int interleaved, float magnitude, void *k_cache, void *v_cache,
                      const int64_t *slot_mapping, int T, int Hq, int Hkv, int D, int64_t num_blocks,
                      pkv_stream_t stream) {
  RopeParams p = {};
  p.q = q; p.k = k_new; p.v = v_new; p.q_out = q_out;
  p.ld_q = ld_q; p.ld_k = ld_k; p.ld_v = ld_v; p.ld_q_out = ld_q_out;
  p.k_cache = k_cache; p.v_cache = v_cache;
  p.turns = turns; p.positions = positions; p.slots = slot_mapping;
  p.num_blocks = num_blocks;
  p.T = T; p.Hq = Hq; p.Hkv = Hkv; p.D = D; p.rot = rot_dim; p.interleaved = interleaved;
  p.magnitude = magnitude;
  if (T > 0 && (!k_cache || !v_cache || !aligned(k_cache, 0, 1) || !aligned(v_cache, 0, 1))) return PKV_EINVAL;
  return rope_append(p, dtype, reinterpret_cast<cudaStream_t>(stream));
}

int paged_kv4_rope_append(void *q_out, int64_t ld_q_out, const void *q, int64_t ld_q, const void *k_new, int64_t ld_k,
                          const void *v_new, int64_t ld_v, int dtype, const int64_t *positions,
                          const uint64_t *turns, int rot_dim, int interleaved, float magnitude, void *cache,
                          const int64_t *slot_mapping, int T, int Hq, int Hkv, int D, int64_t num_blocks,
                          float k_unit, float v_unit, pkv_stream_t stream) {
  RopeParams p = {};
  p.q = q; p.k = k_new; p.v = v_new; p.q_out = q_out;
  p.ld_q = ld_q; p.ld_k = ld_k; p.ld_v = ld_v; p.ld_q_out = ld_q_out;
  p.kv4 = static_cast<uint8_t *>(cache);
  p.turns = turns; p.positions = positions; p.slots = slot_mapping;
  p.num_blocks = num_blocks;
  p.T = T; p.Hq = Hq; p.Hkv = Hkv; p.D = D; p.rot = rot_dim; p.interleaved = interleaved;
  p.magnitude = magnitude; p.k_unit = k_unit; p.v_unit = v_unit;
  if (!kv4_unit_ok(k_unit) || !kv4_unit_ok(v_unit)) return PKV_EINVAL;
  if (T > 0 && (!cache || !aligned(cache, 0, 1))) return PKV_EINVAL;
  return rope_append(p, dtype, reinterpret_cast<cudaStream_t>(stream));
}

}  // extern "C"
