// tree_commit.cu — the accepted path of a tree of drafted tokens, moved
// together in the paged cache (paged_tree_commit): for k = 0 .. len - 1 the K / V
// row of node path[k] (position start + path[k]) becomes that of position
// start + k, where start is the tree's first position.  The tokens that stay
// are then consecutive positions, as the block table ("LLM推理优化实战" §2.2)
// and the next step want them.
//
// In place and without scratch: node indices grow along a path, so path[k] >= k
// and a row is never overwritten before it has been read when rows move in
// order of k.  One warp per (sequence, kv head, K or V): its lanes hold the
// whole path's source and destination slots (two entries each), then move rows
// of row_bytes / 16 lanes, several rows per load, every load of a group issued
// before its first store.  The kernel is three dependent latencies (path,
// block table, rows) and a few KB per warp; nothing else bounds it: 1 sequence of 16
// nodes 1.9 us, 128 of 64 (fp8, rows between blocks re-quantised) 3.8 us on the device; out of
// cold caches 6 and 8 us.
//
// FP8 caches: a row moved inside its block keeps its bytes; one that changes
// blocks is re-quantised with the destination block's scale (which stays),
// e4m3_rne_sat( fp32( decode(q) * s_src ) / s_dst ).
//
// Calibrated caches (paged_tree_commit_calibrated) promise that no stored value
// saturates.  There a destination block whose scale does not cover a row moved into it
// first gets the smallest power of two that does, its rows re-quantised, as a token that
// outgrows its block does in the calibrated append.  The rows of a warp then depend on
// one another through the scales, and move one after another: 128 sequences of 64 nodes
// 6 us more than the plain call, 25 us out of cold caches.
#include "common.cuh"
#include "internal.h"
#include "pow2_scale.cuh"
#include "tree.h"

namespace pkv {

__device__ __forceinline__ uint32_t requant4(uint32_t w, float from, float to) {
  uint32_t r = 0;
#pragma unroll
  for (int e = 0; e < 4; e += 2) {
    const float2 v = unpack2_e4m3((uint16_t)(w >> (8 * e)));
    const uint32_t a = __nv_cvt_float_to_fp8(__fdiv_rn(__fmul_rn(v.x, from), to), __NV_SATFINITE, __NV_E4M3);
    const uint32_t c = __nv_cvt_float_to_fp8(__fdiv_rn(__fmul_rn(v.y, from), to), __NV_SATFINITE, __NV_E4M3);
    r |= (a | c << 8) << (8 * e);
  }
  return r;
}

// What one warp moves: rows k = lane and lane + 32 of its sequence's path, source and
// destination (block * 16 + offset; -1: no move).
struct Moves {
  int64_t src[2], dst[2];
  int start, n, len;
};
__device__ __forceinline__ Moves path_moves(const CommitParams &p, int b, int lane) {
  Moves w;
  w.n = p.tree_lens ? min(max(__ldg(p.tree_lens + b), 0), p.n) : p.n;
  w.start = __ldg(p.context_lens + b) - w.n;
  w.len = min(max(__ldg(p.path_len + b), 0), w.n);
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int k = lane + 32 * j;
    w.src[j] = w.dst[j] = -1;
    if (k < w.len) {
      const int from = __ldg(p.path + (int64_t)b * p.n + k);
      const int64_t sp = (int64_t)w.start + from, dp = (int64_t)w.start + k;
      // (an entry out of order or out of range moves nothing)
      if (from > k && from < w.n && dp >= 0 && sp < (int64_t)p.max_blocks * kBlock) {
        const int32_t *row = p.block_table + (int64_t)b * p.max_blocks;
        const int sb = __ldg(row + sp / kBlock), db = __ldg(row + dp / kBlock);
        if (sb >= 0 && sb < p.num_blocks && db >= 0 && db < p.num_blocks) {
          w.src[j] = (int64_t)sb * kBlock + sp % kBlock;
          w.dst[j] = (int64_t)db * kBlock + dp % kBlock;
        }
      }
    }
  }
  return w;
}

// LPR = lanes per row (row_bytes / 16).
template <int LPR, bool kFp8>
__global__ void __launch_bounds__(128) tree_commit_kernel(const __grid_constant__ CommitParams p) {
  constexpr int ROWS = 32 / LPR;  // rows of one warp-wide access
  constexpr int BATCH = 4;        // accesses in flight
  grid_dep_wait();
  const int64_t gw = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) >> 5;
  const int lane = threadIdx.x & 31;
  if (gw >= (int64_t)p.B * p.Hkv * 2) return;
  const int kv = (int)(gw & 1), h = (int)((gw >> 1) % p.Hkv), b = (int)((gw >> 1) / p.Hkv);
  const Moves mv = path_moves(p, b, lane);
  if (p.new_lens != nullptr && kv == 0 && h == 0 && lane == 0) p.new_lens[b] = max(0, mv.start + mv.len);
  const int len = mv.len;
  const unsigned m0 = __ballot_sync(kFull, mv.src[0] >= 0), m1 = __ballot_sync(kFull, mv.src[1] >= 0);
  if ((m0 | m1) == 0) return;
  uint8_t *cache = kv ? p.v_cache : p.k_cache;
  const float *scale = kv ? p.v_scale : p.k_scale;
  const int part = lane % LPR;
  for (int k0 = 0; k0 < len; k0 += ROWS * BATCH) {
    uint4 x[BATCH];
    int64_t to[BATCH];
    float sf[BATCH], st[BATCH];
#pragma unroll
    for (int t = 0; t < BATCH; ++t) {
      const int k = k0 + t * ROWS + lane / LPR;
      // every lane takes part in the shuffles; k < 64 + ROWS * BATCH
      const int64_t s0 = __shfl_sync(kFull, mv.src[0], k & 31), s1 = __shfl_sync(kFull, mv.src[1], k & 31);
      const int64_t d0 = __shfl_sync(kFull, mv.dst[0], k & 31), d1 = __shfl_sync(kFull, mv.dst[1], k & 31);
      const int64_t s = k < 32 ? s0 : (k < 64 ? s1 : -1), d = k < 32 ? d0 : d1;
      to[t] = -1;
      if (s >= 0) {
        // element row of [num_blocks][Hkv][16] holding (block, h, offset)
        const int64_t sr = ((s / kBlock) * p.Hkv + h) * kBlock + s % kBlock;
        to[t] = ((d / kBlock) * p.Hkv + h) * kBlock + d % kBlock;
        x[t] = *reinterpret_cast<const uint4 *>(cache + sr * p.row_bytes + part * 16);
        if constexpr (kFp8) {
          sf[t] = st[t] = 1.f;
          if (s / kBlock != d / kBlock) {
            sf[t] = __ldg(scale + (s / kBlock) * p.Hkv + h);
            st[t] = __ldg(scale + (d / kBlock) * p.Hkv + h);
            x[t] = make_uint4(requant4(x[t].x, sf[t], st[t]), requant4(x[t].y, sf[t], st[t]),
                              requant4(x[t].z, sf[t], st[t]), requant4(x[t].w, sf[t], st[t]));
          }
        }
      }
    }
    __syncwarp();  // the group's rows are in registers before any is overwritten
#pragma unroll
    for (int t = 0; t < BATCH; ++t)
      if (to[t] >= 0) *reinterpret_cast<uint4 *>(cache + to[t] * p.row_bytes + part * 16) = x[t];
    __syncwarp();
  }
}

// The calibrated form (fp8): one row of the path after another, every lane the same.
template <int LPR>
__global__ void __launch_bounds__(128) tree_commit_calibrated_kernel(const __grid_constant__ CommitParams p) {
  constexpr int ROWS = 32 / LPR;
  grid_dep_wait();
  const int64_t gw = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) >> 5;
  const int lane = threadIdx.x & 31;
  if (gw >= (int64_t)p.B * p.Hkv * 2) return;
  const int kv = (int)(gw & 1), h = (int)((gw >> 1) % p.Hkv), b = (int)((gw >> 1) / p.Hkv);
  const Moves mv = path_moves(p, b, lane);
  if (p.new_lens != nullptr && kv == 0 && h == 0 && lane == 0) p.new_lens[b] = max(0, mv.start + mv.len);
  uint8_t *cache = kv ? p.v_cache : p.k_cache;
  float *scale = kv ? p.v_scale : p.k_scale;
  const int part = lane % LPR;
  uint64_t todo = (uint64_t)__ballot_sync(kFull, mv.src[0] >= 0) | (uint64_t)__ballot_sync(kFull, mv.src[1] >= 0) << 32;
  for (; todo; todo &= todo - 1) {
    const int k = __ffsll((long long)todo) - 1;
    const int64_t s = __shfl_sync(kFull, k < 32 ? mv.src[0] : mv.src[1], k & 31);
    const int64_t d = __shfl_sync(kFull, k < 32 ? mv.dst[0] : mv.dst[1], k & 31);
    uint8_t *from = cache + (((s / kBlock) * p.Hkv + h) * kBlock + s % kBlock) * p.row_bytes;
    uint8_t *block = cache + ((d / kBlock) * p.Hkv + h) * (int64_t)(kBlock * p.row_bytes);  // the destination's
    uint4 x = *reinterpret_cast<const uint4 *>(from + part * 16);
    if (s / kBlock != d / kBlock) {
      const float ss = scale[(s / kBlock) * p.Hkv + h];
      float sd = scale[(d / kBlock) * p.Hkv + h];
      float top = 0.f;
      const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 u = unpack2_e4m3((uint16_t)(w[i] & 0xffff)), v = unpack2_e4m3((uint16_t)(w[i] >> 16));
        top = fmaxf(top, fmaxf(fmaxf(fabsf(u.x), fabsf(u.y)), fmaxf(fabsf(v.x), fabsf(v.y))));
      }
#pragma unroll
      for (int o = LPR / 2; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(kFull, top, o));
      const float amax = __fmul_rn(top, ss);
      const float need = amax > 0.f && amax < INFINITY ? pow2_scale(amax) : 0.f;  // (nothing covers an overflowed row)
      if (need > sd) {
        // the block's rows up to the tree's end: the prefix, what has moved in, and what may still move
        const int used = (int)min((int64_t)kBlock, (int64_t)(mv.start + mv.n) - (mv.start + k - d % kBlock));
        for (int r = lane / LPR; r < used; r += ROWS) {
          uint4 *row = reinterpret_cast<uint4 *>(block + (int64_t)r * p.row_bytes + part * 16);
          const uint4 y = *row;
          *row = make_uint4(requant4(y.x, sd, need), requant4(y.y, sd, need), requant4(y.z, sd, need), requant4(y.w, sd, need));
        }
        sd = need;
        __syncwarp();  // (the scale has been read, and the rows written, by all)
        if (lane == 0) scale[(d / kBlock) * p.Hkv + h] = sd;
      }
      x = make_uint4(requant4(x.x, ss, sd), requant4(x.y, ss, sd), requant4(x.z, ss, sd), requant4(x.w, ss, sd));
    }
    __syncwarp();
    if (lane < LPR) *reinterpret_cast<uint4 *>(block + (d % kBlock) * p.row_bytes + part * 16) = x;
    __syncwarp();
  }
}

template <int LPR, bool kFp8>
static cudaError_t launch_commit_t(const CommitParams &p, cudaStream_t stream) {
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(((int64_t)p.B * p.Hkv * 2 + 3) / 4));
  cfg.blockDim = dim3(128);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = stream != nullptr ? 1 : 0;  // early launch on explicit streams only
  if constexpr (kFp8)
    if (p.calibrated) return cudaLaunchKernelEx(&cfg, tree_commit_calibrated_kernel<LPR>, p);
  return cudaLaunchKernelEx(&cfg, tree_commit_kernel<LPR, kFp8>, p);
}

cudaError_t launch_tree_commit(const CommitParams &p, cudaStream_t stream) {
  if (p.k_scale != nullptr) {
    if (p.row_bytes == 64) return launch_commit_t<4, true>(p, stream);
    return launch_commit_t<8, true>(p, stream);
  }
  switch (p.row_bytes) {
    case 128: return launch_commit_t<8, false>(p, stream);
    case 256: return launch_commit_t<16, false>(p, stream);
    case 512: return launch_commit_t<32, false>(p, stream);
  }
  return cudaErrorNotSupported;
}

}  // namespace pkv
