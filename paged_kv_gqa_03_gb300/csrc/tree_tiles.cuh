// tree_tiles.cuh — the schedule and the masks shared by the row-tile kernels for
// a tree of drafted tokens (tree_tiles.cu: 16-bit caches, tree_tiles_fp8.cu).
#pragma once

#include "mq_walk.cuh"
#include "tree_finite.cuh"
#include "tree_tiles.h"

namespace pkv {

// What group g's range is, for the merge kernel: its first tile, and the item
// that tile cuts ([a, e) its tiles), e = 0 if the range starts at an item's end.
struct TreeCut {
  int t0, b, h, a, e;
};

// The schedule of one CTA: range [t0, t1) of the tiles, starting in sequence b0
// whose first tile is base0.
struct TreeRange {
  int t0, t1, b0, base0;
};
// Block-wide; `find` is shared memory for the scan: the sequences holding the
// range's ends.
struct TreeFind {
  int32_t wsum[8], b[2], base[2], T[2];
};
template <int THREADS>
__device__ __forceinline__ TreeRange tree_plan(const MqParams &p, int group, int groups, TreeFind *find, int *cta_flags) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int B = p.B, per = (B + THREADS - 1) / THREADS, b_end = min(B, (tid + 1) * per);
  int own = 0, incl = 0;
  // (loops, not unrolled: this code runs once, from a cold instruction cache)
  if (tid < THREADS) {
    bool bad = false;
#pragma unroll 1
    for (int b = tid * per; b < b_end; ++b) {
      const MqSeq s = mq_seq(p, b);
      own += s.T * p.Hkv;
      bad |= s.bad_ctx;
    }
    incl = own;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int n = __shfl_up_sync(kFull, incl, o);
      if (lane >= o) incl += n;
    }
    if (lane == 31) find->wsum[warp] = incl;
    if (blockIdx.x == 0 && __any_sync(kFull, bad) && lane == 0) atomicOr(cta_flags, PKV_FLAG_BAD_LEN);
  }
  __syncthreads();
  int W = 0, run = incl - own;
#pragma unroll
  for (int w = 0; w < THREADS / 32; ++w) {
    const int n = find->wsum[w];
    run += w < warp ? n : 0;
    W += n;
  }
  const int active = mq_active(W, groups);
  TreeRange r;
  r.t0 = mq_cut(W, active, group);
  r.t1 = mq_cut(W, active, group + 1);
  if (tid < THREADS && ((run <= r.t0 && r.t0 < run + own) || (run <= r.t1 && r.t1 < run + own))) {
#pragma unroll 1
    for (int b = tid * per; b < b_end; ++b) {
      const int T = mq_seq(p, b).T, n = T * p.Hkv;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int t = i == 0 ? r.t0 : r.t1;
        if (run <= t && t < run + n) {
          find->b[i] = b;
          find->base[i] = run;
          find->T[i] = T;
        }
      }
      run += n;
    }
  }
  __syncthreads();
  auto snap = [&](int t, int i) -> int {
    const int T = find->T[i], d = (t - find->base[i]) % T;
    return d <= kSnapTiles ? t - d : (T - d <= kSnapTiles ? t + T - d : t);
  };
  r.b0 = B;
  r.base0 = W;
  if (r.t0 < W) {  // (else an empty range)
    r.b0 = find->b[0];
    r.base0 = find->base[0];
    r.t0 = snap(r.t0, 0);
  }
  if (r.t1 < W) r.t1 = snap(r.t1, 1);
  return r;
}

// Which of the 64 cache positions from `pos` on a row sees, as bits: the cached
// ones in [lo, start), then node t at start + t iff bit t of mask.
__device__ __forceinline__ uint64_t tree_columns(uint64_t mask, int start, int lo, int pos) {
  const int c0 = start - pos;  // the tree's first column
  uint64_t sees = c0 >= 64 ? ~0ull : (c0 > 0 ? ~(~0ull << c0) | mask << c0 : (c0 > -64 ? mask >> -c0 : 0ull));
  const int cl = lo - pos;     // the first cached column this row sees
  if (cl > 0) {
    const uint64_t hidden = cl >= 64 ? ~0ull : ~(~0ull << cl);
    sees &= ~(c0 >= 64 ? hidden : (c0 > 0 ? hidden & ~(~0ull << c0) : 0ull));  // (the nodes are the mask's alone)
  }
  return sees;
}

// warp_wait (prefill_common.cuh) with all but its first try out of line: the tile
// loops hold many waits, and most are over when they are reached.  ROLE: a copy for
// warps with another register count (setmaxnreg).
template <int ROLE>
static __device__ __noinline__ bool wait_longer(uint64_t *bar, uint32_t parity, uint64_t limit_ns) {
  return warp_wait(bar, parity, limit_ns);
}
template <int ROLE = 0>
__device__ __forceinline__ bool tile_wait(uint64_t *bar, uint32_t parity, uint64_t limit_ns) {
  return __all_sync(kFull, mbar_try_wait(bar, parity)) || wait_longer<ROLE>(bar, parity, limit_ns);
}

// What a softmax warp does to its 64 columns of a tile's S, P or its half of O only
// now and then, each in a function of its own on tensor memory: the tile loop
// itself stays a short run of instructions (inline, these rare parts cost every tile
// instruction-cache misses).  All are warp-wide.
//
// Hides the columns of S whose bit of `sees` is 0; `k`, where given, holds the block
// scales {k_b, v_b} of literal products: S of such blocks is multiplied by k_b.
static __device__ __noinline__ void fix_scores(uint32_t scol, uint64_t sees, const float2 *raw, uint32_t literal) {
#pragma unroll 1
  for (int q = 0; q < 8; ++q) {  // 8 columns
    uint32_t s[8];
    tc::ld8(scol + (uint32_t)(q * 8), s);
    const float k = (literal >> (q >> 1)) & 1 ? raw[q >> 1].x : 1.f;
    const uint32_t bits = (uint32_t)(sees >> (q * 8));
#pragma unroll
    for (int e = 0; e < 8; ++e)
      s[e] = (bits >> e) & 1 ? __float_as_uint(__uint_as_float(s[e]) * k) : 0xff800000u;  // hidden: -inf
    tc::st8(scol + (uint32_t)(q * 8), s[0], s[1], s[2], s[3], s[4], s[5], s[6], s[7]);
  }
  tc::wait_st();
}
// Multiplies the packed f16 weights (32 columns at pcol) of literal blocks by v_b.
static __device__ __noinline__ void fix_weights(uint32_t pcol, const float2 *raw, uint32_t literal) {
#pragma unroll 1
  for (int b = 0; b < 4; ++b) {
    if (!((literal >> b) & 1)) continue;
    uint32_t w[8];
    tc::ld8(pcol + (uint32_t)(b * 8), w);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float2 x = unpack2(F16{}, w[e]);
      w[e] = pack_f16x2(x.x * raw[b].y, x.y * raw[b].y);
    }
    tc::st8(pcol + (uint32_t)(b * 8), w[0], w[1], w[2], w[3], w[4], w[5], w[6], w[7]);
  }
  tc::wait_st();
}
// Multiplies `cols` columns of O at ta by alpha.
static __device__ __noinline__ void rescale_o(uint32_t ta, float alpha, int cols) {
#pragma unroll 1
  for (int q = 0; q < cols; q += 8) {
    uint32_t o[8];
    tc::ld8(ta + (uint32_t)q, o);
#pragma unroll
    for (int e = 0; e < 8; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
    tc::st8(ta + (uint32_t)q, o[0], o[1], o[2], o[3], o[4], o[5], o[6], o[7]);
  }
  tc::wait_st();
}

// The items of a CTA as its S-issuing warp publishes them for the softmax warps, one item ahead
// (four entries: the softmax may still write an item's output while the one after the
// next is published).  Kept in shared memory, they cost the tile loop no registers, which
// are what it is short of.
struct TreeItem {
  MqSeg s;
  int have;  // 0: past the last
};

// What not every row of an item sees (tree_finite.cuh), and which of its tiles hold such
// positions: j >= tree or j < edge.
__device__ __forceinline__ TreePartial tree_partial(const MqParams &p, const MqSeg &sg) {
  const int start = sg.ctx - sg.n;
  return TreePartial{sg.first, p.window > 0 ? start + p.q_len - p.window : 0, start};
}
struct PartialTiles {
  int tree, edge;
  __device__ __forceinline__ bool has(int j) const { return j >= tree || j < edge; }
};
__device__ __forceinline__ PartialTiles partial_tiles(const MqParams &p, const MqSeg &sg) {
  const TreePartial t = tree_partial(p, sg);
  return PartialTiles{max(t.start, 0) / 128 - sg.j_first, t.edge > 0 ? (t.edge - 1) / 128 + 1 - sg.j_first : 0};
}
// Adds the elements of the item's noted V rows that are not finite to O, for the rows that
// see them: columns col0 .. col0 + D / 2 - 1, at ta.  Warp-wide.
template <class T, int D>
static __device__ __noinline__ void add_spoiled(const TreeTileParams &tp, uint32_t ta, int b, int h, int start, int first,
                                                uint64_t nodes, uint64_t edges, uint64_t mask, int lo, int col0) {
  const MqParams &p = tp.m;
#pragma unroll 1
  for (int edge = 0; edge < 2; ++edge) {
#pragma unroll 1
    for (uint64_t m = edge ? edges : nodes; m; m &= m - 1) {
      const int bit = __ffsll((long long)m) - 1, pos = (edge ? first : start) + bit;
      const bool sees = edge ? pos >= lo : ((mask >> bit) & 1) != 0;
      const int64_t blk = __ldg(p.block_table + (size_t)b * p.max_blocks + pos / kBlock);
      const size_t row = ((size_t)(blk * p.Hkv + h) * kBlock + pos % kBlock) * D + col0;
#pragma unroll 1
      for (int q = 0; q < D / 2; q += 8) {
        uint32_t o[8];
        tc::ld8(ta + (uint32_t)q, o);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float x = nonfinite_value<T>(tp.v_cache, row + q + e);
          if (sees) o[e] = __float_as_uint(__uint_as_float(o[e]) + x);
        }
        tc::st8(ta + (uint32_t)q, o[0], o[1], o[2], o[3], o[4], o[5], o[6], o[7]);
      }
    }
  }
  tc::wait_st();
}

// Log-sum-exp (log2) of a partial with running max m and sum l: -inf where the row
// sees nothing, +inf for a sum that is NaN, so that the merge gives NaN.
__device__ __forceinline__ float partial_lse(float m, float l) {
  return l > 0.f ? m + log2f(l) : (l == 0.f ? -INFINITY : INFINITY);
}

// A CTA's status bits: for the merge kernel, or into the header if none follows.
__device__ __forceinline__ void write_status(const TreeTileParams &tp, int flags) {
  if (tp.cta_status == nullptr) {
    tp.m.cta_flags[blockIdx.x] = flags;
    return;
  }
  tp.cta_status[blockIdx.x] = (uint8_t)flags;
  if (blockIdx.x == 0) *tp.m.status = kStatusPerCta | (int)gridDim.x;
}

// The schedule's launch (tree_tiles.cu): joins the items cut between groups.
cudaError_t launch_tree_merge(const TreeTileParams &p, int grid, int out_bf16, cudaStream_t stream);

}  // namespace pkv
