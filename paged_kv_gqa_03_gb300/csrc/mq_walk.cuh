// mq_walk.cuh — the stream-K schedule shared by the tensor-core kernels for
// several new tokens per sequence (mq_decode.cu, tree_tiles.cu): the K / V tiles of
// 128 positions of all (sequence, kv head) items form one sequence that is cut
// into equal contiguous ranges.
#pragma once

#include "common.cuh"
#include "mq_decode.h"

namespace pkv {

// Tile facts of one sequence: the clamped context, the first position any
// new token's window reaches, the first K / V tile and the tile count T (per
// kv head).  Token i sees positions [ctx - q_len + 1 + i - window, ctx - q_len
// + 1 + i) (no lower bound without a window).
struct MqSeq {
  int ctx, first, j_first, T;
  int n;  // new tokens: q_len, or the tree's nodes
  bool bad_ctx;
};
__device__ __forceinline__ MqSeq mq_seq(const MqParams &p, int b) {
  MqSeq s;
  s.n = p.q_len;
  bool bad_n = false;
  if (p.tree_lens != nullptr) {
    const int n = __ldg(p.tree_lens + b);
    s.n = min(max(n, 0), p.q_len);
    bad_n = n != s.n;
  }
  const int raw = __ldg(p.context_lens + b);
  const int cap = p.max_blocks * kBlock;
  s.ctx = raw < 0 ? 0 : (raw > cap ? cap : raw);
  s.bad_ctx = raw != s.ctx || bad_n;
  const int lim_lo = s.ctx - s.n + 1;  // exclusive end of token 0's positions
  s.first = p.window > 0 ? max(0, lim_lo - p.window) : 0;
  s.j_first = s.first / 128;
  s.T = s.ctx > 0 && s.n > 0 ? (s.ctx - 1) / 128 - s.j_first + 1 : 0;
  return s;
}

// A CTA's share of the stream-K order: tiles [t0, t1) of the sequence of all
// items' tiles (item (b, h) holds tiles [prefix[b] + h * T_b, ... + T_b)).
// One segment = the part of one item inside the range; every role walks the
// same segments.
struct MqSeg {
  int b, h, j0, j1, T, ctx, first, j_first, n;
  int slot;    // partial-output slot of a cut item: 0 if the segment starts the CTA's range, else 1
  bool whole;  // the segment is the whole item (the CTA writes the output itself)
};
struct MqWalk {
  int t, t0, t1, b, base;  // next tile; the range; the sequence holding tile t and its first tile
  __device__ __forceinline__ void start(int b0, int base0, int tile0, int tile1) {
    b = b0;
    base = base0;
    t = t0 = tile0;
    t1 = tile1;
  }
  __device__ __forceinline__ bool next(const MqParams &p, MqSeg &sg) {
    if (t >= t1) return false;
    MqSeq s = mq_seq(p, b);
    while (t >= base + s.T * p.Hkv) {  // on to the sequence holding tile t (skipping empty ones)
      base += s.T * p.Hkv;
      s = mq_seq(p, ++b);
    }
    const int off = t - base;
    sg.b = b;
    sg.T = s.T;
    sg.h = off / s.T;
    sg.j0 = off - sg.h * s.T;
    sg.j1 = min(s.T, sg.j0 + (t1 - t));
    sg.ctx = s.ctx;
    sg.first = s.first;
    sg.j_first = s.j_first;
    sg.n = s.n;
    sg.slot = t == t0 ? 0 : 1;
    sg.whole = sg.j0 == 0 && sg.j1 == s.T;
    t += sg.j1 - sg.j0;
    return true;
  }
};

// ---- the plan: every CTA scans the sequences' tile counts (THREADS threads, up
// to kMqMaxBatch / THREADS sequences each) and finds its range's start; CTA 0 also
// writes the prefix for the merge kernel.  `part` of `parts` ranges; with
// fewer tiles than ranges each of the first W ranges gets one tile. ----
struct MqPlan {
  int32_t wsum[8], b0, base0;  // per-warp tile sums; where the range starts
};
// Ranges that receive work.
__device__ __forceinline__ int mq_active(int W, int parts) { return W < parts ? (W > 0 ? W : 1) : parts; }
// floor(W part / active), in 32 bits (active is at most the SM count)
__device__ __forceinline__ int mq_cut(int W, int active, int part) {
  const unsigned q = (unsigned)W / (unsigned)active, rem = (unsigned)W - q * (unsigned)active;
  return part < active ? (int)(q * (unsigned)part + rem * (unsigned)part / (unsigned)active) : W;
}
// Block-wide (every thread of the CTA calls it).
template <int THREADS>
__device__ __forceinline__ void mq_plan(const MqParams &p, int part, int parts, MqPlan *plan, int *cta_flags, int *t0_out,
                                        int *t1_out, int *b0_out, int *base0_out) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int B = p.B;
  const int per = (B + THREADS - 1) / THREADS;
  int tk[kMqMaxBatch / THREADS];
  int own = 0, incl = 0;
  if (tid < THREADS) {
    int bad = 0;
#pragma unroll
    for (int k = 0; k < kMqMaxBatch / THREADS; ++k) {
      const int b = tid * per + k;
      tk[k] = 0;
      if (k < per && b < B) {
        const MqSeq s = mq_seq(p, b);
        tk[k] = s.T * p.Hkv;
        bad |= s.bad_ctx ? 1 : 0;
      }
      own += tk[k];
    }
    incl = own;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int n = __shfl_up_sync(kFull, incl, o);
      if (lane >= o) incl += n;
    }
    if (lane == 31) plan->wsum[warp] = incl;
    if (blockIdx.x == 0 && __any_sync(kFull, bad) && lane == 0) atomicOr(cta_flags, PKV_FLAG_BAD_LEN);
  }
  __syncthreads();
  int W = 0;
#pragma unroll
  for (int w = 0; w < THREADS / 32; ++w) W += plan->wsum[w];
  const int active = mq_active(W, parts);
  const int t0 = mq_cut(W, active, part), t1 = mq_cut(W, active, part + 1);
  if (tid == 0) {  // an empty range (t0 == W): nothing to walk
    plan->b0 = B;
    plan->base0 = W;
    if (blockIdx.x == 0) p.prefix[B] = W;
  }
  __syncthreads();
  if (tid < THREADS) {
    int run = incl - own;
    for (int w = 0; w < warp; ++w) run += plan->wsum[w];
#pragma unroll
    for (int k = 0; k < kMqMaxBatch / THREADS; ++k) {
      const int b = tid * per + k;
      if (k < per && b < B) {
        if (blockIdx.x == 0) p.prefix[b] = run;
        if (run <= t0 && t0 < run + tk[k]) {  // the sequence holding the range's first tile
          plan->b0 = b;
          plan->base0 = run;
        }
        run += tk[k];
      }
    }
  }
  __syncthreads();
  *t0_out = t0;
  *t1_out = t1;
  *b0_out = plan->b0;
  *base0_out = plan->base0;
}

}  // namespace pkv
