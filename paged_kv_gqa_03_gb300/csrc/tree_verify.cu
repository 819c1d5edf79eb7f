// tree_verify.cu — which drafted tokens of a tree the target model accepts
// (paged_tree_verify): the acceptance step of speculative decoding
// ("LLM推理优化实战" §4), on a tree of drafts, from given random numbers.
//
// The walk starts at node 0 and tries a node's children in index order.  With
// p the target's and q the draft's distribution at the node and j children
// refused there so far, the residual the next child is tried against is
//   w_j(t) = max(p(t) - a_j q(t), 0),  z_j = sum_t w_j(t) (z_0 = 1),
//   a_0 = 0, a_(j+1) = a_j + z_j:
// each refusal replaces the normalised residual r by max(r - q, 0), and since a
// weight that reaches 0 stays there, j of those steps collapse into one
// subtraction with the scalar a_j.  Child c is accepted iff
// u_c q(c) z_j < w_j(c).  The token after the walk is drawn from the last
// node's residual by inverse CDF.
//
// What bounds it.  Only refusals and the final draw read whole rows (p and q,
// V values each); accepted drafts need two numbers each, gathered for all
// nodes at once.  So the kernel is a few dependent latencies plus one or two
// row passes: a cluster of CTAs serves one sequence, each CTA a contiguous
// slice of the vocabulary, each warp a contiguous part of it.  CTA 0's first
// warp walks; it hands the others one command at a time through distributed
// shared memory, so that no CTA ever decides on its own how many cluster
// barriers there are.
//
// Exactness.  A draw compares partial sums of up to V terms with u times the
// total; sums in 32 bits would move such a border by ~1e-7, and with it one
// token in some thousands.  The terms and sums are therefore kept as
// unevaluated pairs of floats (Knuth's two-sum, Dekker's product by fma,
// ~48 bits): the fp64 pipe of this GPU is far too narrow for V terms.
#include <cooperative_groups.h>

#include "common.cuh"
#include "internal.h"
#include "tree.h"

namespace pkv {

namespace cg = cooperative_groups;

namespace {

constexpr int kTree = PKV_MAX_Q_LEN;
constexpr int kMaxCluster = 8;

// An unevaluated sum h + l of two floats.
struct F2 {
  float h, l;
};
__device__ __forceinline__ F2 two_sum(float a, float b) {
  const float s = __fadd_rn(a, b), t = __fsub_rn(s, a);
  return {s, __fadd_rn(__fsub_rn(a, __fsub_rn(s, t)), __fsub_rn(b, t))};
}
__device__ __forceinline__ F2 f2_plus(F2 a, F2 b) {
  const F2 s = two_sum(a.h, b.h);
  const float e = __fadd_rn(s.l, __fadd_rn(a.l, b.l));
  const float h = __fadd_rn(s.h, e);
  return {h, __fsub_rn(e, __fsub_rn(h, s.h))};
}
__device__ __forceinline__ double f2_double(F2 a) { return (double)a.h + (double)a.l; }

enum : int { kExit = 0, kSum = 1, kArgmax = 2 };

struct Cmd {
  int op, node;
  F2 a;  // residual coefficient of the draft row
};

// max(p - a q, 0)
__device__ __forceinline__ F2 residual(float p, float q, F2 a) {
  const float m = __fmul_rn(a.h, q);
  const float ml = __fmaf_rn(a.l, q, __fmaf_rn(a.h, q, -m));
  F2 d = two_sum(p, -m);
  d.l = __fsub_rn(d.l, ml);
  return __fadd_rn(d.h, d.l) > 0.f ? d : F2{0.f, 0.f};  // (a NaN gives 0)
}

template <class T>
__device__ __forceinline__ void load4(const void *row, int64_t i, bool vec, int64_t end, float (&x)[4]) {
  if (vec) {  // 4 elements, aligned, inside the row
    if constexpr (T::kBytes == 4) {
      const float4 v = *reinterpret_cast<const float4 *>(static_cast<const float *>(row) + i);
      x[0] = v.x; x[1] = v.y; x[2] = v.z; x[3] = v.w;
    } else {
      const uint2 v = *reinterpret_cast<const uint2 *>(static_cast<const uint16_t *>(row) + i);
      const float2 a = unpack2(T{}, v.x), b = unpack2(T{}, v.y);
      x[0] = a.x; x[1] = a.y; x[2] = b.x; x[3] = b.y;
    }
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) x[e] = i + e < end ? load_scalar(T{}, row, (size_t)(i + e)) : 0.f;
  }
}

}  // namespace

// The nodes, as bits, that are children of `node` with a token in [lo, hi)
// (warp-wide).
__device__ __forceinline__ uint64_t lost_in(const int *parent, const int *tok, int node, int lo, int hi, int lane) {
  const bool l0 = parent[lane] == node && tok[lane] >= lo && tok[lane] < hi;
  const bool l1 = parent[lane + 32] == node && tok[lane + 32] >= lo && tok[lane + 32] < hi;
  return (uint64_t)__ballot_sync(kFull, l0) | (uint64_t)__ballot_sync(kFull, l1) << 32;
}

// The elements [lo, hi) of the vocabulary that warp `w` of `total` serves:
// equal parts in order, multiples of 4 elements.
__device__ __forceinline__ void warp_part(int V, int w, int total, int *lo, int *hi) {
  const int per = ((V + total - 1) / total + 3) & ~3;
  *lo = min(V, w * per);
  *hi = min(V, *lo + per);
}

template <class T, int THREADS>
__global__ void __launch_bounds__(THREADS) tree_verify_kernel(const __grid_constant__ VerifyParams p) {
  constexpr int WARPS = THREADS / 32;
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = (int)cluster.block_rank(), C = (int)cluster.num_blocks();
  const int b = blockIdx.x / C;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  __shared__ Cmd cmd;
  __shared__ int s_parent[kTree];
  __shared__ int s_tok[kTree];  // -1: outside the vocabulary
  __shared__ float s_p[kTree], s_q[kTree], s_u[kTree];
  __shared__ int s_path[kTree];
  // (leader) each warp's sum, or argmax
  __shared__ double s_sum[kMaxCluster * WARPS];
  __shared__ float s_best[kMaxCluster * WARPS];
  __shared__ int s_at[kMaxCluster * WARPS];
  __shared__ F2 s_scan[WARPS];
  // (leader) the final draw: the warp part, the first element past the border, the last with any weight
  __shared__ int s_hit, s_node, s_first, s_last;
  __shared__ double s_base, s_thr;
  __shared__ F2 s_a;
  grid_dep_wait();

  const int n = p.lens ? min(max(p.lens[b], 0), p.n) : p.n;
  const bool draft = p.draft != nullptr, greedy = p.u == nullptr;
  auto row = [&](const void *base, int64_t ld, int node) {
    return static_cast<const void *>(static_cast<const uint8_t *>(base) + ((int64_t)b * p.n + node) * ld * T::kBytes);
  };
  if (tid < kTree) {
    int up = -1, tok = -1;
    if (tid < n) {
      const uint64_t below = p.mask[(int64_t)b * p.mask_stride + tid] & ((1ull << tid) - 1);
      up = below ? 63 - __clzll(below) : -1;
      const int64_t t = p.tokens[(int64_t)b * p.n + tid];
      tok = t >= 0 && t < p.V ? (int)t : -1;
    }
    s_parent[tid] = up;
    s_tok[tid] = tok;
    if (rank == 0) {
      const bool ask = up >= 0 && tok >= 0 && !greedy;
      s_p[tid] = ask ? load_scalar(T{}, row(p.target, p.ld_target, up), (size_t)tok) : 0.f;
      s_q[tid] = ask && draft ? load_scalar(T{}, row(p.draft, p.ld_draft, up), (size_t)tok) : 1.f;
      s_u[tid] = !greedy && tid < n ? p.u[(int64_t)b * p.n + tid] : 0.f;
    }
  }
  cluster.sync();  // (every CTA of the cluster is running before its shared memory is written)

  // ---- the walk's state (first warp of the leader; every lane the same) ----
  int cur = 0, i = 1, len = 1, best = -1;
  double a = 0.0, z = 1.0, left = 1.0;
  bool summed = false, done = false;
  auto take = [&](int node) {
    cur = node;
    if (lane == 0) s_path[len] = node;
    ++len;
    a = 0.0;
    z = left = 1.0;
    summed = false;
  };
  // runs to the next row pass, or to the end (kExit)
  auto advance = [&]() -> Cmd {
    Cmd c{kExit, 0, {0.f, 0.f}};
    if (greedy) {
      if (best >= 0) {  // cur's most likely token is known: its child, if drafted
        int found = -1;
        for (; i < n && found < 0; ++i)
          if (s_parent[i] == cur && s_tok[i] == best) found = i;
        if (found < 0) return c;
        take(found);
        best = -1;
      } else if (done) {
        return c;
      }
      done = true;
      c.op = kArgmax;
      c.node = cur;
      return c;
    }
    bool ask = false;
    for (; i < n && !ask; ++i) {
      if (s_parent[i] != cur) continue;
      bool ok;
      if (draft) {
        const double qc = s_q[i], w = (double)s_p[i] - a * qc;
        ok = s_tok[i] >= 0 && (double)s_u[i] * qc * z < (w > 0.0 ? w : 0.0);
      } else {
        bool again = false;  // a token one of its siblings already lost
        for (int k = 1; k < i; ++k) again |= s_parent[k] == cur && s_tok[k] == s_tok[i];
        const double pc = again ? 0.0 : (double)s_p[i];
        ok = s_tok[i] >= 0 && (double)s_u[i] * left < pc;
        if (!ok) left -= pc;
      }
      if (ok) {
        take(i);
      } else if (draft) {
        a += z;
        ask = true;
      }
    }
    if (!ask && summed) return c;  // the last pass was the last node's residual
    c.op = kSum;
    c.node = cur;
    c.a.h = (float)a;
    c.a.l = (float)(a - (double)c.a.h);
    return c;
  };

  for (;;) {
    if (rank == 0 && warp == 0) {
      const Cmd c = n > 0 ? advance() : Cmd{kExit, 0, {0.f, 0.f}};
      __syncwarp();
      if (lane < C) *cluster.map_shared_rank(&cmd, lane) = c;
    }
    cluster.sync();
    const Cmd c = cmd;
    if (c.op == kExit) break;
    const int W = C * WARPS, me = rank * WARPS + warp;
    int lo, hi;
    warp_part(p.V, me, W, &lo, &hi);
    const void *pr = row(p.target, p.ld_target, c.node);
    const void *qr = draft ? row(p.draft, p.ld_draft, c.node) : nullptr;
    constexpr uintptr_t kAlign = 4 * T::kBytes;
    const bool vec = reinterpret_cast<uintptr_t>(pr) % kAlign == 0 &&
                     (qr == nullptr || reinterpret_cast<uintptr_t>(qr) % kAlign == 0);
    if (c.op == kArgmax) {
      float m = -INFINITY;
      int at = INT32_MAX;
      for (int t = lo + 4 * lane; t < hi; t += 128) {
        float x[4];
        load4<T>(pr, t, vec && t + 4 <= hi, hi, x);
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (t + e < hi && (x[e] > m || (x[e] == m && at == INT32_MAX))) {
            m = x[e];
            at = t + e;
          }
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        const float om = __shfl_xor_sync(kFull, m, o);
        const int oa = __shfl_xor_sync(kFull, at, o);
        if (om > m || (om == m && oa < at)) {
          m = om;
          at = oa;
        }
      }
      if (lane == 0) {
        *cluster.map_shared_rank(&s_best[me], 0) = m;
        *cluster.map_shared_rank(&s_at[me], 0) = at;
      }
    } else {
      // (deterministic drafts) which of this node's children's tokens, all
      // refused, lie in this warp's part: their weight is 0
      const uint64_t lost = draft ? 0 : lost_in(s_parent, s_tok, c.node, lo, hi, lane);
      F2 s{0.f, 0.f};
      for (int t = lo + 4 * lane; t < hi; t += 128) {
        float x[4], y[4] = {0.f, 0.f, 0.f, 0.f};
        load4<T>(pr, t, vec && t + 4 <= hi, hi, x);
        if (draft) load4<T>(qr, t, vec && t + 4 <= hi, hi, y);
        for (uint64_t l = lost; l; l &= l - 1) {
          const int off = s_tok[__ffsll((long long)l) - 1] - t;
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (off == e) x[e] = 0.f;
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const F2 w = residual(x[e], y[e], c.a);
          const F2 r = two_sum(s.h, w.h);
          s.h = r.h;
          s.l = __fadd_rn(s.l, __fadd_rn(r.l, w.l));
        }
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        const F2 other{__shfl_xor_sync(kFull, s.h, o), __shfl_xor_sync(kFull, s.l, o)};
        s = f2_plus(s, other);
      }
      if (lane == 0) *cluster.map_shared_rank(&s_sum[me], 0) = f2_double(s);
    }
    cluster.sync();
    if (rank == 0 && warp == 0) {  // the pass's result, summed in a fixed order
      if (c.op == kArgmax) {
        float m = -INFINITY;
        int at = INT32_MAX;
        for (int k = lane; k < W; k += 32)
          if (s_best[k] > m || (s_best[k] == m && s_at[k] < at)) {
            m = s_best[k];
            at = s_at[k];
          }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
          const float om = __shfl_xor_sync(kFull, m, o);
          const int oa = __shfl_xor_sync(kFull, at, o);
          if (om > m || (om == m && oa < at)) {
            m = om;
            at = oa;
          }
        }
        best = at < p.V ? at : -1;  // -1: a row of NaN
      } else {
        double part = 0.0;
        for (int k = lane; k < W; k += 32) part += s_sum[k];
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) part += __shfl_xor_sync(kFull, part, o);
        z = part;
        summed = true;
      }
    }
  }
  if (rank != 0) return;

  // ---- the leader: the token after the walk, and the outputs ----
  int token = -1;
  if (n > 0 && !greedy) {
    if (warp == 0) {  // the warp part in which the partial sums pass u_0 times the total
      const int W = C * WARPS, per = (W + 31) / 32;
      const double thr = (double)s_u[0] * z;
      double own = 0.0;
      for (int k = lane * per; k < min(W, (lane + 1) * per); ++k) own += s_sum[k];
      double incl = own;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const double up = __shfl_up_sync(kFull, incl, o);
        if (lane >= o) incl += up;
      }
      // (rounding, or u_0 >= 1: the last part with any weight)
      const unsigned past = __ballot_sync(kFull, own > 0.0 && incl > thr), any = __ballot_sync(kFull, own > 0.0);
      const int who = past ? __ffs(past) - 1 : 31 - __clz(any);  // -1: no weight at all
      if (lane == 0) {
        s_hit = -1;
        s_node = cur;
        s_a = F2{(float)a, (float)(a - (double)(float)a)};
        s_thr = thr;
        s_first = INT32_MAX;
        s_last = -1;
      }
      __syncwarp();
      if (lane == who) {
        double run = incl - own;
        for (int k = lane * per; k < min(W, (lane + 1) * per); ++k) {
          if (s_sum[k] > 0.0) {
            s_hit = k;
            s_base = run;
            if (run + s_sum[k] > thr) break;
          }
          run += s_sum[k];
        }
      }
    }
    __syncthreads();
    if (s_hit >= 0) {
      int lo, hi;
      warp_part(p.V, s_hit, C * WARPS, &lo, &hi);
      const int node = s_node;
      const F2 ca = s_a;
      const double base = s_base, thr = s_thr;
      const void *pr = row(p.target, p.ld_target, node);
      const void *qr = draft ? row(p.draft, p.ld_draft, node) : nullptr;
      const uint64_t lost = draft ? 0 : lost_in(s_parent, s_tok, node, lo, hi, lane);
      const int per = (hi - lo + THREADS - 1) / THREADS;  // elements of a thread, consecutive
      const int t0 = min(hi, lo + tid * per), t1 = min(hi, t0 + per);
      auto weight = [&](int t) -> F2 {
        float x = load_scalar(T{}, pr, (size_t)t);
        for (uint64_t l = lost; l; l &= l - 1)
          if (s_tok[__ffsll((long long)l) - 1] == t) x = 0.f;
        return residual(x, draft ? load_scalar(T{}, qr, (size_t)t) : 0.f, ca);
      };
      F2 mine{0.f, 0.f};
      for (int t = t0; t < t1; ++t) {
        const F2 w = weight(t);
        if (__fadd_rn(w.h, w.l) > 0.f) atomicMax(&s_last, t);
        mine = f2_plus(mine, w);
      }
      F2 incl = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const F2 up{__shfl_up_sync(kFull, incl.h, o), __shfl_up_sync(kFull, incl.l, o)};
        if (lane >= o) incl = f2_plus(up, incl);
      }
      if (lane == 31) s_scan[warp] = incl;
      __syncthreads();
      F2 run{0.f, 0.f};  // the weights before this thread's
      for (int k = 0; k < warp; ++k) run = f2_plus(run, s_scan[k]);
      const F2 ex{__shfl_up_sync(kFull, incl.h, 1), __shfl_up_sync(kFull, incl.l, 1)};
      if (lane > 0) run = f2_plus(run, ex);
      if (base + f2_double(f2_plus(run, mine)) > thr) {
        for (int t = t0; t < t1; ++t) {
          const F2 w = weight(t);
          run = f2_plus(run, w);
          if (__fadd_rn(w.h, w.l) > 0.f && base + f2_double(run) > thr) {
            atomicMin(&s_first, t);
            break;
          }
        }
      }
      __syncthreads();
      token = s_first != INT32_MAX ? s_first : s_last;
    }
  } else if (n > 0) {
    token = best;  // (the leader's first warp holds it)
  }
  if (warp == 0) {
    const int m = n > 0 ? len : 0;
    for (int k = lane; k < p.n; k += 32) p.path[(int64_t)b * p.n + k] = k >= m ? -1 : (k == 0 ? 0 : s_path[k]);
    if (lane == 0) {
      p.path_len[b] = m;
      p.next_token[b] = token;
    }
  }
}

template <class T, int THREADS>
static cudaError_t launch_verify_t(const VerifyParams &p, int B, cudaStream_t stream) {
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = kMaxCluster;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)B * kMaxCluster);
  cfg.blockDim = dim3(THREADS);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = stream != nullptr ? 2 : 1;  // early launch on explicit streams only
  return cudaLaunchKernelEx(&cfg, tree_verify_kernel<T, THREADS>, p);
}

cudaError_t launch_tree_verify(const VerifyParams &p, int dtype, int B, cudaStream_t stream) {
  if (dtype == PKV_F32) return launch_verify_t<F32, 256>(p, B, stream);
  if (dtype == PKV_F16) return launch_verify_t<F16, 256>(p, B, stream);
  if (dtype == PKV_BF16) return launch_verify_t<BF16, 256>(p, B, stream);
  return cudaErrorNotSupported;
}

}  // namespace pkv
