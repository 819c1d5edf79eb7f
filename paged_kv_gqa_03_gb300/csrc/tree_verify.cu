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
// nodes at once.  So the kernel is a few dependent latencies plus one row pass
// per refusal: a cluster of 8 CTAs serves one sequence, each CTA a contiguous
// slice of the vocabulary, each warp a contiguous part of it.  CTA 0 gathers
// what the walk needs and hands it to the others through distributed shared
// memory; from then on every CTA walks by itself on the same numbers (the row
// sums, exchanged the same way, included), so that one cluster barrier per
// pass is all they share, and all of them reach the same ones whatever
// happens to the inputs meanwhile.  The CTA whose slice holds the drawn token
// finds it.
//
// Exactness.  A draw compares partial sums of up to V terms with u times the
// total; sums in 32 bits would move such a border by ~1e-7, and with it one
// token in some thousands.  The fp64 pipe of this GPU is far too narrow for V
// terms, so the sums and the walk's scalars are unevaluated pairs of floats
// (Knuth's two-sum, products by fma, ~46 bits), and the sum of max(p - a q, 0)
// is sum p - a sum q over the terms that are positive: 19 operations a term, about
// two thirds of the time the terms take to arrive from HBM.
//
// Measured (fp32 rows, device time): a chain of 6, V 32000 9 us (15 out of cold caches); 64 trees
// of 24, V 128000 46 - 54 us: every refusal reads 64 x 2 rows of 512 KB, the first from HBM (10 us),
// the next from L2 (8 us each); 16 trees of 16, greedy, 17 - 21 us (2 - 3 passes of ~4 us, each a
// round trip to memory, a cluster barrier and the join); 32 trees of 64 with deterministic
// drafts, V 50257, bf16, 12 - 14 us.  (The fp32 kernels spill 32 bytes at their 64 registers.)  1024 threads a CTA: chain 13.5 us, and fewer clusters fit
// side by side.
#include <cooperative_groups.h>

#include "common.cuh"
#include "internal.h"
#include "tree.h"

namespace pkv {

namespace cg = cooperative_groups;

namespace {

constexpr int kTree = PKV_MAX_Q_LEN;
constexpr int kCluster = 8;  // CTAs per sequence

// An unevaluated sum h + l of two floats, |l| <= ulp(h) / 2.
struct F2 {
  float h, l;
};
__device__ __forceinline__ F2 two_sum(float a, float b) {
  const float s = __fadd_rn(a, b), t = __fsub_rn(s, a);
  return {s, __fadd_rn(__fsub_rn(a, __fsub_rn(s, t)), __fsub_rn(b, t))};
}
__device__ __forceinline__ F2 renorm(float h, float l) {  // |h| >= |l|, or h = 0
  const float s = __fadd_rn(h, l);
  return {s, __fsub_rn(l, __fsub_rn(s, h))};
}
__device__ __forceinline__ F2 operator+(F2 a, F2 b) {
  const F2 s = two_sum(a.h, b.h), t = two_sum(a.l, b.l);
  const F2 r = renorm(s.h, __fadd_rn(s.l, t.h));
  return renorm(r.h, __fadd_rn(r.l, t.l));
}
__device__ __forceinline__ F2 operator-(F2 a, F2 b) { return a + F2{-b.h, -b.l}; }
__device__ __forceinline__ F2 operator*(F2 a, F2 b) {
  const float m = __fmul_rn(a.h, b.h);
  float e = __fmaf_rn(a.h, b.h, -m);
  e = __fmaf_rn(a.h, b.l, e);
  e = __fmaf_rn(a.l, b.h, e);
  return renorm(m, e);
}
__device__ __forceinline__ bool less(F2 a, F2 b) { return (b - a).h > 0.f; }

// A running sum hi + lo of floats.
struct Split {
  float hi, lo;
  __device__ __forceinline__ void add(float x) {
    const F2 r = two_sum(hi, x);
    hi = r.h;
    lo = __fadd_rn(lo, r.l);
  }
  __device__ __forceinline__ void add(Split o) {
    const F2 r = two_sum(hi, o.hi);
    hi = r.h;
    lo = __fadd_rn(__fadd_rn(lo, o.lo), r.l);
  }
  __device__ __forceinline__ F2 value() const { return renorm(hi, lo); }
};
// Sums over the terms p - a q that are positive.
struct Sums {
  Split p, q;
  __device__ __forceinline__ F2 value(F2 a) const { return p.value() - a * q.value(); }
};

enum : int { kExit = 0, kSum = 1, kArgmax = 2 };

struct Cmd {
  int op, node;
  F2 a;  // residual coefficient of the draft row
};

// What the walk of one sequence needs; the same in every CTA of its cluster.
struct Walk {
  uint64_t kids[kTree];  // a node's children
  uint64_t again;        // (deterministic drafts) nodes whose token an earlier sibling has
  uint64_t ok;           // nodes accepted if tried: all of them (deterministic drafts), or a node's first child
  float p[kTree], q[kTree], u[kTree];  // target's and draft's probability of the node's token; its number
  int tok[kTree];        // -1: outside the vocabulary
  int n, pad[3];
};
static_assert(sizeof(Walk) % 16 == 0, "copied in 16-byte words");

// p - a q where it is positive, rounded to fp32: its sign is exact to 2^-48 of p.
// (A NaN is not positive.)
__device__ __forceinline__ bool positive(float p, float q, F2 a) {
  return __fmaf_rn(-a.l, q, __fmaf_rn(-a.h, q, p)) > 0.f;
}

// Four neighbouring elements of a row as they are stored, element i first; those
// outside [lo, end) are 0.  One load where all four are inside and `vec` (i's
// address is a multiple of the four).
template <class T>
struct Quad {
  using Raw = uint2;
  Raw v;
  __device__ __forceinline__ void load(const void *row, int i, int lo, int end, bool vec) {
    const uint16_t *x = static_cast<const uint16_t *>(row);
    if (vec && i >= lo && i + 4 <= end) {
      v = *reinterpret_cast<const Raw *>(x + i);
    } else {
      uint32_t e[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) e[k] = i + k >= lo && i + k < end ? x[i + k] : 0u;
      v = make_uint2(e[0] | e[1] << 16, e[2] | e[3] << 16);
    }
  }
  __device__ __forceinline__ float4 get() const {
    const float2 a = unpack2(T{}, v.x), b = unpack2(T{}, v.y);
    return make_float4(a.x, a.y, b.x, b.y);
  }
};
template <>
struct Quad<F32> {
  using Raw = float4;
  Raw v;
  __device__ __forceinline__ void load(const void *row, int i, int lo, int end, bool vec) {
    const float *x = static_cast<const float *>(row);
    if (vec && i >= lo && i + 4 <= end) {
      v = *reinterpret_cast<const Raw *>(x + i);
    } else {
      v.x = i >= lo && i < end ? x[i] : 0.f;
      v.y = i + 1 >= lo && i + 1 < end ? x[i + 1] : 0.f;
      v.z = i + 2 >= lo && i + 2 < end ? x[i + 2] : 0.f;
      v.w = i + 3 >= lo && i + 3 < end ? x[i + 3] : 0.f;
    }
  }
  __device__ __forceinline__ float4 get() const { return v; }
};

}  // namespace

// The nodes of `kids`, as bits, whose token is in [lo, hi) (warp-wide).
__device__ __forceinline__ uint64_t lost_in(const Walk &w, uint64_t kids, int lo, int hi, int lane) {
  const bool l0 = ((kids >> lane) & 1) && w.tok[lane] >= lo && w.tok[lane] < hi;
  const bool l1 = ((kids >> (lane + 32)) & 1) && w.tok[lane + 32] >= lo && w.tok[lane + 32] < hi;
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
__global__ void __launch_bounds__(THREADS, 1024 / THREADS) tree_verify_kernel(const __grid_constant__ VerifyParams p) {
  constexpr int WARPS = THREADS / 32, C = kCluster;
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = (int)cluster.block_rank();
  const int b = blockIdx.x / C;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  __shared__ __align__(16) Walk walk;
  __shared__ Cmd cmd;
  __shared__ int s_path[kTree];
  // every warp's result of a pass, of the whole cluster; alternating between passes
  __shared__ __align__(16) float4 s_part[2][C * WARPS];
  __shared__ float4 s_scan[WARPS];
  __shared__ F2 s_base, s_thr;
  __shared__ Cmd s_draw;  // the last row pass
  __shared__ int s_hit, s_first, s_last;  // the final draw: the part, the first element past the border, the last with weight
  cluster.barrier_arrive();  // (shared memory of the others is written only after all of them run)
  grid_dep_wait();

  const bool draft = p.draft != nullptr, greedy = p.u == nullptr;
  auto row = [&](const void *base, int64_t ld, int node) {
    return static_cast<const void *>(static_cast<const uint8_t *>(base) + ((int64_t)b * p.n + node) * ld * T::kBytes);
  };
  if (rank == 0) {
    if (tid < kTree) walk.kids[tid] = 0;
    if (tid == kTree) walk.again = walk.ok = 0;
    __syncthreads();
    int up = -1, tok = -1;
    if (tid < kTree) {
      const int n = p.lens ? min(max(p.lens[b], 0), p.n) : p.n;
      if (tid < n) {
        const uint64_t below = p.mask[(int64_t)b * p.mask_stride + tid] & ((1ull << tid) - 1);
        const int64_t t = p.tokens[(int64_t)b * p.n + tid];
        up = below ? 63 - __clzll(below) : -1;
        tok = t >= 0 && t < p.V ? (int)t : -1;
      }
      const bool ask = up >= 0 && tok >= 0 && !greedy;
      walk.p[tid] = ask ? load_scalar(T{}, row(p.target, p.ld_target, up), (size_t)tok) : 0.f;
      walk.q[tid] = ask && draft ? load_scalar(T{}, row(p.draft, p.ld_draft, up), (size_t)tok) : 1.f;
      walk.u[tid] = !greedy && tid < n ? p.u[(int64_t)b * p.n + tid] : 0.f;
      walk.tok[tid] = tok;
      if (up >= 0) atomicOr(reinterpret_cast<unsigned long long *>(&walk.kids[up]), 1ull << tid);
      if (tid == 0) walk.n = n;
    }
    __syncthreads();
    if (!greedy && !draft) {
      if (up >= 0) {
        bool again = false;
        for (uint64_t k = walk.kids[up] & ((1ull << tid) - 1); k; k &= k - 1) again |= walk.tok[__ffsll((long long)k) - 1] == tok;
        if (again) atomicOr(reinterpret_cast<unsigned long long *>(&walk.again), 1ull << tid);
      }
      __syncthreads();
    }
    if (!greedy && up >= 0) {  // u q z < w (see the top of the file), as far as it is known without a row sum
      bool ok = tok >= 0;
      const F2 u{walk.u[tid], 0.f};
      if (draft) {
        ok &= less(u * F2{walk.q[tid], 0.f}, F2{walk.p[tid], 0.f});
      } else {
        F2 left{1.f, 0.f};
        for (uint64_t k = walk.kids[up] & ((1ull << tid) - 1) & ~walk.again; k; k &= k - 1)
          left = left - F2{walk.p[__ffsll((long long)k) - 1], 0.f};
        ok &= less(u * left, F2{(walk.again >> tid) & 1 ? 0.f : walk.p[tid], 0.f});
      }
      if (ok) atomicOr(reinterpret_cast<unsigned long long *>(&walk.ok), 1ull << tid);
    }
    __syncthreads();
    cluster.barrier_wait();
    constexpr int WORDS = (int)(sizeof(Walk) / 16);
    const uint4 *src = reinterpret_cast<const uint4 *>(&walk);
    for (int i = tid; i < WORDS * (C - 1); i += THREADS)
      reinterpret_cast<uint4 *>(cluster.map_shared_rank(&walk, 1 + i / WORDS))[i % WORDS] = src[i % WORDS];
  } else {
    cluster.barrier_wait();
  }
  cluster.sync();

  // ---- the walk (first warp of every CTA; every lane the same) ----
  const int n = walk.n;
  int cur = 0, len = 1, best = -1;
  uint64_t kids = walk.kids[0];  // cur's children not tried yet
  F2 a{0.f, 0.f}, z{1.f, 0.f};
  int last_pass = 0;  // its sums are the final draw's
  bool summed = false, seen = false, first = true;
  auto take = [&](int node) {
    cur = node;
    kids = walk.kids[node];
    if (lane == 0) s_path[len] = node;
    ++len;
    a = F2{0.f, 0.f};
    z = F2{1.f, 0.f};
    summed = seen = false;
    first = true;
  };
  // runs to the next row pass, or to the end (kExit)
  auto advance = [&]() -> Cmd {
    Cmd c{kExit, 0, {0.f, 0.f}};
    if (n == 0) return c;
    if (greedy) {
      if (seen) {  // cur's most likely token is known: is it drafted?
        const bool m0 = ((kids >> lane) & 1) && walk.tok[lane] == best, m1 = ((kids >> (lane + 32)) & 1) && walk.tok[lane + 32] == best;
        const uint64_t m = (uint64_t)__ballot_sync(kFull, m0) | (uint64_t)__ballot_sync(kFull, m1) << 32;
        if (best < 0 || m == 0) return c;
        take(__ffsll((long long)m) - 1);
      }
      c.op = kArgmax;
      c.node = cur;
      return c;
    }
    if (!draft) {
      for (uint64_t m; (m = kids & walk.ok) != 0;) take(__ffsll((long long)m) - 1);
    } else {
      bool ask = false;
      while (kids != 0 && !ask) {
        const int i = __ffsll((long long)kids) - 1;
        kids &= kids - 1;
        bool ok;
        if (first) {
          ok = (walk.ok >> i) & 1;
        } else {
          const F2 q{walk.q[i], 0.f}, w = F2{walk.p[i], 0.f} - a * q;
          ok = walk.tok[i] >= 0 && w.h > 0.f && less(F2{walk.u[i], 0.f} * q * z, w);
        }
        first = false;
        if (ok) {
          take(i);
        } else {
          a = a + z;
          ask = true;
        }
      }
      if (ask) summed = false;
    }
    if (summed) return c;  // the last pass was the last node's residual
    c.op = kSum;
    c.node = cur;
    c.a = a;
    return c;
  };

  const int me = rank * WARPS + warp;
  int lo, hi;  // this warp's part of the vocabulary
  warp_part(p.V, me, C * WARPS, &lo, &hi);
  // loads in flight per lane, of one row and of each of two: 8 are a warp's part of a vocabulary
  // of 128000 in one round trip to memory (what the registers allow for two fp32 rows is 4)
  constexpr int U1 = 8, U2 = T::kBytes == 4 ? 4 : 8;
  for (int pass = 0;; ++pass) {
    if (warp == 0) {
      const Cmd c = advance();
      if (lane == 0) {
        cmd = c;
        if (c.op != kExit) s_draw = c;
      }
    }
    __syncthreads();
    const Cmd c = cmd;
    if (c.op == kExit) break;
    const int par = pass & 1;
    const void *pr = row(p.target, p.ld_target, c.node);
    const void *qr = draft ? row(p.draft, p.ld_draft, c.node) : nullptr;
    // quads start where p's addresses are multiples of four elements (before lo, if need
    // be); q's are there too if its row has the same offset
    const int off = (int)(reinterpret_cast<uintptr_t>(pr) / T::kBytes + (unsigned)lo) & 3, from = lo - off + 4 * lane;
    const bool vec = ((reinterpret_cast<uintptr_t>(pr) - reinterpret_cast<uintptr_t>(qr)) / T::kBytes & 3) == 0;
    if (c.op == kArgmax) {
      float m = -INFINITY;
      int at = INT32_MAX;
      for (int t = from; t < hi; t += 128 * U1) {
        Quad<T> x[U1];
#pragma unroll
        for (int k = 0; k < U1; ++k) x[k].load(pr, t + 128 * k, lo, hi, true);
#pragma unroll
        for (int k = 0; k < U1; ++k) {
          const float4 v = x[k].get();
          const float f[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {  // (a lane's indexes grow: the first of equals stays)
            const int i = t + 128 * k + e;
            if (i >= lo && i < hi && (f[e] > m || (f[e] == m && at == INT32_MAX))) {
              m = f[e];
              at = i;
            }
          }
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
      if (lane < C) *cluster.map_shared_rank(&s_part[par][me], lane) = make_float4(m, __int_as_float(at), 0.f, 0.f);
    } else {
      // (deterministic drafts) this node's children's tokens in this warp's
      // part, all refused: their weight is 0
      const uint64_t lost = draft ? 0 : lost_in(walk, walk.kids[c.node], lo, hi, lane);
      Sums s{{0.f, 0.f}, {0.f, 0.f}};
      if (c.a.h == 0.f) {  // no refusal of a sampled draft: the weights are p, and q is not read
        for (int t = from; t < hi; t += 128 * U1) {
          Quad<T> x[U1];
#pragma unroll
          for (int k = 0; k < U1; ++k) x[k].load(pr, t + 128 * k, lo, hi, true);
#pragma unroll
          for (int k = 0; k < U1; ++k)
            if (t + 128 * k < hi) {
              const float4 v = x[k].get();
              float f[4] = {v.x, v.y, v.z, v.w};
              for (uint64_t l = lost; l; l &= l - 1) {
                const int tok = walk.tok[__ffsll((long long)l) - 1] - (t + 128 * k);
#pragma unroll
                for (int e = 0; e < 4; ++e)
                  if (e == tok) f[e] = 0.f;
              }
#pragma unroll
              for (int e = 0; e < 4; ++e) s.p.add(f[e] > 0.f ? f[e] : 0.f);
            }
        }
      } else {
        for (int t = from; t < hi; t += 128 * U2) {
          Quad<T> x[U2], y[U2];
#pragma unroll
          for (int k = 0; k < U2; ++k) {
            x[k].load(pr, t + 128 * k, lo, hi, true);
            y[k].load(qr, t + 128 * k, lo, hi, vec);
          }
#pragma unroll
          for (int k = 0; k < U2; ++k)
            if (t + 128 * k < hi) {
              const float4 v = x[k].get(), w = y[k].get();
              const float f[4] = {v.x, v.y, v.z, v.w}, g[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const bool pos = positive(f[e], g[e], c.a);
                s.p.add(pos ? f[e] : 0.f);
                s.q.add(pos ? g[e] : 0.f);
              }
            }
        }
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        s.p.add(Split{__shfl_xor_sync(kFull, s.p.hi, o), __shfl_xor_sync(kFull, s.p.lo, o)});
        s.q.add(Split{__shfl_xor_sync(kFull, s.q.hi, o), __shfl_xor_sync(kFull, s.q.lo, o)});
      }
      if (lane < C) *cluster.map_shared_rank(&s_part[par][me], lane) = make_float4(s.p.hi, s.p.lo, s.q.hi, s.q.lo);
    }
    cluster.sync();
    if (warp == 0) {  // every warp's results joined in a fixed order
      if (c.op == kArgmax) {
        float m = -INFINITY;
        int at = INT32_MAX;
        for (int k = lane; k < C * WARPS; k += 32) {
          const float om = s_part[par][k].x;
          const int oa = __float_as_int(s_part[par][k].y);
          if (om > m || (om == m && oa < at)) {
            m = om;
            at = oa;
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
        best = at < p.V ? at : -1;  // -1: a row of NaN
        seen = true;
      } else {
        Sums s{{0.f, 0.f}, {0.f, 0.f}};
        for (int k = lane; k < C * WARPS; k += 32) {
          const float4 v = s_part[par][k];
          s.p.add(Split{v.x, v.y});
          s.q.add(Split{v.z, v.w});
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
          s.p.add(Split{__shfl_xor_sync(kFull, s.p.hi, o), __shfl_xor_sync(kFull, s.p.lo, o)});
          s.q.add(Split{__shfl_xor_sync(kFull, s.q.hi, o), __shfl_xor_sync(kFull, s.q.lo, o)});
        }
        z = s.value(c.a);
        if (z.h < 0.f) z = F2{0.f, 0.f};
        summed = true;
        last_pass = pass;
      }
    }
  }

  // ---- the outputs (leader) and the token after the walk ----
  if (rank == 0 && warp == 0) {
    const int m = n > 0 ? len : 0;
    __syncwarp();
    for (int k = lane; k < p.n; k += 32) p.path[(int64_t)b * p.n + k] = k >= m ? -1 : (k == 0 ? 0 : s_path[k]);
    if (lane == 0) {
      p.path_len[b] = m;
      if (n == 0 || greedy) p.next_token[b] = n > 0 ? best : -1;
    }
  }
  if (n == 0 || greedy) return;
  const Cmd last = s_draw;
  if (warp == 0) {
    // the part (warp of the cluster) in which the sums pass the border u_0 z; by
    // rounding, or for u_0 >= 1, none may: then the last part with any weight
    constexpr int PER = C * WARPS / 32;  // consecutive parts of a lane
    const float4 *part = s_part[last_pass & 1];
    const F2 thr = F2{walk.u[0], 0.f} * z;
    auto sums = [&](int k) { return Sums{{part[k].x, part[k].y}, {part[k].z, part[k].w}}; };
    Sums own{{0.f, 0.f}, {0.f, 0.f}};
    bool any = false;
    for (int k = lane * PER; k < (lane + 1) * PER; ++k) {
      const Sums v = sums(k);
      any |= v.value(last.a).h > 0.f;
      own.p.add(v.p);
      own.q.add(v.q);
    }
    Sums incl = own;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const Split up{__shfl_up_sync(kFull, incl.p.hi, o), __shfl_up_sync(kFull, incl.p.lo, o)};
      const Split uq{__shfl_up_sync(kFull, incl.q.hi, o), __shfl_up_sync(kFull, incl.q.lo, o)};
      if (lane >= o) {
        incl.p.add(up);
        incl.q.add(uq);
      }
    }
    const unsigned past = __ballot_sync(kFull, any && less(thr, incl.value(last.a))), some = __ballot_sync(kFull, any);
    const int who = past ? __ffs(past) - 1 : 31 - __clz(some);  // -1: no weight at all
    if (lane == 0) {
      s_hit = -1;
      s_first = INT32_MAX;
      s_last = -1;
      if (who < 0 && rank == 0) p.next_token[b] = -1;
    }
    __syncwarp();
    if (lane == who) {
      Sums run = incl;  // the sums before this lane's parts
      run.p.add(Split{-own.p.hi, -own.p.lo});
      run.q.add(Split{-own.q.hi, -own.q.lo});
      int hit = -1;
      F2 base{0.f, 0.f};
      for (int k = lane * PER; k < (lane + 1) * PER; ++k) {
        const Sums v = sums(k);
        const F2 before = run.value(last.a);
        run.p.add(v.p);
        run.q.add(v.q);
        if (v.value(last.a).h > 0.f) {
          hit = k;
          base = before;
          if (less(thr, run.value(last.a))) break;
        }
      }
      if (hit / WARPS == rank) {  // this CTA holds the token
        s_hit = hit;
        s_base = base;
        s_thr = thr;
      }
    }
  }
  __syncthreads();
  if (s_hit < 0) return;
  warp_part(p.V, s_hit, C * WARPS, &lo, &hi);
  const F2 base = s_base, thr = s_thr;
  const void *pr = row(p.target, p.ld_target, last.node);
  const void *qr = last.a.h != 0.f ? row(p.draft, p.ld_draft, last.node) : nullptr;
  const uint64_t lost = draft ? 0 : lost_in(walk, walk.kids[last.node], lo, hi, lane);
  // each thread a run of consecutive elements: their sums, the sums before
  // them, and in the thread that passes the border the element that does
  const int per = (hi - lo + THREADS - 1) / THREADS;
  const int t0 = min(hi, lo + tid * per), t1 = min(hi, t0 + per);
  auto add = [&](Sums &s, int t) -> bool {
    float x = load_scalar(T{}, pr, (size_t)t);
    const float y = qr ? load_scalar(T{}, qr, (size_t)t) : 0.f;
    for (uint64_t l = lost; l; l &= l - 1)
      if (walk.tok[__ffsll((long long)l) - 1] == t) x = 0.f;
    const bool pos = positive(x, y, last.a);
    if (pos) {
      s.p.add(x);
      s.q.add(y);
    }
    return pos;
  };
  Sums mine{{0.f, 0.f}, {0.f, 0.f}};
  for (int t = t0; t < t1; ++t)
    if (add(mine, t)) atomicMax(&s_last, t);
  Sums incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const Split up{__shfl_up_sync(kFull, incl.p.hi, o), __shfl_up_sync(kFull, incl.p.lo, o)};
    const Split uq{__shfl_up_sync(kFull, incl.q.hi, o), __shfl_up_sync(kFull, incl.q.lo, o)};
    if (lane >= o) {
      incl.p.add(up);
      incl.q.add(uq);
    }
  }
  if (lane == 31) s_scan[warp] = make_float4(incl.p.hi, incl.p.lo, incl.q.hi, incl.q.lo);
  Sums run{{__shfl_up_sync(kFull, incl.p.hi, 1), __shfl_up_sync(kFull, incl.p.lo, 1)},
           {__shfl_up_sync(kFull, incl.q.hi, 1), __shfl_up_sync(kFull, incl.q.lo, 1)}};
  if (lane == 0) run = Sums{{0.f, 0.f}, {0.f, 0.f}};
  __syncthreads();
  for (int k = 0; k < warp; ++k) {
    run.p.add(Split{s_scan[k].x, s_scan[k].y});
    run.q.add(Split{s_scan[k].z, s_scan[k].w});
  }
  auto past = [&](const Sums &s) { return less(thr, base + s.value(last.a)); };
  Sums after = run;
  after.p.add(mine.p);
  after.q.add(mine.q);
  if (t0 < t1 && past(after)) {
    for (int t = t0; t < t1; ++t)
      if (add(run, t) && past(run)) {
        atomicMin(&s_first, t);
        break;
      }
  }
  __syncthreads();
  if (tid == 0) p.next_token[b] = s_first != INT32_MAX ? s_first : s_last;
}

template <class T, int THREADS>
static cudaError_t launch_verify_t(const VerifyParams &p, int B, cudaStream_t stream) {
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = kCluster;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)B * kCluster);
  cfg.blockDim = dim3(THREADS);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = stream != nullptr ? 2 : 1;  // early launch on explicit streams only
  return cudaLaunchKernelEx(&cfg, tree_verify_kernel<T, THREADS>, p);
}

// Threads per CTA: 512 while two CTAs per SM hold the batch's clusters side by
// side (a GPC has room for few clusters at one CTA per SM), else 256, four to an SM.
template <class T>
static cudaError_t launch_verify(const VerifyParams &p, int B, int sms, cudaStream_t stream) {
  return B * kCluster <= 2 * sms ? launch_verify_t<T, 512>(p, B, stream) : launch_verify_t<T, 256>(p, B, stream);
}

cudaError_t launch_tree_verify(const VerifyParams &p, int dtype, int B, int sms, cudaStream_t stream) {
  if (dtype == PKV_F32) return launch_verify<F32>(p, B, sms, stream);
  if (dtype == PKV_F16) return launch_verify<F16>(p, B, sms, stream);
  if (dtype == PKV_BF16) return launch_verify<BF16>(p, B, sms, stream);
  return cudaErrorNotSupported;
}

}  // namespace pkv
