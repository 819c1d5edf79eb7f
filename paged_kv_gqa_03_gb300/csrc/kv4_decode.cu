// kv4_decode.cu — decode attention over the 4-bit cache (kv4.cuh).
//
// The mathematics, the work split and the workspace are the decode kernel's
// (decode.cuh): units of 8 or 16 query rows of a (sequence, kv head), their
// blocks cut into equal ranges, one per warp, an online softmax per warp, and the
// split-KV merge.  What differs is what 4 bits change.
//
// Bound.  A token and kv head are 144 bytes (D = 128) for 256 elements to be
// widened, so at HBM speed an SM has 0.4 cycles an element: instructions, not bytes,
// are what to save.  Every element costs half a conversion (cvt.f16x2.e2m1x2) and half
// a multiplication by its scale, exact in f16 (2 + 4 significant bits), and feeds
// mma.sync m16n8k16 in f16 with 32-bit sums.
//  * A stage is NB = 4 blocks of one unit: one barrier, one record and one softmax
//    update (maximum exchange, rescale) for 64 tokens.
//  * A block's tile is one bulk copy, issued by the lane of its own block.
//  * K: a lane owns 32 consecutive elements (two scale groups) of rows gid and
//    gid + 8: one 16-byte load a row, the order of d within the contraction being free
//    (q's fragments are loaded in the same order).
//  * V: a lane owns 16 elements (D = 64: 8) of d for token pairs tig and tig + 4.  A
//    fragment pairs neighbouring tokens, so the two tokens' words are interleaved by
//    nibbles (a shift and a lop3 for 8 pairs) before the conversion.
//  * Blocks that every row of the unit sees whole take no mask.
//
// Weights.  exp2(x - m + 15): f16 then holds a weight to 11 bits down to 2^-29 of
// the largest and to 2^-39 at all; l sums the same numbers in 32 bits.  bf16 queries
// enter f16 scaled by a power of two per row (their largest element in [2^14, 2^15)).
//
// Not finite.  A group's NaN scale makes NaN of the scores, or of the output elements,
// of the rows that see the position, as the formula does, and of no others: hidden
// scores are selected away; in blocks that some row does not see whole, V scales of
// NaN are set to 0 and NaN is added to the rows that see them.
#include "decode.cuh"
#include "kv4.cuh"
#include "kv4.h"

namespace pkv {

template <class QT, int D_, int NH_, int WARPS_, int STAGES_, int NB_>
struct Kv4Cfg {
  using Q = QT;
  static constexpr int D = D_, NH = NH_, GC = 8 * NH_, WARPS = WARPS_, STAGES = STAGES_, NB = NB_;
  static constexpr int TILE = Kv4Tile<D>::kBytes;
  static constexpr int STAGE_BYTES = NB * TILE;
  static constexpr int KS = D / 16, MT = D / 16;
  static constexpr size_t TILES_BYTES = (size_t)WARPS * STAGES * STAGE_BYTES;
  static constexpr size_t META_BYTES = (size_t)WARPS * STAGES * 32;
  static constexpr size_t BAR_BYTES = (size_t)WARPS * STAGES * 8;
  static constexpr size_t SMEM = TILES_BYTES + META_BYTES + BAR_BYTES + (size_t)kInlinePrefix * 4;
  static_assert(SMEM <= 232448, "shared memory of a CTA");
};

struct Kv4Meta {
  int32_t b, hu, j, rem;  // first block, and the sequence's positions from it on
  int32_t flags, nb, bad; // bad: bit i: block i's id is out of range
  int32_t pad;
};

struct Kv4Producer {
  int pi, e, s;
  int b, hu, j, n, ctx, j0;
  int seg_j0, seg_wfirst;
  int win_b, win_j0, win_id, nxt_id;  // 32 block-table entries, a lane each, and the 32 after them
};

__device__ __forceinline__ void bulk_load(void *dst, const void *src, uint32_t bytes, uint64_t *bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                   smem_u32(dst)),
               "l"(reinterpret_cast<uint64_t>(src)), "r"(bytes), "r"(smem_u32(bar))
               : "memory");
}

__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ void load_seq(Kv4Producer &pr, const DecodeParams &p) {
  pr.ctx = clamped_len(p, __ldg(p.context_lens + pr.b));
  pr.n = (pr.ctx + kBlock - 1) / kBlock;
  pr.j0 = first_block<false>(p, pr.b, pr.ctx);
}

// Fills a stage with the next blocks (up to NB) of the worker's current unit.
template <class Cfg>
__device__ __forceinline__ int produce(Kv4Producer &pr, const Kv4Params &kp, uint8_t *tiles, Kv4Meta *meta,
                                       uint64_t *bars, int stage, int lane, int *cta_flags) {
  const DecodeParams &p = kp.d;
  __syncwarp();
  const int nb = min(Cfg::NB, min(pr.e - pr.pi, pr.n - pr.j));
  if (!(pr.b == pr.win_b && pr.j >= pr.win_j0 && pr.j + nb <= pr.win_j0 + 32)) {
    const int32_t *row = p.block_table + (size_t)pr.b * p.max_blocks;
    if (pr.b == pr.win_b && pr.j == pr.win_j0 + 32)
      pr.win_id = pr.nxt_id;
    else
      pr.win_id = pr.j + lane < pr.n ? __ldg(row + pr.j + lane) : 0;
    pr.win_b = pr.b;
    pr.win_j0 = pr.j;
    pr.nxt_id = pr.j + 32 + lane < pr.n ? __ldg(row + pr.j + 32 + lane) : 0;
  }
  int id = __shfl_sync(kFull, pr.win_id, (pr.j - pr.win_j0 + lane) & 31);
  const bool bad = lane < nb && (id < 0 || (int64_t)id >= p.num_blocks);
  if (bad) id = 0;  // read, and its values taken as zeros
  const uint32_t badmask = __ballot_sync(kFull, bad);
  int flags = 0;
  if (pr.pi == pr.s || pr.j == pr.j0) {
    flags |= kFirst;
    pr.seg_j0 = pr.j;
    pr.seg_wfirst = (pr.pi == pr.s);
  }
  const int jn = pr.j + nb;
  if (pr.pi + nb == pr.e || jn == pr.n) {
    flags |= kLast;
    if (pr.seg_j0 == pr.j0 && jn == pr.n) flags |= kComplete;
  }
  if (pr.seg_wfirst) flags |= kWFirst;
  if (lane == 0) {
    Kv4Meta m;
    m.b = pr.b;
    m.hu = pr.hu;
    m.j = pr.j;
    m.rem = pr.ctx - pr.j * kBlock;
    m.flags = flags;
    m.nb = nb;
    m.bad = (int)badmask;
    m.pad = 0;
    meta[stage] = m;
    if (badmask) atomicOr(cta_flags, PKV_FLAG_BAD_BLOCK);
    mbar_arrive_expect_tx(&bars[stage], nb * Cfg::TILE);
  }
  __syncwarp();
  if (lane < nb)
    bulk_load(tiles + (size_t)stage * Cfg::STAGE_BYTES + lane * Cfg::TILE,
              kp.cache + ((size_t)id * p.Hkv + pr.hu / p.NC) * Cfg::TILE, Cfg::TILE, &bars[stage]);
  pr.pi += nb;
  pr.j = jn;
  if (pr.j == pr.n && pr.pi < pr.e) {
    if (++pr.hu == p.HU) {
      pr.hu = 0;
      do {
        ++pr.b;
        load_seq(pr, p);
      } while (pr.n == 0 && pr.b < p.B - 1);
    }
    pr.j = pr.j0;
  }
  return nb;
}

template <class Cfg>
struct Kv4State {
  uint32_t qb[Cfg::NH][Cfg::KS][2];
  float acc[Cfg::NH][Cfg::MT][4];
  float m[Cfg::NH][2], l[Cfg::NH][2];  // of score columns 8 nh + 2 tig, + 1; m: largest raw score
  float sc[Cfg::NH][2];                // raw score -> log2 domain
  int back[Cfg::NH][2];
  int bk_lo, bk_hi;
};

template <class Cfg>
__device__ __forceinline__ void begin(Kv4State<Cfg> &st, const DecodeParams &p, const Kv4Meta &m, int lane) {
  const int gid = lane >> 2, tig = lane & 3;
  const int h = m.hu / p.NC, r0 = (m.hu % p.NC) * Cfg::GC;
  const int gc = min(Cfg::GC, p.R - r0);
  st.bk_lo = row_back(p, r0 + Cfg::GC - 1);
  st.bk_hi = row_back(p, r0);
  // a negative scale is the queries' sign, a scale of 0 a query of zeros
  const uint32_t flip = p.scale_log2 < 0.f ? 0x80008000u : 0u;
  const bool none = p.scale_log2 == 0.f;
#pragma unroll
  for (int nh = 0; nh < Cfg::NH; ++nh) {
    const int rq = 8 * nh + gid;
    const bool live = rq < gc && !none;
    const uint16_t *q = reinterpret_cast<const uint16_t *>(p.q) + (live ? query_row(p, m.b, h, r0 + rq) : 0) +
                        (Cfg::D / 4) * tig;
    uint2 raw[Cfg::KS];
#pragma unroll
    for (int ks = 0; ks < Cfg::KS; ++ks)
      raw[ks] = live ? *reinterpret_cast<const uint2 *>(q + 4 * ks) : make_uint2(0, 0);
    float down = 1.f;
    if constexpr (Cfg::Q::kCode == PKV_BF16) {
      uint32_t top = 0;
#pragma unroll
      for (int ks = 0; ks < Cfg::KS; ++ks)
        top = __vmaxu2(top, __vmaxu2(raw[ks].x & 0x7fff7fffu, raw[ks].y & 0x7fff7fffu));
      top = __vmaxu2(top, __shfl_xor_sync(kFull, top, 1));
      top = __vmaxu2(top, __shfl_xor_sync(kFull, top, 2));
      const int e = (int)(max(top & 0xffffu, top >> 16) >> 7);  // the largest element's exponent field
      const int f = e > 0 && e < 255 ? min(254 + 14 - e, 253) : 127;  // 2^(14 - exponent), as one
      const float up = __int_as_float(f << 23);
      down = __int_as_float((254 - f) << 23);
#pragma unroll
      for (int ks = 0; ks < Cfg::KS; ++ks) {
        const float2 a = unpack2(BF16{}, raw[ks].x), b = unpack2(BF16{}, raw[ks].y);
        raw[ks].x = pack_f16x2(a.x * up, a.y * up);
        raw[ks].y = pack_f16x2(b.x * up, b.y * up);
      }
    }
#pragma unroll
    for (int ks = 0; ks < Cfg::KS; ++ks) {
      st.qb[nh][ks][0] = raw[ks].x ^ flip;
      st.qb[nh][ks][1] = raw[ks].y ^ flip;
    }
    const float sc = none ? 1.f : fabsf(p.scale_log2);
    st.sc[nh][0] = sc * __shfl_sync(kFull, down, 8 * tig);  // rows 2 tig and 2 tig + 1: lanes of gid 2 tig, 2 tig + 1
    st.sc[nh][1] = sc * __shfl_sync(kFull, down, 8 * tig + 4);
    st.back[nh][0] = row_back(p, r0 + 8 * nh + 2 * tig);
    st.back[nh][1] = row_back(p, r0 + 8 * nh + 2 * tig + 1);
    st.m[nh][0] = st.m[nh][1] = -INFINITY;
    st.l[nh][0] = st.l[nh][1] = 0.f;
#pragma unroll
    for (int mt = 0; mt < Cfg::MT; ++mt)
#pragma unroll
      for (int r = 0; r < 4; ++r) st.acc[nh][mt][r] = 0.f;
  }
}

__device__ __forceinline__ uint32_t mul2(uint32_t a, __half2 s) {
  const __half2 r = __hmul2(*reinterpret_cast<const __half2 *>(&a), s);
  return *reinterpret_cast<const uint32_t *>(&r);
}
__device__ __forceinline__ __half2 scales2(uint32_t w) {  // two E4M3 bytes -> f16x2
  const uint32_t r = e4m3x2_to_f16x2((uint16_t)w);
  return *reinterpret_cast<const __half2 *>(&r);
}

// S^T = K . Q^T of one block's 16 tokens.
template <class Cfg>
__device__ __forceinline__ void scores(const Kv4State<Cfg> &st, uint32_t tile, int lane, bool zero,
                                       float (&s)[Cfg::NH][4]) {
  constexpr int W = Cfg::D / 32;  // words of a lane's run of a row
  uint32_t k[2][W];
  __half2 sc[2][2];               // scale of the run's first and second half, by row
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    if constexpr (Cfg::D == 128) {
      const uint4 v = lds128(tile + r * 512 + lane * 16);
      k[r][0] = v.x; k[r][1] = v.y; k[r][2] = v.z; k[r][3] = v.w;
      const __half2 two = scales2(zero ? 0u : lds16(tile + Kv4Tile<128>::kKScales + r * 64 + lane * 2));
      sc[r][0] = __half2half2(__low2half(two));
      sc[r][1] = __half2half2(__high2half(two));
    } else {
      const uint2 v = lds64(tile + r * 256 + lane * 8);
      k[r][0] = v.x; k[r][1] = v.y;
      // row gid's four scales are one word; the run's is byte tig
      const uint32_t w = lds32(tile + Kv4Tile<64>::kKScales + r * 32 + (lane & ~3));
      const __half2 two = scales2(zero ? 0u : (w >> (8 * (lane & 3))) & 0xffu);
      sc[r][0] = sc[r][1] = __half2half2(__low2half(two));
    }
  }
  float t[Cfg::NH][4];
  uint32_t x[2][4];
#pragma unroll
  for (int nh = 0; nh < Cfg::NH; ++nh)
#pragma unroll
    for (int i = 0; i < 4; ++i) s[nh][i] = t[nh][i] = 0.f;
#pragma unroll
  for (int ks = 0; ks < Cfg::KS; ++ks) {
    const int half = ks >= Cfg::KS / 2, by = 2 * (ks & 1);
    if (by == 0) {
      e2m1x8_to_f16(k[0][ks / 2], x[0]);
      e2m1x8_to_f16(k[1][ks / 2], x[1]);
    }
    uint32_t a[4];
    a[0] = mul2(x[0][by], sc[0][half]);
    a[1] = mul2(x[1][by], sc[1][half]);
    a[2] = mul2(x[0][by + 1], sc[0][half]);
    a[3] = mul2(x[1][by + 1], sc[1][half]);
#pragma unroll
    for (int nh = 0; nh < Cfg::NH; ++nh) {
      if (Cfg::NH == 1 && (ks & 1))  // two chains
        mma16816<false>(t[nh], a, st.qb[nh][ks][0], st.qb[nh][ks][1]);
      else
        mma16816<false>(s[nh], a, st.qb[nh][ks][0], st.qb[nh][ks][1]);
    }
  }
  if constexpr (Cfg::NH == 1)
#pragma unroll
    for (int i = 0; i < 4; ++i) s[0][i] += t[0][i];
}

// A block's V scales of the lane's tokens (pairs tig, tig + 4) and group; for a block that some row
// does not see whole, those past the context and those of NaN as 0, the latter's tokens noted.
template <class Cfg>
__device__ __forceinline__ void v_scales(uint32_t tile, int lane, bool zero, bool edge, int rem, uint32_t (&w)[2],
                                         uint32_t &spoiled) {
  const int gid = lane >> 2, tig = lane & 3;
  const int g = Cfg::D == 128 ? gid : gid >> 1;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    w[i] = zero ? 0u : lds16(tile + Kv4Tile<Cfg::D>::kVScales + (tig + 4 * i) * (Cfg::D / 8) + 2 * g);
    if (edge) {
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const int tok = 2 * tig + 8 * i + c;
        const uint32_t mask = 0xffu << (8 * c);
        if (tok >= rem) {
          w[i] &= ~mask;
        } else if (((w[i] >> (8 * c)) & 0x7fu) == 0x7fu) {
          w[i] &= ~mask;
          spoiled |= 1u << tok;
        }
      }
    }
  }
}

// O^T += V^T . P^T of one block.
template <class Cfg>
__device__ __forceinline__ void values(Kv4State<Cfg> &st, uint32_t tile, int lane, const uint32_t (&w)[2],
                                       const uint32_t (&pb)[Cfg::NH][2]) {
  const int gid = lane >> 2, tig = lane & 3;
  constexpr int NW = Cfg::D / 64;  // words of a token's run
  uint32_t lo[2][NW], hi[2][NW];   // nibbles of the pair's two tokens side by side: even and odd d
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int u = tig + 4 * i;
    uint32_t a[NW], b[NW];
    if constexpr (Cfg::D == 128) {
      const uint4 v = lds128(tile + Kv4Tile<128>::kVCodes + u * 128 + ((gid ^ (2 * (u & 3))) << 4));
      a[0] = v.x; a[1] = v.y; b[0] = v.z; b[1] = v.w;
    } else {
      const uint2 v = lds64(tile + Kv4Tile<64>::kVCodes + u * 64 + ((gid ^ (4 * ((u >> 1) & 1))) << 3));
      a[0] = v.x; b[0] = v.y;
    }
#pragma unroll
    for (int n = 0; n < NW; ++n) {
      lo[i][n] = (a[n] & 0x0f0f0f0fu) | ((b[n] << 4) & 0xf0f0f0f0u);
      hi[i][n] = ((a[n] >> 4) & 0x0f0f0f0fu) | (b[n] & 0xf0f0f0f0u);
    }
  }
  const __half2 s0 = scales2(w[0]), s1 = scales2(w[1]);
  uint32_t x[4][4];
#pragma unroll
  for (int mt = 0; mt < Cfg::MT; ++mt) {  // rows gid and gid + 8: d = run + 2 mt, 2 mt + 1
    if (mt % 4 == 0) {
      e2m1x8_to_f16(lo[0][mt / 4], x[0]);
      e2m1x8_to_f16(hi[0][mt / 4], x[1]);
      e2m1x8_to_f16(lo[1][mt / 4], x[2]);
      e2m1x8_to_f16(hi[1][mt / 4], x[3]);
    }
    uint32_t a[4];
    a[0] = mul2(x[0][mt % 4], s0);
    a[1] = mul2(x[1][mt % 4], s0);
    a[2] = mul2(x[2][mt % 4], s1);
    a[3] = mul2(x[3][mt % 4], s1);
#pragma unroll
    for (int nh = 0; nh < Cfg::NH; ++nh) mma16816<false>(st.acc[nh][mt], a, pb[nh][0], pb[nh][1]);
  }
}

constexpr float kWeightShift = 15.f;  // the largest weight is 2^15

template <class Cfg>
__device__ __forceinline__ void stage_step(Kv4State<Cfg> &st, const DecodeParams &p, const Kv4Meta &m, uint32_t tiles,
                                           int lane) {
  constexpr int NB = Cfg::NB, NH = Cfg::NH;
  const int gid = lane >> 2;
  float s[NB][NH][4];
#pragma unroll
  for (int i = 0; i < NB; ++i) {
    if (i < m.nb) {
      scores<Cfg>(st, tiles + i * Cfg::TILE, lane, (m.bad >> i) & 1, s[i]);
    } else {
#pragma unroll
      for (int nh = 0; nh < NH; ++nh)
#pragma unroll
        for (int c = 0; c < 4; ++c) s[i][nh][c] = -INFINITY;
    }
  }
  // every row of the unit sees every position of the stage
  const bool edge = m.rem - st.bk_hi < kBlock * m.nb || m.rem - st.bk_lo > p.wlen;
  const uint32_t wl = (uint32_t)p.wlen;
  uint32_t pb[NB][NH][2];
#pragma unroll
  for (int nh = 0; nh < NH; ++nh) {
    if (edge) {
      const int base0 = m.rem - st.back[nh][0] - p.wlen, base1 = m.rem - st.back[nh][1] - p.wlen;
#pragma unroll
      for (int i = 0; i < NB; ++i) {
        const int r = gid + kBlock * i;
        if ((uint32_t)(r - base0) >= wl) s[i][nh][0] = -INFINITY;
        if ((uint32_t)(r - base1) >= wl) s[i][nh][1] = -INFINITY;
        if ((uint32_t)(r + 8 - base0) >= wl) s[i][nh][2] = -INFINITY;
        if ((uint32_t)(r + 8 - base1) >= wl) s[i][nh][3] = -INFINITY;
      }
    }
    float mx0 = -INFINITY, mx1 = -INFINITY;
#pragma unroll
    for (int i = 0; i < NB; ++i) {
      mx0 = fmaxf(mx0, fmaxf(s[i][nh][0], s[i][nh][2]));
      mx1 = fmaxf(mx1, fmaxf(s[i][nh][1], s[i][nh][3]));
    }
    // exchange and rescale only when some lane holds a larger score
    if (__any_sync(kFull, (mx0 > st.m[nh][0]) | (mx1 > st.m[nh][1]))) {
#pragma unroll
      for (int off = 4; off < 32; off <<= 1) {
        mx0 = fmaxf(mx0, __shfl_xor_sync(kFull, mx0, off));
        mx1 = fmaxf(mx1, __shfl_xor_sync(kFull, mx1, off));
      }
      const float mn0 = fmaxf(st.m[nh][0], mx0), mn1 = fmaxf(st.m[nh][1], mx1);
      const float al0 = st.m[nh][0] == -INFINITY ? 0.f : exp2_fast((st.m[nh][0] - mn0) * st.sc[nh][0]);
      const float al1 = st.m[nh][1] == -INFINITY ? 0.f : exp2_fast((st.m[nh][1] - mn1) * st.sc[nh][1]);
      st.l[nh][0] *= al0;
      st.l[nh][1] *= al1;
      st.m[nh][0] = mn0;
      st.m[nh][1] = mn1;
#pragma unroll
      for (int mt = 0; mt < Cfg::MT; ++mt) {
        st.acc[nh][mt][0] *= al0;
        st.acc[nh][mt][1] *= al1;
        st.acc[nh][mt][2] *= al0;
        st.acc[nh][mt][3] *= al1;
      }
    }
    // (a column that has seen nothing: its scores are -inf, its weights 0)
    const float o0 = kWeightShift - (st.m[nh][0] == -INFINITY ? 0.f : st.m[nh][0] * st.sc[nh][0]);
    const float o1 = kWeightShift - (st.m[nh][1] == -INFINITY ? 0.f : st.m[nh][1] * st.sc[nh][1]);
#pragma unroll
    for (int i = 0; i < NB; ++i) {
      const float p0 = exp2_fast(fmaf(s[i][nh][0], st.sc[nh][0], o0)), p1 = exp2_fast(fmaf(s[i][nh][1], st.sc[nh][1], o1));
      const float p2 = exp2_fast(fmaf(s[i][nh][2], st.sc[nh][0], o0)), p3 = exp2_fast(fmaf(s[i][nh][3], st.sc[nh][1], o1));
      st.l[nh][0] += p0 + p2;
      st.l[nh][1] += p1 + p3;
      pb[i][nh][0] = movmatrix_trans(pack_f16x2(p0, p1));
      pb[i][nh][1] = movmatrix_trans(pack_f16x2(p2, p3));
    }
  }
#pragma unroll
  for (int i = 0; i < NB; ++i) {
    if (i < m.nb) {
      uint32_t w[2], spoiled = 0;
      v_scales<Cfg>(tiles + i * Cfg::TILE, lane, (m.bad >> i) & 1, edge, m.rem - kBlock * i, w, spoiled);
      values<Cfg>(st, tiles + i * Cfg::TILE, lane, w, pb[i]);
      if (edge && __any_sync(kFull, spoiled != 0)) {
        spoiled |= __shfl_xor_sync(kFull, spoiled, 1);  // the group's 16 tokens
        spoiled |= __shfl_xor_sync(kFull, spoiled, 2);
#pragma unroll
        for (int nh = 0; nh < NH; ++nh)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const int base = m.rem - kBlock * i - st.back[nh][c] - p.wlen;
            uint32_t sees = 0;
#pragma unroll 1
            for (int tok = 0; tok < kBlock; ++tok) sees |= (uint32_t)(tok - base) < wl ? 1u << tok : 0u;
            if (spoiled & sees)
#pragma unroll
              for (int mt = 0; mt < Cfg::MT; ++mt)
                st.acc[nh][mt][c] = st.acc[nh][mt][2 + c] = __int_as_float(0x7fc00000);
          }
      }
    }
  }
}

template <class Cfg>
__device__ __forceinline__ void finish(Kv4State<Cfg> &st, const Kv4Params &kp, const Kv4Meta &m, int w, int lane) {
  const DecodeParams &p = kp.d;
  const int gid = lane >> 2, tig = lane & 3;
  const int h = m.hu / p.NC, r0 = (m.hu % p.NC) * Cfg::GC;
  const int gc = min(Cfg::GC, p.R - r0);
  constexpr int RUN = Cfg::D / 8;  // a lane's run of d: RUN gid ..
  const size_t base = ((size_t)w * 2 + ((m.flags & kWFirst) ? 0 : 1)) * Cfg::GC;
#pragma unroll
  for (int nh = 0; nh < Cfg::NH; ++nh)
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      float l = st.l[nh][c];
#pragma unroll
      for (int off = 4; off < 32; off <<= 1) l += __shfl_xor_sync(kFull, l, off);
      const int row = 8 * nh + 2 * tig + c;
      if (row >= gc) continue;
      // a row that sees nothing gives 0; a sum of NaN gives NaN
      const float inv = l == 0.f ? 0.f : kp.v_unit / l;
      float y[RUN];
#pragma unroll
      for (int mt = 0; mt < Cfg::MT; ++mt) {
        y[2 * mt] = st.acc[nh][mt][c] * inv;
        y[2 * mt + 1] = st.acc[nh][mt][2 + c] * inv;
      }
      if (m.flags & kComplete) {
        uint16_t *o = reinterpret_cast<uint16_t *>(p.out) + query_row(p, m.b, h, r0 + row) + RUN * gid;
#pragma unroll
        for (int i = 0; i < RUN / 8; ++i)
          reinterpret_cast<uint4 *>(o)[i] = make_uint4(
              pack2(typename Cfg::Q{}, y[8 * i], y[8 * i + 1]), pack2(typename Cfg::Q{}, y[8 * i + 2], y[8 * i + 3]),
              pack2(typename Cfg::Q{}, y[8 * i + 4], y[8 * i + 5]), pack2(typename Cfg::Q{}, y[8 * i + 6], y[8 * i + 7]));
      } else {
        float4 *o = reinterpret_cast<float4 *>(p.part_o + (base + row) * Cfg::D + RUN * gid);
#pragma unroll
        for (int i = 0; i < RUN / 4; ++i) o[i] = make_float4(y[4 * i], y[4 * i + 1], y[4 * i + 2], y[4 * i + 3]);
        // (a sum of NaN as +inf: the merge then gives NaN)
        if (gid == 0)
          p.part_lse[base + row] = l != l ? INFINITY
                                   : l == 0.f ? -INFINITY : st.m[nh][c] * st.sc[nh][c] - kWeightShift + log2f(l);
      }
    }
}

template <class Cfg>
__global__ void __launch_bounds__(Cfg::WARPS * 32, 1) kv4_decode_kernel(const __grid_constant__ Kv4Params kp) {
  extern __shared__ __align__(128) uint8_t smem[];
  const DecodeParams &p = kp.d;
  const int lane = threadIdx.x & 31, wib = threadIdx.x >> 5;
  uint8_t *tiles = smem + (size_t)wib * Cfg::STAGES * Cfg::STAGE_BYTES;
  Kv4Meta *meta = reinterpret_cast<Kv4Meta *>(smem + Cfg::TILES_BYTES) + wib * Cfg::STAGES;
  uint64_t *bars = reinterpret_cast<uint64_t *>(smem + Cfg::TILES_BYTES + Cfg::META_BYTES) + wib * Cfg::STAGES;
  int32_t *s_prefix = reinterpret_cast<int32_t *>(smem + Cfg::TILES_BYTES + Cfg::META_BYTES + Cfg::BAR_BYTES);
  __shared__ int32_t s_scan[32];
  __shared__ int cta_flags;
  __shared__ __align__(8) uint64_t dead_bar;  // failure-path test hook: nothing ever arrives on it
  if (threadIdx.x == 0) cta_flags = 0;
  if (lane == 0) {
    for (int s = 0; s < Cfg::STAGES; ++s) mbar_init(&bars[s], 1);
    fence_barrier_init();
  }
  __syncthreads();
  grid_dep_wait();
  if (p.inline_plan) inline_plan<false>(p, s_prefix, s_scan, &cta_flags);

  const int w = blockIdx.x * Cfg::WARPS + wib;
  if (w < p.P) {
    int e;
    int4 st0;
    if (p.inline_plan) {
      st0 = locate<false>(p, s_prefix, w, &e);
    } else {
      st0 = p.starts[w];
      e = p.starts[w + 1].x;
    }
    const int total = e - st0.x;
    const bool stall = p.stall_ns != 0 && st0.x == 0 && total > 0;
    if (stall) {
      if (lane == 0) {
        mbar_init(&dead_bar, 1);
        fence_barrier_init();
      }
      __syncwarp();
    }
    if (total > 0) {
      Kv4Producer pr;
      pr.pi = pr.s = st0.x;
      pr.e = e;
      pr.b = st0.y;
      pr.hu = st0.z;
      pr.j = st0.w;
      pr.seg_j0 = pr.seg_wfirst = 0;
      pr.win_b = -1;
      pr.win_j0 = pr.win_id = pr.nxt_id = 0;
      load_seq(pr, p);
      int issued = 0, nst = 0;
      for (; nst < Cfg::STAGES && issued < total; ++nst)
        issued += produce<Cfg>(pr, kp, tiles, meta, bars, nst, lane, &cta_flags);
      Kv4State<Cfg> state;
      for (int done = 0, i = 0; done < total; ++i) {
        const int stage = i % Cfg::STAGES;
        const uint32_t parity = (uint32_t)(i / Cfg::STAGES) & 1u;
        if ((stall && i == 0) ? !mbar_wait_bounded(&dead_bar, 0, p.timeout_ns)
                              : !mbar_wait_bounded(&bars[stage], parity, p.timeout_ns)) {
          if (lane == 0) atomicOr(&cta_flags, PKV_FLAG_TIMEOUT);
          // let the copies still in flight land before the CTA's memory goes away
          for (int k = i; k < nst; ++k)
            mbar_wait_bounded(&bars[k % Cfg::STAGES], (uint32_t)(k / Cfg::STAGES) & 1u, p.timeout_ns);
          break;
        }
        const Kv4Meta m = meta[stage];
        if (m.flags & kFirst) begin<Cfg>(state, p, m, lane);
        stage_step<Cfg>(state, p, m, smem_u32(tiles + (size_t)stage * Cfg::STAGE_BYTES), lane);
        if (issued < total) {  // refilled once its fragments are consumed
          issued += produce<Cfg>(pr, kp, tiles, meta, bars, stage, lane, &cta_flags);
          ++nst;
        }
        if (m.flags & kLast) finish<Cfg>(state, kp, m, w, lane);
        done += m.nb;
      }
    }
  }
  __syncthreads();
  if (threadIdx.x == 0) p.cta_flags[blockIdx.x] = cta_flags;
  grid_dep_launch();
}

template <class Cfg>
static DecodeKernel kv4_entry() {
  DecodeKernel k;
  k.fn = reinterpret_cast<const void *>(&kv4_decode_kernel<Cfg>);
  k.mma = 1;
  k.cache_dtype = kKv4;
  k.q_dtype = Cfg::Q::kCode;
  k.D = Cfg::D;
  k.GC = Cfg::GC;
  k.warps = Cfg::WARPS;
  k.stages = Cfg::STAGES;
  k.smem_bytes = Cfg::SMEM;
  k.tree = 0;
  return k;
}

int register_decode_kv4(DecodeKernel *out) {
  int n = 0;
  out[n++] = kv4_entry<Kv4Cfg<BF16, 128, 1, 12, 2, 4>>();
  out[n++] = kv4_entry<Kv4Cfg<F16, 128, 1, 12, 2, 4>>();
  out[n++] = kv4_entry<Kv4Cfg<BF16, 64, 1, 12, 4, 4>>();
  out[n++] = kv4_entry<Kv4Cfg<F16, 64, 1, 12, 4, 4>>();
  out[n++] = kv4_entry<Kv4Cfg<BF16, 128, 2, 12, 4, 2>>();
  out[n++] = kv4_entry<Kv4Cfg<F16, 128, 2, 12, 4, 2>>();
  out[n++] = kv4_entry<Kv4Cfg<BF16, 64, 2, 12, 4, 4>>();
  out[n++] = kv4_entry<Kv4Cfg<F16, 64, 2, 12, 4, 4>>();
  return n;
}

}  // namespace pkv
