// kv4_decode.cu — decode attention over the 4-bit cache (kv4.cuh).
//
// The mathematics is the decode kernel's (decode.cuh): units of 8 or 16 query rows of a
// (sequence, kv head), an online softmax per warp, partial results joined by their log-sum-exp.
//
// Split.  A unit is 8 or 16 rows of hg = 4 (2, 1) neighbouring kv heads of a sequence, which are
// neighbours in the cache too: hg warps share a ring, one copy of hg tiles feeds them all, each takes its head's.  (The
// issue of copies bounds otherwise: a warp issues one in 220 cycles, four warps of an SM one in 85, so
// that copies of one tile reach 27 bytes a cycle out of L2 where 4-tile copies reach 70.)  The list
// of all units' blocks is cut into equal ranges, one per CTA, and a range into one per ring.
// What rings hold of one unit is joined in the CTA, through the rings' shared memory; a unit cut
// between CTAs leaves one partial result in each, which a merge kernel joins.  (Joined there ring by
// ring, a long context's 228 partial results a unit took the merge 53 us.)  A CTA's cut that falls into a unit of at
// most kKv4Whole blocks moves to the unit's nearer end: 2 us of work at most, where the merge launch
// costs 3 to 5; with no longer table it is not launched at all.
//
// Bound.  A token and kv head are 144 bytes (D = 128) for 256 elements to be
// widened, so at HBM speed an SM has 0.4 cycles an element: instructions, not bytes,
// are what to save.  Every element costs half a conversion (cvt.f16x2.e2m1x2) and half
// a multiplication by its scale, exact in f16 (2 + 4 significant bits), and feeds
// mma.sync m16n8k16 in f16 with 32-bit sums.
//  * A stage is NB = 4 blocks of one unit: one barrier, one record and one softmax
//    update (maximum exchange, rescale) for 64 tokens.
//  * Four producer warps fill the rings, a lane each: the walk over units and table entries and the copies
//    then cost the consumers nothing; they were 80 instructions a block.  (16-byte cp.async by the consumers
//    reaches HBM speed later, 4.3 TB/s while the rings fill.)
//  * K: a lane owns 32 consecutive elements (two scale groups) of rows gid and
//    gid + 8: one 16-byte load a row, the order of d within the contraction being free
//    (q's fragments are loaded in the same order).
//  * V: a lane owns 16 elements (D = 64: 8) of d for token pairs tig and tig + 4.  A
//    fragment pairs neighbouring tokens, and so do the cache's bytes: one conversion is one
//    register of the fragment.
//  * Blocks that every row of the unit sees whole take no mask.
//
// Measured, cold inputs, 64 / 8 heads of 128, bf16: 64 x 8192 (604 MB) 118 us, 5.1 TB/s; another 64 sequences cost
// 91 us, 6.6 TB/s; the rest is the launch and first fills (~10 us), the last units' imbalance and the merge (~9).
// 1 x 131072 48 us; 1 x 333 14 us, of which 8 until the first tile has landed.  16-row units, 32 / 8 heads,
// 4 new tokens, 16 x 1000-32768: 90 us; more rows widen the codes again, 16 rows at a time: 16 x 8192, 64 / 8 heads,
// 1, 2, 4, 8 new tokens (8 to 64 rows a kv head) 43, 55, 85, 144 us.  16-row units of D = 128 issue 0.44 instructions a
// clock from two warps a scheduler, the tensor pipe active for a third of the time: bound by waits, of dependent
// instructions first.  D = 64 costs the instructions of a softmax on half the bytes: 64 x 8192, 32 / 8 heads (302 MB)
// 79 us.
//
// Weights.  exp2((s - m) * c + 15), s a raw score, m the largest, c its factor (scale and units): the difference comes
// first, so that the largest weight is 2^15 exactly, however large the scores; what is joined goes by the same
// differences of raw maxima, next to sums that are not turned into logarithms.  f16 then holds a weight to 11 bits
// down to 2^-29 of the largest and to 2^-39 at all.  l sums the weights in 32 bits before they are rounded to f16: a
// weight counts by up to 2^-11 of itself differently above and below.  bf16 queries enter f16 scaled by a power of two
// per row (their largest element in [2^14, 2^15)).
//
// Not finite.  A group's NaN scale makes NaN of the scores, or of the output elements,
// of the rows that see the position, as the formula does, and of no others: hidden
// scores are selected away; in blocks that some row does not see whole, V scales of
// NaN are set to 0 and NaN is added to the rows that see them.
#include <cfloat>

#include "decode.cuh"
#include "kv4.cuh"
#include "kv4.h"

namespace pkv {

// WARPS_ consumer warps (a multiple of 4), rings of STAGES_ stages of NB_ blocks (per head of a unit), and four
// producer warps.  Registers: the launch's even share, moved to the consumers.
template <class QT, int D_, int NH_, int WARPS_, int STAGES_, int NB_>
struct Kv4Cfg {
  using Q = QT;
  static constexpr int D = D_, NH = NH_, GC = 8 * NH_, WARPS = WARPS_, STAGES = STAGES_, NB = NB_;
  static constexpr int THREADS = (WARPS + 4) * 32;
  static constexpr int REGS_LAUNCH = 65536 / THREADS / 8 * 8;
  static constexpr int REGS_PRODUCER = 56;
  static constexpr int REGS_CONSUMER = REGS_LAUNCH + (REGS_LAUNCH - REGS_PRODUCER) * 4 / WARPS / 8 * 8;
  static_assert(WARPS % 4 == 0, "warpgroups");
  static_assert(REGS_CONSUMER * WARPS + REGS_PRODUCER * 4 <= REGS_LAUNCH * (WARPS + 4), "registers of the launch");
  static constexpr int TILE = Kv4Tile<D>::kBytes;
  static constexpr int STAGE_BYTES = NB * TILE;
  static constexpr int KS = D / 16, MT = D / 16;
  // A whole stage at a context's or window's end takes masks in one go (in 16-row units, whose registers that
  // costs: 16 x 1000-32768, 4 new 92.6 -> 98.5 us, it goes block by block).
  static constexpr bool kWholeEdges = NH == 1;
  static constexpr size_t TILES_BYTES = (size_t)WARPS * STAGES * STAGE_BYTES;
  static constexpr size_t META_BYTES = (size_t)WARPS * STAGES * 16;
  static constexpr size_t BAR_BYTES = (size_t)WARPS * STAGES * 16;  // full, empty
  static constexpr size_t SMEM = TILES_BYTES + META_BYTES + BAR_BYTES + (size_t)kKv4Prefix * 4;
  static_assert(SMEM + WARPS * (16 * GC + 256) + 1024 <= 232448, "shared memory of a CTA");
};

// Short ranges spend most of their time on instructions that are fetched for the first time (a small call's warps
// issue for one cycle in six and wait for instructions the others), so what runs once is kept short: one copy of
// each part, no division where the common shapes need none.
struct UnitAt {
  int head, row;  // first kv head and first query row
};
__device__ __forceinline__ UnitAt unit_at(const Kv4Params &kp, int hu, int GC) {
  if (kp.d.NC == 1) return UnitAt{hu << kp.hg_log2, 0};
  const int g = hu / kp.d.NC;
  return UnitAt{g << kp.hg_log2, (hu - g * kp.d.NC) * GC};
}
// Query row r of kv head h of sequence b, in elements of q / out; positions hidden from it at the end.
__device__ __forceinline__ size_t row_at(const DecodeParams &p, int b, int h, int r) {
  const int i = p.q_len == 1 ? 0 : r / p.G;
  return ((size_t)((b * p.q_len + i) * p.Hq + h * p.G + (r - i * p.G))) * (size_t)p.D;  // (fewer than 2^31 rows)
}
__device__ __forceinline__ int hidden_behind(const DecodeParams &p, int r) { return p.q_len == 1 ? 0 : row_back(p, r); }

// (beside kFirst, kLast of decode.cuh)
constexpr int32_t kOpens = 4;   // the segment begins with the unit's first block
constexpr int32_t kCloses = 8;  // it ends with its last
constexpr int32_t kEnds = 16;   // the worker's last segment

constexpr int kPollNs = 100;   // between a producer's looks at rings that are all full

constexpr int kMinItems = 24;  // blocks (of a head each) of a CTA's range, at least

// A stage's record: its unit, the sequence's positions from its first block on, and
// flags | blocks << 8 | (bit i: block i's id is out of range) << 16.
struct __align__(16) Kv4Meta {
  int32_t b, hu, rem, flags;
  __device__ __forceinline__ int nb() const { return (flags >> 8) & 0xff; }
  __device__ __forceinline__ uint32_t bad() const { return (uint32_t)flags >> 16; }
};

__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ void bulk_load(void *dst, const void *src, uint32_t bytes, uint64_t *bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                   smem_u32(dst)),
               "l"(reinterpret_cast<uint64_t>(src)), "r"(bytes), "r"(smem_u32(bar))
               : "memory");
}
__device__ __forceinline__ void mbar_arrive(uint64_t *bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}
__device__ __forceinline__ bool mbar_test(uint64_t *bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n .reg .pred p;\n"
      " mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n"
      " selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}
__device__ __forceinline__ void cp_async4(uint32_t dst, const void *src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_wait() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// A producer lane: walks the range of items [pi, e) of its ring's consumer.
// Table entries come through shared memory, 64 a ring: windows k (entries 32 k ..) of the current sequence, k even and odd,
// fetched by the whole warp with cp.async, the next one ahead (a register load by one lane would hold up
// the other lanes' fills for its latency).
template <int NB>
struct Kv4Producer {
  int pi, e, s;
  int b, hu, j, n, ctx, j0;
  int opens;             // kOpens of the current segment
  int tag_b, tag0, tag1;  // the windows that are there or on their way; ready: bit per window
  uint32_t ready;

  __device__ __forceinline__ void load_seq(const DecodeParams &p) {
    ctx = clamped_len(p, __ldg(p.context_lens + b));
    n = (ctx + kBlock - 1) / kBlock;
    j0 = first_block<false>(p, b, ctx);
  }
  __device__ __forceinline__ int blocks() const { return min(NB, min(e - pi, n - j)); }
  __device__ __forceinline__ bool has(int k) const { return tag_b == b && ((k & 1) ? tag1 : tag0) == k; }
  // Window k of the current sequence will be there.
  __device__ __forceinline__ void expect(int k) {
    if (tag_b != b) tag0 = tag1 = -1, ready = 0;
    tag_b = b;
    if (k & 1)
      tag1 = k;
    else
      tag0 = k;
    ready &= ~(1u << (k & 1));
  }
  // Fills a stage with the next blocks (up to NB) of the current unit.
  template <class Cfg>
  __device__ __forceinline__ void fill(const Kv4Params &kp, const int32_t *ids, uint8_t *tiles, Kv4Meta *meta,
                                       uint64_t *full, int *cta_flags) {
    const DecodeParams &p = kp.d;
    const int nb = blocks();
    int flags = nb << 8;
    if (pi == s || j == j0) {
      flags |= kFirst;
      opens = j == j0 ? kOpens : 0;
    }
    flags |= opens;
    const int jn = j + nb;
    if (pi + nb == e) flags |= kLast | kEnds;
    if (jn == n) flags |= kLast | kCloses;
    const int bytes = Cfg::TILE << kp.hg_log2;  // a block's tiles of the unit's heads
    const uint8_t *head = kp.cache + (size_t)unit_at(kp, hu, 0).head * Cfg::TILE;
    // (a bad id: block 0 is read, and its values taken as zeros)
    auto good = [&](int i) { return (uint64_t)(int64_t)ids[(j + i) & 63] < (uint64_t)p.num_blocks; };
#pragma unroll
    for (int i = 0; i < NB; ++i)
      if (i < nb && !good(i)) flags |= 0x10000 << i;
    if (flags >> 16) atomicOr(cta_flags, PKV_FLAG_BAD_BLOCK);
    *meta = Kv4Meta{b, hu, ctx - j * kBlock, flags};
    mbar_arrive_expect_tx(full, nb * bytes);
#pragma unroll 1
    for (int i = 0; i < nb; ++i)
      bulk_load(tiles + i * bytes, head + (size_t)(good(i) ? ids[(j + i) & 63] : 0) * p.Hkv * Cfg::TILE, bytes, full);
    pi += nb;
    j = jn;
    if (pi < e && j == n) {
      if (++hu == p.HU) {
        hu = 0;
        do {
          ++b;
          load_seq(p);
        } while (n == 0 && b < p.B - 1);
      }
      j = j0;
    }
  }
};

template <class Cfg>
struct Kv4State {
  uint32_t qb[Cfg::NH][Cfg::KS][2];
  float acc[Cfg::NH][Cfg::MT][4];
  float m[Cfg::NH][2], l[Cfg::NH][2];  // of score columns 8 nh + 2 tig, + 1; m: largest raw score
  float sc[Cfg::NH][2], at[Cfg::NH][2];  // weight = 2^((raw score + at) * sc + kWeightShift); at: -m, or 0 while m is -inf
  int back[Cfg::NH][2];
  int bk_lo, bk_hi;
};

template <class Cfg>
__device__ __forceinline__ void begin(Kv4State<Cfg> &st, const Kv4Params &kp, int b, int hu, int sub, int lane) {
  const DecodeParams &p = kp.d;
  const int gid = lane >> 2, tig = lane & 3;
  const UnitAt u = unit_at(kp, hu, Cfg::GC);
  const int h = u.head + sub, r0 = u.row;
  const int gc = min(Cfg::GC, p.R - r0);
  st.bk_lo = hidden_behind(p, r0 + Cfg::GC - 1);
  st.bk_hi = hidden_behind(p, r0);
  // a negative scale is the queries' sign, a scale of 0 a query of zeros
  const uint32_t flip = p.scale_log2 < 0.f ? 0x80008000u : 0u;
  const bool none = p.scale_log2 == 0.f;
#pragma unroll
  for (int nh = 0; nh < Cfg::NH; ++nh) {
    const int rq = 8 * nh + gid;
    const bool live = rq < gc && !none;
    const uint16_t *q = reinterpret_cast<const uint16_t *>(p.q) + (live ? row_at(p, b, h, r0 + rq) : 0) +
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
    // Within the normal numbers: a product of 0 would make NaN of a hidden score's -inf, one of inf of a difference of 0.
    // (Raw scores differ by less than 2^36 and, where they do, by 2^-34 or more: the weights are those of the product.)
    st.sc[nh][0] = fminf(fmaxf(sc * __shfl_sync(kFull, down, 8 * tig), FLT_MIN), FLT_MAX);  // rows 2 tig and 2 tig + 1:
    st.sc[nh][1] = fminf(fmaxf(sc * __shfl_sync(kFull, down, 8 * tig + 4), FLT_MIN), FLT_MAX);  // lanes of gid 2 tig, ..
    st.back[nh][0] = hidden_behind(p, r0 + 8 * nh + 2 * tig);
    st.back[nh][1] = hidden_behind(p, r0 + 8 * nh + 2 * tig + 1);
    st.m[nh][0] = st.m[nh][1] = -INFINITY;
    st.l[nh][0] = st.l[nh][1] = st.at[nh][0] = st.at[nh][1] = 0.f;
#pragma unroll
    for (int mt = 0; mt < Cfg::MT; ++mt)
#pragma unroll
      for (int r = 0; r < 4; ++r) st.acc[nh][mt][r] = 0.f;
  }
}

// mma16816<false> onto 0.
__device__ __forceinline__ void mma16816_zero(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%10,%10,%10,%10};"
      : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
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
__device__ __forceinline__ void scores(const Kv4State<Cfg> &st, uint32_t tile, int lane, float (&s)[Cfg::NH][4]) {
  constexpr int W = Cfg::D / 32;  // words of a lane's run of a row
  uint32_t k[2][W], x[2][4];
  __half2 sc[2][2];               // scale of the run's first and second half, by row
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    if constexpr (Cfg::D == 128) {
      const uint4 v = lds128(tile + r * 512 + lane * 16);
      k[r][0] = v.x; k[r][1] = v.y; k[r][2] = v.z; k[r][3] = v.w;
      const __half2 two = scales2(lds16(tile + Kv4Tile<128>::kKScales + r * 64 + lane * 2));
      sc[r][0] = __half2half2(__low2half(two));
      sc[r][1] = __half2half2(__high2half(two));
    } else {
      const uint2 v = lds64(tile + r * 256 + lane * 8);
      k[r][0] = v.x; k[r][1] = v.y;
      // row gid's four scales are one word; the run's is byte tig
      const uint32_t w = lds32(tile + Kv4Tile<64>::kKScales + r * 32 + (lane & ~3));
      const __half2 two = scales2((w >> (8 * (lane & 3))) & 0xffu);
      sc[r][0] = sc[r][1] = __half2half2(__low2half(two));
    }
  }
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
      if (ks == 0)
        mma16816_zero(s[nh], a, st.qb[nh][ks][0], st.qb[nh][ks][1]);
      else
        mma16816<false>(s[nh], a, st.qb[nh][ks][0], st.qb[nh][ks][1]);
    }
  }
}

// A block's V scales of the lane's tokens (pairs tig, tig + 4) and group.
template <class Cfg>
__device__ __forceinline__ void v_scales(uint32_t tile, int lane, uint32_t (&w)[2]) {
  const int gid = lane >> 2, tig = lane & 3;
  const int g = Cfg::D == 128 ? gid : gid >> 1;
#pragma unroll
  for (int i = 0; i < 2; ++i) w[i] = lds16(tile + Kv4Tile<Cfg::D>::kVScales + (tig + 4 * i) * (Cfg::D / 8) + 2 * g);
}
// Those past the context (rem positions are left) as 0, those of NaN too and their tokens noted.
__device__ __forceinline__ uint32_t clean_scales(uint32_t (&w)[2], int lane, int rem) {
  uint32_t spoiled = 0;
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const int tok = 2 * (lane & 3) + 8 * i + c;
      const uint32_t mask = 0xffu << (8 * c);
      if (tok >= rem) {
        w[i] &= ~mask;
      } else if (((w[i] >> (8 * c)) & 0x7fu) == 0x7fu) {
        w[i] &= ~mask;
        spoiled |= 1u << tok;
      }
    }
  return spoiled;
}

// O^T += V^T . P^T of one block.
template <class Cfg>
__device__ __forceinline__ void values(Kv4State<Cfg> &st, uint32_t tile, int lane, const uint32_t (&w)[2],
                                       const uint32_t (&pb)[Cfg::NH][2]) {
  const int gid = lane >> 2, tig = lane & 3;
  constexpr int NW = Cfg::D / 32;  // words of a pair's run
  uint32_t c[2][NW], x[2][4];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int u = tig + 4 * i;
    if constexpr (Cfg::D == 128) {
      const uint4 v = lds128(tile + Kv4Tile<128>::kVCodes + u * 128 + ((gid ^ (2 * (u & 3))) << 4));
      c[i][0] = v.x; c[i][1] = v.y; c[i][2] = v.z; c[i][3] = v.w;
    } else {
      const uint2 v = lds64(tile + Kv4Tile<64>::kVCodes + u * 64 + ((gid ^ (4 * ((u >> 1) & 1))) << 3));
      c[i][0] = v.x; c[i][1] = v.y;
    }
  }
  const __half2 s0 = scales2(w[0]), s1 = scales2(w[1]);
#pragma unroll
  for (int mt = 0; mt < Cfg::MT; ++mt) {  // rows gid and gid + 8: d = run + 2 mt, 2 mt + 1
    const int by = 2 * (mt & 1);
    if (by == 0) {
      e2m1x8_to_f16(c[0][mt / 2], x[0]);
      e2m1x8_to_f16(c[1][mt / 2], x[1]);
    }
    uint32_t a[4];
    a[0] = mul2(x[0][by], s0);
    a[1] = mul2(x[0][by + 1], s0);
    a[2] = mul2(x[1][by], s1);
    a[3] = mul2(x[1][by + 1], s1);
#pragma unroll
    for (int nh = 0; nh < Cfg::NH; ++nh) mma16816<false>(st.acc[nh][mt], a, pb[nh][0], pb[nh][1]);
  }
}

constexpr float kWeightShift = 15.f;  // the largest weight is 2^15

// (s + at) * sc + kWeightShift of two columns, in packed instructions (64 x 8192, 32 / 8 heads of 64: 79.2 us, one by one
// 81.5; 16 x 8192, 4 new, 64 / 8 heads of 128: 84.6 and 85.8).
__device__ __forceinline__ float2 exponents(float2 s, float2 at, float2 sc) {
  return __ffma2_rn(__fadd2_rn(s, at), sc, make_float2(kWeightShift, kWeightShift));
}

// NaN into the rows that see a token of `spoiled` (the lane's tokens of NaN scales in a block), in the lane's run of d.
template <class Cfg>
__device__ __forceinline__ void spoil(Kv4State<Cfg> &st, const DecodeParams &p, int rem, uint32_t spoiled) {
  spoiled |= __shfl_xor_sync(kFull, spoiled, 1);  // the group's 16 tokens
  spoiled |= __shfl_xor_sync(kFull, spoiled, 2);
#pragma unroll
  for (int nh = 0; nh < Cfg::NH; ++nh)
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const int base = rem - st.back[nh][c] - p.wlen;
      uint32_t sees = 0;
#pragma unroll 1
      for (int tok = 0; tok < kBlock; ++tok) sees |= (uint32_t)(tok - base) < (uint32_t)p.wlen ? 1u << tok : 0u;
      if (spoiled & sees)
#pragma unroll
        for (int mt = 0; mt < Cfg::MT; ++mt) st.acc[nh][mt][c] = st.acc[nh][mt][2 + c] = __int_as_float(0x7fc00000);
    }
}

// The running maximum and sum of one 8-row group over n blocks' raw scores, and the weights as B operands.
template <class Cfg, int N>
__device__ __forceinline__ void softmax(Kv4State<Cfg> &st, int nh, const float (&s)[N][Cfg::NH][4],
                                        uint32_t (&pb)[N][Cfg::NH][2]) {
  float mx0 = -INFINITY, mx1 = -INFINITY;
#pragma unroll
  for (int i = 0; i < N; ++i) {
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
    // (a column that has seen nothing: its scores are -inf, its weights 0)
    st.at[nh][0] = mn0 == -INFINITY ? 0.f : -mn0;
    st.at[nh][1] = mn1 == -INFINITY ? 0.f : -mn1;
  }
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const float2 at = make_float2(st.at[nh][0], st.at[nh][1]), sc = make_float2(st.sc[nh][0], st.sc[nh][1]);
    const float2 x = exponents(make_float2(s[i][nh][0], s[i][nh][1]), at, sc);
    const float2 y = exponents(make_float2(s[i][nh][2], s[i][nh][3]), at, sc);
    const float p0 = exp2_fast(x.x), p1 = exp2_fast(x.y), p2 = exp2_fast(y.x), p3 = exp2_fast(y.y);
    st.l[nh][0] += p0 + p2;
    st.l[nh][1] += p1 + p3;
    pb[i][nh][0] = movmatrix_trans(pack_f16x2(p0, p1));
    pb[i][nh][1] = movmatrix_trans(pack_f16x2(p2, p3));
  }
}

// A whole stage.  `edge`: some row of the unit does not see all of it (a context's or a window's end).
template <class Cfg>
__device__ __forceinline__ void full_stage(Kv4State<Cfg> &st, const DecodeParams &p, int rem, bool edge, uint32_t tiles,
                                           uint32_t step, int lane) {
  constexpr int NB = Cfg::NB, NH = Cfg::NH;
  float s[NB][NH][4];
  uint32_t pb[NB][NH][2];
#pragma unroll
  for (int i = 0; i < NB; ++i) scores<Cfg>(st, tiles + i * step, lane, s[i]);
  if (Cfg::kWholeEdges && edge) {
#pragma unroll
    for (int nh = 0; nh < NH; ++nh)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const int r = (lane >> 2) - (rem - st.back[nh][c] - p.wlen);
#pragma unroll
        for (int i = 0; i < NB; ++i) {
          if ((uint32_t)(r + kBlock * i) >= (uint32_t)p.wlen) s[i][nh][c] = -INFINITY;
          if ((uint32_t)(r + kBlock * i + 8) >= (uint32_t)p.wlen) s[i][nh][2 + c] = -INFINITY;
        }
      }
  }
#pragma unroll
  for (int nh = 0; nh < NH; ++nh) softmax<Cfg, NB>(st, nh, s, pb);
  if constexpr (Cfg::kWholeEdges) {
    uint32_t w[NB][2];
#pragma unroll
    for (int i = 0; i < NB; ++i) v_scales<Cfg>(tiles + i * step, lane, w[i]);
    if (edge) {
#pragma unroll
      for (int i = 0; i < NB; ++i) {
        const uint32_t spoiled = clean_scales(w[i], lane, rem - kBlock * i);
        if (__any_sync(kFull, spoiled != 0)) spoil<Cfg>(st, p, rem - kBlock * i, spoiled);
      }
    }
#pragma unroll
    for (int i = 0; i < NB; ++i) values<Cfg>(st, tiles + i * step, lane, w[i], pb[i]);
  } else {
#pragma unroll
    for (int i = 0; i < NB; ++i) {
      uint32_t w[2];
      v_scales<Cfg>(tiles + i * step, lane, w);
      values<Cfg>(st, tiles + i * step, lane, w, pb[i]);
    }
  }
}

// One block of another stage: of fewer blocks, with a bad id (its values are zeros), or see kWholeEdges.
template <class Cfg>
__device__ __forceinline__ void edge_block(Kv4State<Cfg> &st, const DecodeParams &p, int rem, bool zero, uint32_t tile,
                                           int lane) {
  float s[1][Cfg::NH][4];
  uint32_t pb[1][Cfg::NH][2];
  const int gid = lane >> 2;
  scores<Cfg>(st, tile, lane, s[0]);
#pragma unroll
  for (int nh = 0; nh < Cfg::NH; ++nh) {
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      if (zero) s[0][nh][c] = 0.f;
      if ((uint32_t)(gid + 8 * (c >> 1) - (rem - st.back[nh][c & 1] - p.wlen)) >= (uint32_t)p.wlen) s[0][nh][c] = -INFINITY;
    }
    softmax<Cfg, 1>(st, nh, s, pb);
  }
  uint32_t w[2];
  v_scales<Cfg>(tile, lane, w);
  if (zero) w[0] = w[1] = 0;
  const uint32_t spoiled = clean_scales(w, lane, rem);
  if (__any_sync(kFull, spoiled != 0)) spoil<Cfg>(st, p, rem, spoiled);
  values<Cfg>(st, tile, lane, w, pb[0]);
}

template <class Q>
__device__ __forceinline__ void store4(void *out, size_t at, float4 v) {
  *reinterpret_cast<uint2 *>(reinterpret_cast<uint16_t *>(out) + at) =
      make_uint2(pack2(Q{}, v.x, v.y), pack2(Q{}, v.z, v.w));
}

// Ends a segment: a whole unit's rows go to the output; others leave their sums in part
// ([GC][D]), (largest raw score, l) in ml and the scores' factor in scs.
template <class Cfg>
__device__ __forceinline__ void finish(Kv4State<Cfg> &st, const Kv4Params &kp, const Kv4Meta &m, int sub, float *part,
                                       float2 *ml, float *scs, int lane) {
  const DecodeParams &p = kp.d;
  const int gid = lane >> 2, tig = lane & 3;
  const UnitAt u = unit_at(kp, m.hu, Cfg::GC);
  const int h = u.head + sub, r0 = u.row, gc = min(Cfg::GC, p.R - r0);
  constexpr int RUN = Cfg::D / 8;  // a lane's run of d: RUN gid ..
  const bool whole = (m.flags & kOpens) && (m.flags & kCloses);
#pragma unroll
  for (int nh = 0; nh < Cfg::NH; ++nh)
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      float l = st.l[nh][c];
#pragma unroll
      for (int off = 4; off < 32; off <<= 1) l += __shfl_xor_sync(kFull, l, off);
      const int row = 8 * nh + 2 * tig + c;
      // a row that sees nothing gives 0; a sum of NaN gives NaN
      const float f = !whole ? 1.f : l == 0.f ? 0.f : kp.v_unit / l;
      if (row >= gc) continue;
      if (!whole && gid == 0) {
        ml[row] = make_float2(st.m[nh][c], l);
        scs[row] = st.sc[nh][c];
      }
      const size_t at = whole ? row_at(p, m.b, h, r0 + row) + RUN * gid : 0;
#pragma unroll
      for (int i = 0; i < RUN / 4; ++i) {
        const float4 y = make_float4(st.acc[nh][2 * i][c] * f, st.acc[nh][2 * i][2 + c] * f,
                                     st.acc[nh][2 * i + 1][c] * f, st.acc[nh][2 * i + 1][2 + c] * f);
        if (whole)
          store4<typename Cfg::Q>(p.out, at + 4 * i, y);
        else
          reinterpret_cast<float4 *>(part + row * Cfg::D + RUN * gid)[i] = y;
      }
    }
}

// The plan: blocks before each sequence.  Up to 128 sequences it is in a warp's registers: lane l has sequences
// per l .. per l + per - 1, per = ceil(B / 32), their blocks and those before them; in memory otherwise.
struct Kv4Plan {
  const int32_t *pre;
  int before, items[4], per, total;
  bool small;
};
// Unit and block of item x of the list (a whole warp, the same x).
struct Kv4Item {
  int x, b, hu, off, n;  // block off of the unit's n
};
__device__ __forceinline__ Kv4Item locate_item(const DecodeParams &p, const Kv4Plan &plan, int x) {
  const int lane = threadIdx.x & 31;
  // lo: the largest b with HU * blocks before it <= x (the count of items is within 32 bits)
  int lo = 0, first, items;
  if (plan.small) {
    const int l = 31 - __clz(__ballot_sync(kFull, lane * plan.per < p.B && p.HU * plan.before <= x));
    first = __shfl_sync(kFull, plan.before, l);
    items = __shfl_sync(kFull, plan.items[0], l);
    lo = l * plan.per;
#pragma unroll
    for (int i = 1; i < 4 && plan.per > 1; ++i) {
      const int more = __shfl_sync(kFull, plan.items[i], l);
      if (i < plan.per && lo + 1 < p.B && p.HU * (first + items) <= x) {
        ++lo;
        first += items;
        items = more;
      }
    }
  } else {
    for (int span = p.B; span > 1;) {
      const int step = (span + 31) / 32;
      const bool ok = lane * step < span && p.HU * plan.pre[lo + lane * step] <= x;
      const int c = 31 - __clz(__ballot_sync(kFull, ok));
      lo += c * step;
      span = min(step, span - c * step);
    }
    first = plan.pre[lo];
    items = plan.pre[lo + 1] - first;
  }
  Kv4Item r;
  r.x = x;
  r.b = lo;
  r.n = items;
  const int rr = x - p.HU * first;
  r.hu = rr / r.n;
  r.off = rr - r.hu * r.n;
  return r;
}
template <class Cfg>
__global__ void __launch_bounds__(Cfg::THREADS, 1) kv4_decode_kernel(const __grid_constant__ Kv4Params kp) {
  extern __shared__ __align__(128) uint8_t smem[];
  const DecodeParams &p = kp.d;
  const int tid = threadIdx.x, lane = tid & 31, wib = tid >> 5;
  constexpr int WARPS = Cfg::WARPS, STAGES = Cfg::STAGES, GC = Cfg::GC, D = Cfg::D;
  const int hg = kp.hg, rings = WARPS >> kp.hg_log2;
  const int stage_bytes = hg * Cfg::STAGE_BYTES, ring_bytes = STAGES * stage_bytes;
  Kv4Meta *s_meta = reinterpret_cast<Kv4Meta *>(smem + Cfg::TILES_BYTES);  // [ring][stage]
  uint64_t *s_full = reinterpret_cast<uint64_t *>(smem + Cfg::TILES_BYTES + Cfg::META_BYTES);
  uint64_t *s_empty = s_full + WARPS * STAGES;
  int32_t *s_prefix = reinterpret_cast<int32_t *>(smem + Cfg::TILES_BYTES + Cfg::META_BYTES + Cfg::BAR_BYTES);
  float *s_sc = reinterpret_cast<float *>(s_prefix);  // [segment][head][row], once the plan is done
  static_assert(2 * WARPS * GC <= kKv4Prefix, "factors in the plan's place");
  __shared__ int4 s_cut[WARPS + 1];           // {item, b, unit, block} at which a ring's range begins
  __shared__ int2 s_seg[2 * WARPS];           // segments left to join, two a ring, in the list's order: {unit or -1, flags}
  __shared__ float2 s_ml[2 * WARPS * GC];     // [segment][head][row]
  __shared__ int32_t s_ids[WARPS][64];        // table entries ahead, by ring
  __shared__ int32_t s_scan[32];
  __shared__ int cta_flags, s_abort;          // s_abort: bit r: ring r's consumer gave up
  __shared__ __align__(8) uint64_t dead_bar;  // failure-path test hook: nothing ever arrives on it
  if (tid == 0) {
    cta_flags = s_abort = 0;
    mbar_init(&dead_bar, 1);
  }
  if (tid < rings * STAGES) {
    mbar_init(&s_full[tid], 1);
    mbar_init(&s_empty[tid], hg);
  }
  if (tid < 2 * WARPS) s_seg[tid] = make_int2(-1, 0);
  fence_barrier_init();
  __syncthreads();
  grid_dep_launch();  // the merge may take the place of CTAs that have ended; it waits for all of them
  grid_dep_wait();

  // ---- the plan, and the CTA's range [cs, ce) ----
  Kv4Plan plan;
  plan.small = p.B <= 128;
  if (plan.small) {  // every warp for itself
    plan.per = (p.B + 31) / 32;
    int flags = 0, mine = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int b = lane * plan.per + i;
      plan.items[i] = 0;
      if (i < plan.per && b < p.B)
        plan.items[i] = seq_items<false>(p, b, clamp_len<false>(p, b, __ldg(p.context_lens + b), &flags));
      mine += plan.items[i];
    }
    int x = mine;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int y = __shfl_up_sync(kFull, x, off);
      if (lane >= off) x += y;
    }
    plan.before = x - mine;
    plan.total = __shfl_sync(kFull, x, 31);
    if (wib == 0 && flags) atomicOr(&cta_flags, flags);
  } else {
    if (p.inline_plan) inline_plan<false>(p, s_prefix, s_scan, &cta_flags);
    plan.pre = p.inline_plan ? s_prefix : p.prefix;
    plan.total = plan.pre[p.B];
  }
  // Cuts fall on items of equal numbers; one into a unit of few blocks moves to the unit's nearer end, another to
  // whole stages of its unit.  Warp w finds where ring w begins (ring `rings`: where the last ends).
  if (wib <= rings) {
    const int W = p.HU * plan.total, c = blockIdx.x;
    const int ranges = min(p.P, max(1, (int)((((int64_t)W << kp.hg_log2) + kMinItems - 1) / kMinItems)));
    const int each = W / ranges, more = W - each * ranges;
    int cs = W, x = W, n = 0;
    int4 cut = make_int4(W, p.B, 0, 0);
#pragma unroll 1
    for (int t = 0; t < 3 && c < ranges; ++t) {  // the range's beginning, its end, the ring's beginning
      if (t < 2) {
        x = each * (c + t) + min(c + t, more);
      } else {
        const int ce = x;
        n = ce - cs;
        const int q = n / rings;
        x = cs + q * wib + min(wib, n - q * rings);
        if (wib == rings) x = ce;
      }
      if (x < W) {
        const Kv4Item it = locate_item(p, plan, x);
        int back = it.off % Cfg::NB;
        if (t < 2 && it.n <= kKv4Whole<D>) back = 2 * it.off < it.n ? it.off : it.off - it.n;
        if (t == 2 && (wib == 0 || wib == rings || n < 2 * Cfg::NB * rings)) back = 0;
        x -= back;
        if (t == 2) {
          const int j0 = p.window > 0 ? first_block<false>(p, it.b, clamped_len(p, __ldg(p.context_lens + it.b))) : 0;
          cut = make_int4(x, it.b, it.hu, j0 + it.off - back);
        }
      }
      if (t == 0) cs = x;
    }
    if (lane == 0) s_cut[wib] = cut;
  }
  __syncthreads();

  if (wib >= Cfg::WARPS) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(Cfg::REGS_PRODUCER));
    // ---- producers: a lane fills a ring, rings q, q + 4 .. of warp q ----
    const int q = wib - WARPS, per = (rings - q + 3) / 4, r = q + 4 * min(lane, max(per, 1) - 1);
    int nst = 0;
    Kv4Producer<Cfg::NB> pr;
    pr.pi = pr.e = pr.s = pr.b = pr.hu = pr.j = pr.n = pr.j0 = pr.ctx = pr.opens = 0;
    pr.tag_b = pr.tag0 = pr.tag1 = -1;
    pr.ready = 0;
    if (lane < per && s_cut[r].x < s_cut[r + 1].x) {
      const int4 from = s_cut[r];
      pr.pi = pr.s = from.x;
      pr.e = s_cut[r + 1].x;
      pr.b = from.y;
      pr.hu = from.z;
      pr.j = from.w;
      pr.load_seq(p);
    }
    uint8_t *tiles = smem + r * ring_bytes;
    uint64_t *full = s_full + r * STAGES, *empty = s_empty + r * STAGES;
    // the whole warp fetches window k of the sequence of each of these lanes' rings
    auto fetch = [&](uint32_t lanes, int k) {
      for (; lanes; lanes &= lanes - 1) {
        const int of = __ffs(lanes) - 1;
        const int fb = __shfl_sync(kFull, pr.b, of), fk = __shfl_sync(kFull, k, of), fn = __shfl_sync(kFull, pr.n, of);
        const int at = 32 * fk + lane;
        if (at < fn) cp_async4(smem_u32(&s_ids[q + 4 * of][at & 63]), p.block_table + (size_t)fb * p.max_blocks + at);
      }
    };
    uint64_t idle_since = 0;
    for (uint32_t idle = 0;;) {
      const int aborted = *reinterpret_cast<volatile int *>(&s_abort);
      const bool open = pr.pi < pr.e && !((aborted >> r) & 1);
      if (!__any_sync(kFull, open)) break;
      const int stage = nst % STAGES;
      const bool can = open && (nst < STAGES || mbar_test(&empty[stage], (uint32_t)(nst / STAGES - 1) & 1u));
      if (__any_sync(kFull, can)) {
        idle = 0;
        // the stage's entries lie in windows k0 and k1, at most one further
        const int k0 = pr.j >> 5, k1 = (pr.j + max(pr.blocks(), 1) - 1) >> 5;
#pragma unroll 1
        for (int t = 0; t < 2; ++t) {
          const int k = t ? k1 : k0;
          const bool miss = can && !pr.has(k);
          const uint32_t missing = __ballot_sync(kFull, miss);
          if (missing) fetch(missing, k);
          if (miss) pr.expect(k);
        }
        const uint32_t need = 1u << (k0 & 1) | 1u << (k1 & 1);
        if (__any_sync(kFull, can && (pr.ready & need) != need)) {
          cp_async_wait();
          pr.ready = 3;
        }
        __syncwarp();
        if (can) {
          pr.template fill<Cfg>(kp, s_ids[r], tiles + stage * stage_bytes, &s_meta[r * STAGES + stage],
                                &full[stage], &cta_flags);
          ++nst;
        }
        __syncwarp();
        // the window after this one, ahead of its use
        const int ka = (pr.j >> 5) + 1;
        const bool ahead = can && pr.pi < pr.e && pr.has(ka - 1) && !pr.has(ka) && 32 * ka < pr.n;
        const uint32_t more = __ballot_sync(kFull, ahead);
        if (more) fetch(more, ka);
        if (ahead) pr.expect(ka);
      } else {  // every open ring is full: look again shortly, for a limited time
        __nanosleep(kPollNs);
        if (idle == 0) idle_since = global_timer_ns();
        if ((++idle & 255u) == 0 && global_timer_ns() - idle_since > 2 * p.timeout_ns) {
          if (lane == 0) atomicOr(&cta_flags, PKV_FLAG_TIMEOUT);
          break;
        }
      }
    }
    cp_async_wait();
    // copies that no consumer waits for any more land before the CTA's memory goes away
    for (int k = max(0, nst - STAGES); k < nst; ++k)
      mbar_wait_bounded(&full[k % STAGES], (uint32_t)(k / STAGES) & 1u, p.timeout_ns);
    return;  // (their registers are fewer than what follows uses)
  }

  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(Cfg::REGS_CONSUMER));
  // ---- consumers: hg warps work through a ring, each on its head's tiles ----
  const int ring = wib >> kp.hg_log2, sub = wib & (hg - 1);
  const int4 from = s_cut[ring];
  const int total = s_cut[ring + 1].x - from.x;
  if (total > 0) {
    // failure-path test hook: the worker holding the first work item replaces its first
    // wait by one on dead_bar, which runs out and takes the timeout path
    const bool stall = p.stall_ns != 0 && from.x == 0;
    const uint32_t tiles = smem_u32(smem + ring * ring_bytes) + sub * Cfg::TILE, step = hg * Cfg::TILE;
    Kv4State<Cfg> state;
    Kv4Meta m = {from.y, from.z, 0, kFirst};
    uint32_t parity = 0;
    for (int done = 0, stage = 0;;) {
      if (m.flags & kFirst) begin<Cfg>(state, kp, m.b, m.hu, sub, lane);  // (the first: while its blocks are on their way)
      if (done == 0) {
        uint64_t *bar = stall ? &dead_bar : &s_full[ring * STAGES];
        if (!mbar_wait_bounded(bar, 0, p.timeout_ns)) break;
        m = s_meta[ring * STAGES];
      }
      const int nb = m.nb();
      const uint32_t at = tiles + stage * stage_bytes;
      const bool edge = m.rem - state.bk_hi < kBlock * Cfg::NB || m.rem - state.bk_lo > p.wlen;
      if (nb == Cfg::NB && m.bad() == 0 && (Cfg::kWholeEdges || !edge)) {
        full_stage<Cfg>(state, p, m.rem, edge, at, step, lane);
      } else {
#pragma unroll 1
        for (int k = 0; k < nb; ++k)
          edge_block<Cfg>(state, p, m.rem - kBlock * k, (m.bad() >> k) & 1, at + k * step, lane);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&s_empty[ring * STAGES + stage]);  // (the record is in registers, too)
      done += nb;
      if (m.flags & kLast) {
        // The range's last segment leaves its sums in the ring, once all its warps are through; another's, unless
        // the unit is whole, go to memory.
        const bool ends = m.flags & kEnds;
        if (ends) asm volatile("bar.sync %0, %1;" ::"r"(2 + ring), "r"(hg * 32) : "memory");
        const int seg = 2 * ring + (ends ? 1 : 0);
        finish<Cfg>(state, kp, m, sub,
                    ends ? reinterpret_cast<float *>(smem + ring * ring_bytes) + sub * GC * D
                         : kp.first_o + (((size_t)blockIdx.x * rings + ring) * hg + sub) * GC * D,
                    s_ml + (seg * hg + sub) * GC, s_sc + (seg * hg + sub) * GC, lane);
        if (sub == 0 && lane == 0 && (m.flags & (kOpens | kCloses)) != (kOpens | kCloses))
          s_seg[seg] = make_int2(m.b * p.HU + m.hu, m.flags);
        if (ends) {
          m.flags = 0;
          break;
        }
      }
      if (++stage == STAGES) {
        stage = 0;
        parity ^= 1u;
      }
      if (!mbar_wait_bounded(&s_full[ring * STAGES + stage], parity, p.timeout_ns)) {
        m.flags = kFirst;
        break;
      }
      m = s_meta[ring * STAGES + stage];
    }
    if (m.flags != 0) {  // gave up on a wait
      if (lane == 0) {
        atomicOr(&cta_flags, PKV_FLAG_TIMEOUT);
        atomicOr(&s_abort, 1 << ring);
      }
      asm volatile("bar.sync %0, %1;" ::"r"(2 + ring), "r"(hg * 32) : "memory");
    }
  }
  asm volatile("bar.sync 1, %0;" ::"n"(WARPS * 32) : "memory");  // the consumers

  // ---- join the segments of each unit; what a unit lacks is in the neighbouring CTAs ----
  static_assert(2 * WARPS <= 32, "a lane per segment");
  const int2 seg = lane < 2 * WARPS ? s_seg[lane] : make_int2(-1, 0);
  const uint32_t valid = __ballot_sync(kFull, seg.x >= 0);
  const int prev = 31 - __clz(valid & ((1u << lane) - 1));  // the segment before this one, if any
  const int prev_unit = __shfl_sync(kFull, seg.x, prev & 31);
  const uint32_t heads = __ballot_sync(kFull, seg.x >= 0 && (prev < 0 || prev_unit != seg.x));  // a unit's first
  const int rows = hg * GC;  // of a unit
  int4 record = make_int4(-1, 0, -1, 0);  // {unit that an earlier CTA began, ends here; unit that goes on}
  for (uint32_t todo = heads; todo; todo &= todo - 1) {
    const int g = __ffs(todo) - 1, next = todo & (todo - 1) ? __ffs(todo & (todo - 1)) - 1 : 32;
    const uint32_t members = valid & (0xffffffffu << g) & (0xffffffffu >> (32 - next));
    const int unit = __shfl_sync(kFull, seg.x, g);
    const bool opens = __shfl_sync(kFull, seg.y, g) & kOpens;
    const bool closes = __shfl_sync(kFull, seg.y, 31 - __clz(members)) & kCloses;
    if (!opens)
      record.x = unit, record.y = closes;
    else if (!closes)
      record.z = unit;
    const int b = unit / p.HU;
    const UnitAt u = unit_at(kp, unit - b * p.HU, GC);
    // four float4 of the rows that exist a thread at a time: their loads overlap
    const int live = min(GC, p.R - u.row), part = 65536 / live + 1;  // n / live = n * part >> 16 for n < 256
#pragma unroll 1
    for (int v0 = tid; v0 < hg * live * (D / 4); v0 += 4 * WARPS * 32) {
      float4 acc[4];
      float M[4], l[4], sc[4];
      int row[4];  // [head][row]
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        const int n = min(v0 + t * WARPS * 32, hg * live * (D / 4) - 1) / (D / 4), sub = n * part >> 16;
        row[t] = sub * GC + n - sub * live;
        acc[t] = make_float4(0.f, 0.f, 0.f, 0.f);
        M[t] = -INFINITY;
        l[t] = 0.f;
        sc[t] = s_sc[g * rows + row[t]];  // (the same in all segments of a unit)
      }
      const int d = 4 * (v0 % (D / 4));
      static_assert(WARPS * 32 % (D / 4) == 0, "a thread keeps its elements");
#pragma unroll 1
      for (uint32_t left = members; left; left &= left - 1) {
        const int q = __ffs(left) - 1;
        const float *src = (q & 1) ? reinterpret_cast<const float *>(smem + (q >> 1) * ring_bytes)
                                   : kp.first_o + ((size_t)blockIdx.x * rings + (q >> 1)) * rows * D;
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          const float2 ml = s_ml[q * rows + row[t]];
          const float4 a = *reinterpret_cast<const float4 *>(src + row[t] * D + d);
          // (of a row that saw nothing, or NaN alone: its maximum is -inf, its sum 0 or NaN)
          const float m = fmaxf(M[t], ml.x);
          const float keep = M[t] == -INFINITY ? 1.f : exp2_fast((M[t] - m) * sc[t]);
          const float add = ml.x == -INFINITY ? 1.f : exp2_fast((ml.x - m) * sc[t]);
          if (ml.y == 0.f) continue;
          M[t] = m;
          l[t] = fmaf(l[t], keep, ml.y * add);
          acc[t].x = fmaf(acc[t].x, keep, a.x * add);
          acc[t].y = fmaf(acc[t].y, keep, a.y * add);
          acc[t].z = fmaf(acc[t].z, keep, a.z * add);
          acc[t].w = fmaf(acc[t].w, keep, a.w * add);
        }
      }
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        if (v0 + t * WARPS * 32 >= hg * live * (D / 4)) break;
        const float f = l[t] == 0.f ? 0.f : __fdividef(kp.v_unit, l[t]);
        const float4 y = make_float4(acc[t].x * f, acc[t].y * f, acc[t].z * f, acc[t].w * f);
        if (opens && closes) {
          store4<typename Cfg::Q>(p.out, row_at(p, b, u.head + row[t] / GC, u.row + row[t] % GC) + d, y);
        } else {
          const int slot = (blockIdx.x * 2 + (opens ? 1 : 0)) * rows + row[t];
          *reinterpret_cast<float4 *>(p.part_o + (size_t)slot * D + d) = y;
          // {largest raw score, l, factor} (a sum of NaN as a score of +inf: the merge then gives NaN)
          if (d == 0)
            reinterpret_cast<float4 *>(p.part_lse)[slot] =
                make_float4(l[t] != l[t] ? INFINITY : l[t] == 0.f ? -INFINITY : M[t], l[t] != l[t] ? 1.f : l[t], sc[t], 0.f);
        }
      }
    }
  }
  // sequences without a block: 0
  for (int b = blockIdx.x; b < p.B; b += gridDim.x)
    if (__ldg(p.context_lens + b) <= 0)
      for (int v = tid; v < p.q_len * p.Hq * (D / 8); v += WARPS * 32)
        reinterpret_cast<uint4 *>(static_cast<uint16_t *>(p.out) + (size_t)b * p.q_len * p.Hq * D)[v] = make_uint4(0, 0, 0, 0);
  if (tid == 0) {
    kp.records[blockIdx.x] = record;
    p.hdr->cta_status[blockIdx.x] = (uint8_t)(cta_flags | (p.inline_plan ? 0 : p.hdr->plan_flags));
    if (blockIdx.x == 0) p.hdr->status = kStatusPerCta | gridDim.x;
  }
}

// Joins a unit's partial results: CTA (c, part) does the unit that range c begins and does not end, some rows of a
// head of it.  A team of threads has a float4 of these rows each; teams take the partial results in turn, four
// in flight, and are joined through shared memory (a long context's unit has one partial result for each of 76 CTAs).
constexpr int kMergeThreads = 1024;
template <class Q>
__global__ void __launch_bounds__(kMergeThreads) kv4_merge_kernel(const __grid_constant__ Kv4Params kp) {
  const DecodeParams &p = kp.d;
  __shared__ float4 s_acc[kMergeThreads];
  __shared__ float2 s_ml[kMergeThreads];
  const int lane = threadIdx.x & 31;
  grid_dep_launch();
  grid_dep_wait();
  int c = blockIdx.x, unit = -1;
  if (kp.merge_units) {  // fewer units than ranges: a CTA per unit looks for the range that begins it
    for (int at = 0; at < p.P && unit < 0; at += 32) {
      const uint32_t is = __ballot_sync(kFull, at + lane < p.P && kp.records[at + lane].z == (int)blockIdx.x);
      if (is) {
        c = at + __ffs(is) - 1;
        unit = blockIdx.x;
      }
    }
  } else {
    unit = kp.records[c].z;
  }
  if (unit < 0) return;
  // the ranges that continue it: c + 1 .. last
  int last = c;
  for (int at = c + 1; at < p.P; at += 32) {
    const int4 r = at + lane < p.P ? kp.records[at + lane] : make_int4(-1, 0, -1, 0);
    const uint32_t goes = __ballot_sync(kFull, r.x == unit), ends = __ballot_sync(kFull, r.x != unit || r.y != 0);
    const int stop = __ffs(ends);  // 1-based lane of the last (or of one past it)
    if (stop) {
      last = at + stop - 1 - ((goes >> (stop - 1)) & 1 ? 0 : 1);
      break;
    }
    last = min(at + 31, p.P - 1);
  }
  const int D = p.D, size = kp.merge_rows * D / 4, team = threadIdx.x / size, teams = blockDim.x / size;
  const int parts = p.GC / kp.merge_rows, sub = blockIdx.y / parts;
  const int v = threadIdx.x - team * size, row = blockIdx.y % parts * kp.merge_rows + 4 * v / D, d = 4 * v % D;
  const int b = unit / p.HU;
  const UnitAt u = unit_at(kp, unit - b * p.HU, p.GC);
  const int r = u.row + row;
  constexpr int kBatch = 4;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  float M = -INFINITY, den = 0.f;
  const float4 *ml = reinterpret_cast<const float4 *>(p.part_lse);
  const float sc = ml[((c * 2 + 1) * kp.hg + sub) * p.GC + row].z;  // (the same in all of them)
#pragma unroll 1
  for (int s = c + team; s <= last && r < p.R; s += kBatch * teams) {
    float4 o[kBatch];
    float m[kBatch], l[kBatch];
#pragma unroll
    for (int t = 0; t < kBatch; ++t) {
      const int w = min(s + t * teams, last);
      const int slot = ((w * 2 + (w == c ? 1 : 0)) * kp.hg + sub) * p.GC + row;
      const float4 x = ml[slot];
      m[t] = s + t * teams <= last ? x.x : -INFINITY;
      l[t] = x.y;
      o[t] = *reinterpret_cast<const float4 *>(p.part_o + (size_t)slot * D + d);
    }
    float cm = M;
#pragma unroll
    for (int t = 0; t < kBatch; ++t) cm = fmaxf(cm, m[t]);
    if (cm == -INFINITY) continue;  // nothing seen yet
    const float keep = M == -INFINITY ? 0.f : exp2_fast((M - cm) * sc);
    acc.x *= keep; acc.y *= keep; acc.z *= keep; acc.w *= keep;
    den *= keep;
#pragma unroll
    for (int t = 0; t < kBatch; ++t) {
      const bool on = m[t] != -INFINITY;
      const float wt = on ? l[t] * exp2_fast((m[t] - cm) * sc) : 0.f;
      acc.x = fmaf(wt, on ? o[t].x : 0.f, acc.x);
      acc.y = fmaf(wt, on ? o[t].y : 0.f, acc.y);
      acc.z = fmaf(wt, on ? o[t].z : 0.f, acc.z);
      acc.w = fmaf(wt, on ? o[t].w : 0.f, acc.w);
      den += wt;
    }
    M = cm;
  }
  s_acc[threadIdx.x] = acc;
  s_ml[threadIdx.x] = make_float2(M, den);
  __syncthreads();
  if (team > 0 || r >= p.R) return;
  if (teams > 1) {
    float all = M;
#pragma unroll 1
    for (int t = 1; t < teams; ++t) all = fmaxf(all, s_ml[t * size + v].x);
    den = 0.f;
    acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
    for (int t = 0; t < teams; ++t) {
      const float2 ml = s_ml[t * size + v];
      if (ml.x == -INFINITY) continue;
      const float wt = exp2_fast((ml.x - all) * sc);
      const float4 a = s_acc[t * size + v];
      acc.x = fmaf(wt, a.x, acc.x);
      acc.y = fmaf(wt, a.y, acc.y);
      acc.z = fmaf(wt, a.z, acc.z);
      acc.w = fmaf(wt, a.w, acc.w);
      den = fmaf(wt, ml.y, den);
    }
  }
  const float inv = den == 0.f ? 0.f : 1.f / den;
  store4<Q>(p.out, row_at(p, b, u.head + sub, r) + d, make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv));
}

cudaError_t launch_kv4_merge(Kv4Params p, cudaStream_t stream, bool pdl) {
  cudaLaunchConfig_t cfg = {};
  // many units: a CTA per range and head, one team; few: two rows a CTA and a team per four partial results
  const int units = p.d.B * p.d.HU, each = (p.d.n_ctas + units - 1) / units + 1;
  p.merge_units = units < p.d.n_ctas;
  p.merge_rows = each > 8 ? 2 : p.d.GC;
  const int size = p.merge_rows * p.d.D / 4;
  int teams = 1;
  while (2 * teams * size <= kMergeThreads && teams * 4 < each) teams *= 2;
  cfg.gridDim = dim3(p.merge_units ? units : p.d.n_ctas, p.hg * (p.d.GC / p.merge_rows));
  cfg.blockDim = dim3(teams * size);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pdl ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, p.d.out_dtype == PKV_F16 ? kv4_merge_kernel<F16> : kv4_merge_kernel<BF16>, p);
}

template <class Cfg>
static Kv4Kernel kv4_entry() {
  return Kv4Kernel{reinterpret_cast<const void *>(&kv4_decode_kernel<Cfg>), Cfg::Q::kCode, Cfg::D, Cfg::GC, Cfg::WARPS,
                   Cfg::THREADS, Cfg::SMEM};
}

// Warps: as many as the registers of a unit's sums and queries leave without spills (16-row units, 16 x 1000-32768,
// 4 new, 32 / 8 heads: of D = 64 12 warps 62 us, 8 70; of D = 128 12 warps 101 to 132, 8 93).
void register_decode_kv4(Kv4Kernel (&out)[kKv4Kernels]) {
  int n = 0;
  out[n++] = kv4_entry<Kv4Cfg<BF16, 128, 1, 12, 2, 4>>();
  out[n++] = kv4_entry<Kv4Cfg<F16, 128, 1, 12, 2, 4>>();
  out[n++] = kv4_entry<Kv4Cfg<BF16, 64, 1, 12, 4, 4>>();
  out[n++] = kv4_entry<Kv4Cfg<F16, 64, 1, 12, 4, 4>>();
  out[n++] = kv4_entry<Kv4Cfg<BF16, 128, 2, 8, 3, 4>>();
  out[n++] = kv4_entry<Kv4Cfg<F16, 128, 2, 8, 3, 4>>();
  out[n++] = kv4_entry<Kv4Cfg<BF16, 64, 2, 12, 4, 4>>();
  out[n++] = kv4_entry<Kv4Cfg<F16, 64, 2, 12, 4, 4>>();
}

}  // namespace pkv
