// tree_tiles_fp8.cu — attention of a tree of drafted tokens over an FP8-E4M3 cache
// on the tensor cores, query rows on the M side: the schedule, masks and tile
// pipeline of tree_tiles.cu.
//
// S = Q . K^T takes K as it is stored: kind::f8f6f4 on E4M3, with Q as a sum of E4M3
// parts.  A row of Q is scaled by a power of two to at most 448 and split by
// rounding, q1 = e4m3(x), q2 = e4m3(x - q1), ..: each part holds 4 significant bits, so
// two parts are a bf16 element and three an f16 one exactly, down to E4M3's subnormal
// step of 2^-9: elements below 2^-9 of the row's largest (2^-6 for f16; the largest lies in
// (224, 448]) are held to half that step, 2^-17.8 of the largest.  The MMA
// runs at twice the 16-bit rate, so two parts cost what one f16 product would,
// and K is never widened.
// P . V runs on f16: four warps widen each V tile to f16 in shared memory (exact),
// in the operand layout of a 16-bit cache, once for all 128 rows (the decode kernel's
// units widen an element once per 16).
//
// Block scales.  With k_b, v_b the scales of block b, a position's score is
// s k_b c (c = scale * log2 e) and its value v_b * dec.  Both go into the exponent:
// with lv_b = log2 v_b,
//   p' = 2^(s (c k_b) + lv_b - m),  m = max over positions of s (c k_b) + lv_b,
//   out = sum p' dec / sum p' / v_b,
// so that the weights the tensor core takes are <= 1 whatever the scales
// (weights times v_b would leave f16's normal range for small V), and no
// element is multiplied by a scale at all.  A block with a scale that is not a
// positive finite number takes the literal products instead; one with a scale that is not
// finite (an overflowed branch opened the block) enters as a K scale of NaN and a V
// scale of 0, so that the rows that see it are NaN and hidden weights stay 0 (0 times
// infinity would be NaN in every row).
//
// What bounds it: a tile takes ~1.2 us (head dim 128) against 0.73 for its bytes from
// HBM and 0.7 for its 176 KiB of shared-memory traffic: the softmax of a lane quarter,
// whose two warps share one scheduler, is ~2200 clocks long (1100 of them the weights, 350 the
// exchange of maxima, 290 the block scales).  16 x 32768, 32 / 8 heads, 8 nodes 274 - 278 us (3.9
// TB/s); 16 x 8192, 64 nodes 157 - 162 us (850 - 880 TFLOP/s).  At head dim 64 a tile holds half the bytes
// and costs nearly the same softmax, scales and barriers: 64 x 4096, 32 / 8 heads, 16 nodes 150 us
// (1.4 us a tile, 1.8 TB/s; its bytes alone 40).  Tried and slower: widening K as well (2.1
// us a tile), one K stage less (64 nodes 187), the rows of a small tree copied into all
// four lane quarters, each taking every fourth tile (2.0 us a tile: the others' weights have to
// be cleared).
#include "prefill_common.cuh"
#include "tree_tiles.cuh"

namespace pkv {

template <int D_, class QT>
struct TreeFp8Cfg : PrefillCfg<F16, D_> {
  using Base = PrefillCfg<F16, D_>;
  static constexpr bool OUT_BF = QT::kCode == PKV_BF16;
  static constexpr int QPARTS = OUT_BF ? 2 : 3;        // E4M3 parts of Q
  static constexpr int ROWB = D_;                      // bytes of a K / V / Q-part row
  static constexpr int Q_PART = Base::M * ROWB;
  static constexpr int RAW_BYTES = Base::N * ROWB;     // one E4M3 tile
  static constexpr int KSTAGES = OUT_BF ? 4 : 3, VRAW = 3, VSTAGES = 2;
  static constexpr int K_LINES = kBlock, V_LINES = kBlock * D_ / 128;  // rows of a block's box in the K and V tensor maps
  static constexpr size_t SMEM = 1024 + (size_t)QPARTS * Q_PART + (size_t)(KSTAGES + VRAW) * RAW_BYTES +
                                 (size_t)VSTAGES * Base::KV_BYTES;
  // warps 0-7 softmax, 8 K copies, 9 S issue, 10 P . V issue, 11 V copies, 12-15 widening
  static constexpr int ISSUER = Base::SOFTMAX / 32 + 1, PV_ISSUER = Base::SOFTMAX / 32 + 2,
                       V_PRODUCER = Base::SOFTMAX / 32 + 3, WIDEN = Base::SOFTMAX / 32 + 4;
  static constexpr int WIDENERS = 128;
  static constexpr int SCALES = 8;  // tiles whose block scales are kept: more than can be between K's copy and the softmax
  static constexpr int THREADS = Base::SOFTMAX + 256;
  // registers per thread: 128 at launch; the softmax warpgroups take what the others leave
  static constexpr int REGS_SOFTMAX = 168, REGS_OTHER = 88;
  static_assert(Base::SOFTMAX * REGS_SOFTMAX + 256 * REGS_OTHER <= THREADS * 128 && THREADS * 128 == 65536, "register file");
  static_assert(SMEM + 6144 <= 232448, "shared memory");
};

// Address of 16-byte chunk c of position r in a raw tile (128-byte lines, 128-byte
// swizzle; 64-byte rows lie two to a line).
template <int D>
__device__ __forceinline__ uint32_t raw_off(int r, int c) {
  if constexpr (D == 128)
    return (uint32_t)(r * 128 + ((c ^ (r & 7)) << 4));
  else
    return (uint32_t)((r >> 1) * 128 + (((((r & 1) << 2) | c) ^ ((r >> 1) & 7)) << 4));
}

// Address of 16-byte chunk c of row r in a Q part or K tile: K-major, 128-byte
// rows with the 128-byte swizzle, or 64-byte rows with the 64-byte swizzle.
template <int D>
__device__ __forceinline__ uint32_t kmajor_off(int r, int c) {
  if constexpr (D == 128)
    return (uint32_t)(r * 128 + ((c ^ (r & 7)) << 4));
  else
    return (uint32_t)(r * 64 + ((c ^ ((r >> 1) & 3)) << 4));
}

// S = Q . K^T of one tile into tensor-memory columns dS: every part of Q (at q0)
// against K (at k0), 32 elements per MMA.  Issued by one thread.
template <class Cfg>
__device__ __forceinline__ void mma_s_tile_e4m3(uint32_t dS, uint32_t q0, uint32_t k0) {
  constexpr uint32_t id = tc::idesc_e4m3(Cfg::M, Cfg::N);
  constexpr uint32_t layout = Cfg::D == 128 ? 2u : 4u;  // 128- or 64-byte swizzle, 8-row atoms
#pragma unroll
  for (int part = 0; part < Cfg::QPARTS; ++part)
#pragma unroll
    for (int k = 0; k < Cfg::D / 32; ++k)
      tc::mma_e4m3(dS, tc::desc_sw(q0 + (uint32_t)(part * Cfg::Q_PART + k * 32), 16, 8 * Cfg::ROWB, layout),
                   tc::desc_sw(k0 + (uint32_t)(k * 32), 16, 8 * Cfg::ROWB, layout), id, part > 0 || k > 0 ? 1u : 0u);
}

// The widening warps' part of one tile: chunk i = t, t + 64, ...; rows at or past
// `zero_from` (stale positions past the context) become zeros.
// (tree_finite.cuh) The same chunks of the rows that not every row sees, positions kv0 + r < ctx:
// what is NaN becomes 0, noted in `spoiled`.
template <class Cfg>
__device__ __forceinline__ void clean_raw_tile(uint8_t *raw, int kv0, int ctx, TreePartial t, int thread, unsigned long long *spoiled) {
  constexpr int CPR = Cfg::D / 16;
#pragma unroll 1
  for (int i = thread; i < Cfg::N * CPR; i += Cfg::WIDENERS) {
    const int r = i / CPR, pos = kv0 + r;
    if (pos < ctx && t.holds(pos) && clear_nonfinite<E4M3>(smem_u32(raw) + raw_off<Cfg::D>(r, i % CPR))) {
      TreeSpoiled s{0, 0};
      s.note(t, pos);
      if (s.nodes) atomicOr(&spoiled[0], (unsigned long long)s.nodes);
      if (s.edge) atomicOr(&spoiled[1], (unsigned long long)s.edge);
    }
  }
}
template <class Cfg>
__device__ __forceinline__ void widen_tile(const uint8_t *raw, uint8_t *op, int zero_from, int t) {
  constexpr int CPR = Cfg::D / 16;                       // chunks per row
  constexpr int PER = Cfg::N * CPR / Cfg::WIDENERS, BATCH = PER < 8 ? PER : 8;  // chunks of a thread, in flight
  static_assert(PER * Cfg::WIDENERS == Cfg::N * CPR && PER % BATCH == 0, "whole batches cover the tile");
  const uint32_t rb = smem_u32(raw), ob = smem_u32(op);
#pragma unroll 1
  for (int k0 = 0; k0 < PER; k0 += BATCH) {
    uint4 x[BATCH];
#pragma unroll
    for (int k = 0; k < BATCH; ++k) {
      const int i = t + (k0 + k) * Cfg::WIDENERS;
      x[k] = lds128(rb + raw_off<Cfg::D>(i / CPR, i % CPR));
    }
#pragma unroll
    for (int k = 0; k < BATCH; ++k) {
      const int i = t + (k0 + k) * Cfg::WIDENERS, r = i / CPR, c = i % CPR;
      uint4 a = make_uint4(0, 0, 0, 0), b = make_uint4(0, 0, 0, 0);
      if (r < zero_from) {
        a = make_uint4(e4m3x2_to_f16x2((uint16_t)(x[k].x & 0xffff)), e4m3x2_to_f16x2((uint16_t)(x[k].x >> 16)),
                       e4m3x2_to_f16x2((uint16_t)(x[k].y & 0xffff)), e4m3x2_to_f16x2((uint16_t)(x[k].y >> 16)));
        b = make_uint4(e4m3x2_to_f16x2((uint16_t)(x[k].z & 0xffff)), e4m3x2_to_f16x2((uint16_t)(x[k].z >> 16)),
                       e4m3x2_to_f16x2((uint16_t)(x[k].w & 0xffff)), e4m3x2_to_f16x2((uint16_t)(x[k].w >> 16)));
      }
      // elements 16c .. 16c + 15: panel c / 4, 16-byte chunks 2 (c % 4) and the next.
      // The two panels share banks, so panel 1 stores its odd chunk first.
      const uint32_t row = ob + (uint32_t)((c >> 2) * Cfg::PANEL_KV + r * 128);
      const int ch = (c & 3) * 2;
      const bool odd_first = c >= 4;
      sts128(row + (uint32_t)(((ch + (odd_first ? 1 : 0)) ^ (r & 7)) << 4), odd_first ? b : a);
      sts128(row + (uint32_t)(((ch + (odd_first ? 0 : 1)) ^ (r & 7)) << 4), odd_first ? a : b);
    }
  }
}

// One row of Q (D 16-bit elements at src; null: zeros), chunks ch0 .. ch1 - 1 of 16
// elements, as E4M3 parts into row `row` of the Q tile at q0.  Returns 2^-k, the
// row's scaling undone; NaN for a row that is not finite.
template <class Cfg>
__device__ __noinline__ float stage_q_parts(const uint4 *src, uint32_t q0, int row, int ch0, int ch1) {
  // the row's largest magnitude, as bits (a 16-bit float's order is its bits')
  uint32_t top = 0;
#pragma unroll 4
  for (int k = 0; k < Cfg::D / 8; ++k) {
    const uint4 v = src ? __ldg(src + k) : make_uint4(0, 0, 0, 0);
    top = __vmaxu2(__vmaxu2(__vmaxu2(v.x & 0x7fff7fffu, v.y & 0x7fff7fffu), __vmaxu2(v.z & 0x7fff7fffu, v.w & 0x7fff7fffu)),
                   top);
  }
  const uint32_t big = max(top & 0xffffu, top >> 16);
  const bool finite = big < (Cfg::OUT_BF ? 0x7f80u : 0x7c00u);
  const float m = Cfg::OUT_BF ? __uint_as_float(big << 16) : __half2float(__ushort_as_half((unsigned short)big));
  int e = 0;
  const float f = frexpf(finite ? m : 0.f, &e);  // m = f 2^e; 448 = 0.875 * 2^9
  const int sh = m > 0.f && finite ? min((f <= 0.875f ? 9 : 8) - e, 120) : 0;
  const float up = ldexpf(1.f, sh);
#pragma unroll 1
  for (int ch = ch0; ch < ch1; ++ch) {
    const uint4 v0 = src ? __ldg(src + 2 * ch) : make_uint4(0, 0, 0, 0);
    const uint4 v1 = src ? __ldg(src + 2 * ch + 1) : make_uint4(0, 0, 0, 0);
    const uint32_t w[8] = {v0.x, v0.y, v0.z, v0.w, v1.x, v1.y, v1.z, v1.w};
    uint32_t part[Cfg::QPARTS][4];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float2 x = Cfg::OUT_BF ? unpack2(BF16{}, w[i]) : unpack2(F16{}, w[i]);
      x.x *= up;
      x.y *= up;
#pragma unroll
      for (int q = 0; q < Cfg::QPARTS; ++q) {
        const uint32_t r = __nv_cvt_float2_to_fp8x2(x, __NV_SATFINITE, __NV_E4M3);
        const float2 y = unpack2_e4m3((uint16_t)r);
        x.x -= y.x;
        x.y -= y.y;
        if (i & 1)
          part[q][i >> 1] |= r << 16;
        else
          part[q][i >> 1] = r;
      }
    }
#pragma unroll
    for (int q = 0; q < Cfg::QPARTS; ++q)
      sts128(q0 + q * Cfg::Q_PART + kmajor_off<Cfg::D>(row, ch), make_uint4(part[q][0], part[q][1], part[q][2], part[q][3]));
  }
  fence_proxy_async();
  return finite ? ldexpf(1.f, -sh) : __int_as_float(0x7fc00000);
}

// A wait of the warps beside the softmax: its slow part out of line (tile_wait) at head
// dim 64, where the widening loop's instruction fetch counts (64 x 4096, 16 nodes 150 us, inline
// 166), inline at 128 (16 x 8192, 64 nodes 156 us, out of line 162).
template <class Cfg>
__device__ __forceinline__ bool other_wait(uint64_t *bar, uint32_t parity, uint64_t limit_ns) {
  if constexpr (Cfg::D == 64)
    return tile_wait<1>(bar, parity, limit_ns);
  else
    return warp_wait(bar, parity, limit_ns);
}

template <class Cfg>
__global__ void __launch_bounds__(Cfg::THREADS, 1)
    tree_tile_fp8_kernel(const __grid_constant__ TreeTileParams tp, const __grid_constant__ CUtensorMap tmK,
                         const __grid_constant__ CUtensorMap tmV) {
  const MqParams &p = tp.m;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint8_t *sQ = smem;
  uint8_t *sK = sQ + (size_t)Cfg::QPARTS * Cfg::Q_PART;
  uint8_t *sR = sK + (size_t)Cfg::KSTAGES * Cfg::RAW_BYTES;  // V as it lands
  uint8_t *sV = sR + (size_t)Cfg::VRAW * Cfg::RAW_BYTES;     // V as f16
  __shared__ __align__(8) uint64_t k_full[Cfg::KSTAGES], k_empty[Cfg::KSTAGES];
  __shared__ __align__(8) uint64_t r_full[Cfg::VRAW], r_empty[Cfg::VRAW];  // V landed / widened
  __shared__ __align__(8) uint64_t v_full[Cfg::VSTAGES], v_empty[Cfg::VSTAGES];
  __shared__ __align__(8) uint64_t s_full[Cfg::SBUF], p_full[Cfg::SBUF], pv_done[Cfg::SBUF];
  __shared__ __align__(8) uint64_t q_full, o_free, xl, fin;
  __shared__ __align__(8) uint64_t xch[Cfg::SOFTMAX / 64][2];
  __shared__ float red[2][2][Cfg::M];
  __shared__ float red_l[2][Cfg::M];
  __shared__ TreeItem items[4];
  __shared__ __align__(8) uint64_t item_full[4];
  // [item parity][nodes, window's edge], and what the widening warps noted of a V slot's tile
  __shared__ __align__(16) unsigned long long spoiled[2][2], slot_spoiled[Cfg::VSTAGES][2];
  // per tile, by block: {k_b, log2 v_b, 1 / v_b, 0}, or {1, 0, 1, 1} and {k_b, v_b}
  // in `literal` for scales that are not positive finite numbers
  __shared__ __align__(16) float4 scales[Cfg::SCALES][Cfg::BLOCKS];
  __shared__ float2 literal[Cfg::SCALES][Cfg::BLOCKS];
  __shared__ TreeFind find;
  __shared__ uint32_t tmem_base;
  __shared__ int abort_flag, cta_flags, k_issued, r_issued;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rt = (int)blockIdx.x % tp.RT, group = (int)blockIdx.x / tp.RT;
  if (tid == 0) {
#pragma unroll
    for (int s = 0; s < Cfg::KSTAGES; ++s) {
      mbar_init(&k_full[s], 1);
      mbar_init(&k_empty[s], 1);
    }
#pragma unroll
    for (int s = 0; s < Cfg::VRAW; ++s) {
      mbar_init(&r_full[s], 1);
      mbar_init(&r_empty[s], Cfg::WIDENERS / 32);
    }
#pragma unroll
    for (int s = 0; s < Cfg::VSTAGES; ++s) {
      mbar_init(&v_full[s], Cfg::WIDENERS / 32);
      mbar_init(&v_empty[s], 1);
    }
#pragma unroll
    for (int s = 0; s < Cfg::SBUF; ++s) {
      mbar_init(&s_full[s], 2);  // the MMAs' completion, and the issuer's own arrival (orders the block scales)
      mbar_init(&p_full[s], Cfg::SOFTMAX / 32);
      mbar_init(&pv_done[s], 1);
    }
#pragma unroll
    for (int pr = 0; pr < Cfg::SOFTMAX / 64; ++pr) {
      mbar_init(&xch[pr][0], 2);
      mbar_init(&xch[pr][1], 2);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) mbar_init(&item_full[i], 1);
    mbar_init(&q_full, Cfg::SOFTMAX / 32);
    mbar_init(&o_free, Cfg::SOFTMAX / 32);
    mbar_init(&xl, Cfg::SOFTMAX / 32);
    mbar_init(&fin, 2);  // one commit from each issuing warp
    for (int s = 0; s < Cfg::VSTAGES; ++s) slot_spoiled[s][0] = slot_spoiled[s][1] = 0;
    fence_barrier_init();
    abort_flag = 0;
    cta_flags = 0;
    k_issued = r_issued = 0;
  }
  if (warp == Cfg::ISSUER) tc::alloc(&tmem_base, Cfg::TMEM_COLS);
  if (warp == Cfg::PRODUCER && lane == 0) {
    tma_prefetch_desc(&tmK);
    tma_prefetch_desc(&tmV);
  }
  grid_dep_wait();  // launched early behind the previous kernel: its writes are visible from here on
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  const uint32_t tbase = tmem_base;

  grid_dep_launch();  // the merge kernel's blocks may take the SMs as CTAs leave (it waits for this grid's end)
  const TreeRange rg = tree_plan<Cfg::SOFTMAX>(p, group, tp.groups, &find, &cta_flags);

  // this CTA's next item with rows in its row tile
  auto next_item = [&](MqWalk &wk, MqSeg &sg) -> bool {
    while (wk.next(p, sg))
      if (rt * Cfg::M < sg.n * p.G) return true;
    return false;
  };
  auto fail = [&]() {
    if (lane == 0) {
      atomicOr(&cta_flags, PKV_FLAG_TIMEOUT);
      abort_flag = 1;
    }
  };
  auto aborted = [&]() -> bool { return __any_sync(kFull, *(volatile int *)&abort_flag); };

  if (warp >= Cfg::SOFTMAX / 32) {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(Cfg::REGS_OTHER));
  if (warp == Cfg::PRODUCER || warp == Cfg::V_PRODUCER) {
    // ---------------- TMA producers: K tiles (warp 8), V tiles (warp 11) ----------------
    // lane l < 8 fetches block l of a tile; ids loaded three tiles ahead
    MqWalk wk;
    wk.start(rg.b0, rg.base0, rg.t0, rg.t1);
    MqSeg cs{};
    int cj = 0;
    bool have = false;
    auto step = [&]() -> bool {
      if (have && ++cj < cs.j1) return true;
      have = next_item(wk, cs);
      if (have) cj = cs.j0;
      return have;
    };
    int bad = 0;
    struct Pend {
      int id, h;
      float ks, vs;
      bool none;
    };
    auto fetch = [&]() -> Pend {
      Pend f;
      const int lb = (cs.j_first + cj) * Cfg::BLOCKS + (lane & (Cfg::BLOCKS - 1));
      const int nblk = (cs.ctx + kBlock - 1) / kBlock;
      f.h = cs.h;
      f.none = lb >= nblk || (lb + 1) * kBlock <= cs.first;
      f.id = f.none ? 0 : __ldg(p.block_table + (size_t)cs.b * p.max_blocks + lb);
      f.ks = f.vs = 1.f;  // (a block that does not exist: its columns are masked)
      return f;
    };
    auto load_scales = [&](Pend &f) {  // once the id is here, a tile ahead of their use
      if (warp == Cfg::PRODUCER && !f.none && f.id >= 0 && (int64_t)f.id < p.num_blocks) {
        f.ks = __ldg(p.k_scale + (size_t)f.id * p.Hkv + f.h);
        f.vs = __ldg(p.v_scale + (size_t)f.id * p.Hkv + f.h);
      }
    };
    auto row_of = [&](const Pend &f) -> int64_t {  // the box past the tensor (zeros) for none or a bad id
      if (f.none) return p.num_blocks * p.Hkv;
      const bool good = f.id >= 0 && (int64_t)f.id < p.num_blocks;
      bad |= good ? 0 : 1;
      return good ? (int64_t)f.id * p.Hkv + f.h : p.num_blocks * p.Hkv;
    };
    bool ok = true;
    const Pend nil{0, 0, 1.f, 1.f, true};
    bool h0 = step();
    Pend f0 = h0 ? fetch() : nil;
    bool h1 = h0 && step();
    Pend f1 = h1 ? fetch() : nil;
    bool h2 = h1 && step();
    Pend f2 = h2 ? fetch() : nil;
    const bool vw = warp == Cfg::V_PRODUCER;
    uint8_t *ring = vw ? sR : sK;
    uint64_t *full = vw ? r_full : k_full, *empty = vw ? r_empty : k_empty;
    const int stages = vw ? Cfg::VRAW : Cfg::KSTAGES, lines = vw ? Cfg::V_LINES : Cfg::K_LINES;
    const CUtensorMap *tm = vw ? &tmV : &tmK;
    int *issued = vw ? &r_issued : &k_issued;
    load_scales(f0);
    for (int g = 0; h0; ++g) {
      const bool h3 = h2 && step();
      const Pend f3 = h3 ? fetch() : nil;
      load_scales(f1);
      const int y = (int)(row_of(f0) * lines);
      const int s = g % stages;
      if (g >= stages) ok = other_wait<Cfg>(&empty[s], (uint32_t)((g / stages) - 1) & 1u, p.timeout_ns);
      if (!ok || aborted()) {
        ok = false;
        break;
      }
      if (!vw && lane < Cfg::BLOCKS) {
        const bool plain = f0.ks > 0.f && f0.vs > 0.f && f0.ks <= 3.402823466e38f && f0.vs <= 3.402823466e38f;
        scales[g % Cfg::SCALES][lane] =
            plain ? make_float4(f0.ks, __log2f(f0.vs), __fdividef(1.f, f0.vs), 0.f) : make_float4(1.f, 0.f, 1.f, 1.f);
        const bool finite = fabsf(f0.ks) < INFINITY && fabsf(f0.vs) < INFINITY;
        literal[g % Cfg::SCALES][lane] = finite ? make_float2(f0.ks, f0.vs) : make_float2(__int_as_float(0x7fc00000), 0.f);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive_expect_tx(&full[s], Cfg::RAW_BYTES);
      __syncwarp();
      if (lane < Cfg::BLOCKS)
        tma_load_2d(ring + (size_t)s * Cfg::RAW_BYTES + lane * (kBlock * Cfg::ROWB), tm, 0, y, &full[s]);
      if (lane == 0) *issued = g + 1;
      h0 = h1;
      f0 = f1;
      h1 = h2;
      f1 = f2;
      h2 = h3;
      f2 = f3;
    }
    if (__any_sync(kFull, bad) && lane == 0) atomicOr(&cta_flags, PKV_FLAG_BAD_BLOCK);
    if (!ok) fail();
  } else if (warp >= Cfg::WIDEN) {
    // ---------------- widening: V tiles to f16 operands ----------------
    const int t = tid - Cfg::WIDEN * 32;
    bool ok = true;
    MqWalk wk;
    wk.start(rg.b0, rg.base0, rg.t0, rg.t1);
    MqSeg sg{};
    int g = 0;
    while (ok && next_item(wk, sg)) {
      const PartialTiles part = partial_tiles(p, sg);
      for (int j = sg.j0; ok && j < sg.j1; ++j, ++g) {
        const int rs = g % Cfg::VRAW, os = g % Cfg::VSTAGES;
        ok = other_wait<Cfg>(&r_full[rs], (uint32_t)(g / Cfg::VRAW) & 1u, p.timeout_ns);
        // the operand slot is free once P . V of tile g - VSTAGES has read it
        if (ok && g >= Cfg::VSTAGES) ok = other_wait<Cfg>(&v_empty[os], (uint32_t)((g / Cfg::VSTAGES) - 1) & 1u, p.timeout_ns);
        if (!ok || aborted()) {
          ok = false;
          break;
        }
        if (part.has(j))
          clean_raw_tile<Cfg>(sR + (size_t)rs * Cfg::RAW_BYTES, (sg.j_first + j) * Cfg::N, sg.ctx, tree_partial(p, sg), t,
                              slot_spoiled[os]);
        widen_tile<Cfg>(sR + (size_t)rs * Cfg::RAW_BYTES, sV + (size_t)os * Cfg::KV_BYTES,
                        sg.ctx - (sg.j_first + j) * Cfg::N, t);
        fence_proxy_async();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&r_empty[rs]);
          mbar_arrive(&v_full[os]);
        }
      }
    }
    if (!ok) fail();
  } else if (warp == Cfg::ISSUER) {
    // ---------------- S issue: in tile order as K lands ----------------
    bool ok = true;
    MqWalk wk;
    wk.start(rg.b0, rg.base0, rg.t0, rg.t1);
    MqSeg sg{}, nx{};
    int g = 0;
    auto publish = [&](int k, const MqSeg &s, bool have) {
      if (lane == 0) {
        items[k & 3] = TreeItem{s, have ? 1 : 0};
        mbar_arrive(&item_full[k & 3]);
      }
      __syncwarp();
    };
    bool have = next_item(wk, nx);
    publish(0, nx, have);
    for (int si = 0; ok && have; ++si) {
      sg = nx;
      have = next_item(wk, nx);
      publish(si + 1, nx, have);
      ok = other_wait<Cfg>(&q_full, (uint32_t)si & 1u, p.timeout_ns);
      for (int j = sg.j0; ok && j < sg.j1; ++j, ++g) {
        const int ks = g % Cfg::KSTAGES, sb = g % Cfg::SBUF;
        ok = other_wait<Cfg>(&k_full[ks], (uint32_t)(g / Cfg::KSTAGES) & 1u, p.timeout_ns);
        // S overwrites the buffer whose P . V of tile g - SBUF read P from it
        if (ok && g >= Cfg::SBUF)
          ok = other_wait<Cfg>(&pv_done[sb], (uint32_t)((g / Cfg::SBUF) - 1) & 1u, p.timeout_ns);
        if (!ok) break;
        tc::fence_after();
        if (lane == 0) {
          mma_s_tile_e4m3<Cfg>(tbase + (uint32_t)(sb * Cfg::N), smem_u32(sQ), smem_u32(sK + (size_t)ks * Cfg::RAW_BYTES));
          tc::commit(&s_full[sb]);
          mbar_arrive(&s_full[sb]);
          tc::commit(&k_empty[ks]);
        }
        __syncwarp();
        if (aborted()) ok = false;
      }
    }
    if (!ok) fail();
  } else if (warp == Cfg::PV_ISSUER) {
    // ---------------- P . V issue; an item's first waits until O was read out ----------------
    bool ok = true;
    MqWalk wk;
    wk.start(rg.b0, rg.base0, rg.t0, rg.t1);
    MqSeg sg{};
    int g = 0;
    for (int si = 0; ok && next_item(wk, sg); ++si) {
      if (si > 0) ok = other_wait<Cfg>(&o_free, (uint32_t)(si - 1) & 1u, p.timeout_ns);
      if (lane < 2) spoiled[si & 1][lane] = 0;  // (last used two items ago, whose O was read out)
      const PartialTiles part = partial_tiles(p, sg);
      for (int j = sg.j0; ok && j < sg.j1; ++j, ++g) {
        const int vs = g % Cfg::VSTAGES, sb = g % Cfg::SBUF;
        ok = other_wait<Cfg>(&v_full[vs], (uint32_t)(g / Cfg::VSTAGES) & 1u, p.timeout_ns);
        if (ok && part.has(j) && lane < 2) {
          spoiled[si & 1][lane] |= slot_spoiled[vs][lane];
          slot_spoiled[vs][lane] = 0;
        }
        if (ok) ok = other_wait<Cfg>(&p_full[sb], (uint32_t)(g / Cfg::SBUF) & 1u, p.timeout_ns);
        if (!ok) break;
        tc::fence_after();
        __syncwarp();
        if (lane == 0) {
          mma_pv_tile<Cfg>(tbase + Cfg::COL_O, tbase + (uint32_t)(sb * Cfg::N), smem_u32(sV + (size_t)vs * Cfg::KV_BYTES),
                           j > sg.j0);
          tc::commit(&pv_done[sb]);
          tc::commit(&v_empty[vs]);
        }
        __syncwarp();
        if (aborted()) ok = false;
      }
    }
    if (!ok) fail();
  }
  } else {
    // ---------------- softmax + epilogue: thread (row, half) ----------------
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(Cfg::REGS_SOFTMAX));
    constexpr int SC = Cfg::N / 2;   // S columns of a thread (its half of the row)
    constexpr int NB = SC / kBlock;  // blocks of those columns
    constexpr int OC = Cfg::D / 2;   // O columns of a thread
    const int row = tid & (Cfg::M - 1), half = tid / Cfg::M;
    const int r = rt * Cfg::M + row, node = r / p.G, gq = r - node * p.G;
    const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
    const float c = p.scale_log2;
    // half of this row of an item's Q as E4M3 parts; returns the score factor
    // scale * log2(e) / 2^k of the row (k its scaling; NaN for a row that is not finite)
    auto stage_q = [&](const MqSeg &s) -> float {
      const bool live = node < s.n;
      const uint4 *src = reinterpret_cast<const uint4 *>(
          static_cast<const uint16_t *>(p.q) +
          (((size_t)s.b * p.q_len + (live ? node : 0)) * p.Hq + s.h * p.G + gq) * Cfg::D);
      return c * stage_q_parts<Cfg>(live ? src : nullptr, smem_u32(sQ), row, half * (Cfg::D / 32), (half + 1) * (Cfg::D / 32));
    };
    auto release_q = [&]() {
      __syncwarp();
      if (lane == 0) mbar_arrive(&q_full);
    };
    bool ok = true;
    auto next = [&](int k) -> bool {  // waits until item k is published; whether there is one
      ok = tile_wait(&item_full[k & 3], (uint32_t)(k >> 2) & 1u, p.timeout_ns);
      return ok && items[k & 3].have != 0;
    };
    bool have = next(0);
    float cq = have ? stage_q(items[0].s) : 0.f, cq_next = 0.f;
    if (rt == 0 && tid == 0) {  // (rt 0 has rows in every item with any)
      TreeCut cut{rg.t0, 0, 0, 0, 0};
      const MqSeg &sg = items[0].s;
      if (have && sg.j0 > 0) cut = TreeCut{rg.t0, sg.b, sg.h, rg.t0 - sg.j0, rg.t0 - sg.j0 + sg.T};
      tp.cuts[group] = cut;
    }
    if (have) release_q();
    int g = 0, si = 0, xn = 0;  // tiles and items so far, exchanges of this warp (none in tiles without its rows)
    while (have && ok) {
      const MqSeg &sg = items[si & 3].s;
      const int n = sg.j1 - sg.j0, tile0 = sg.j_first + sg.j0;
      // what this row sees: [lo, start), then node t at start + t iff bit t of mask
      const bool live = node < sg.n;
      const bool dead = rt * Cfg::M + (warp & 3) * 32 >= sg.n * p.G;  // no live row in this warp (nor in the one that shares its rows)
      const int start = sg.ctx - sg.n;
      uint64_t mask = 0;
      int lo = INT32_MAX;
      if (live) {
        mask = __ldg(p.tree_mask + (size_t)sg.b * p.mask_stride + node) & (~0ull >> (64 - sg.n));
        lo = p.window > 0 ? start + max(1, __popcll(mask)) - p.window : 0;
      }
      const int lo_all = p.window > 0 ? start + p.q_len - p.window : 0;  // no row's lo is above it
      // a row that sees nothing gives 0 whatever its query holds: -inf times the factor NaN
      // of a query that is not finite would be NaN
      if (start <= max(lo, 0) && (start < 0 ? mask >> -start : mask) == 0) cq = 1.f;
      float m_run = -INFINITY, l = 0.f;  // l: sum of p' / v_b
      for (int j = 0; j < n; ++j) {
        const int gj = g + j, sb = gj % Cfg::SBUF;
        const bool last = j + 1 == n;
        ok = tile_wait(&s_full[sb], (uint32_t)(gj / Cfg::SBUF) & 1u, p.timeout_ns);
        if (!ok) break;
        tc::fence_after();
        // the item's last S has read Q: the next item's may come in
        if (last) {
          have = next(si + 1);
          if (!ok) break;
          if (have) cq_next = stage_q(items[(si + 1) & 3].s);
        }
        if (dead) {  // (rows past the nodes: their P and O are never looked at)
          tc::fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&p_full[sb]);
          continue;
        }
        const uint32_t scol = tbase + lane_base + (uint32_t)(sb * Cfg::N + half * SC);
        const int kvh = (tile0 + j) * Cfg::N + half * SC;  // first position of this half
        // per block: the score's factor c k_b, log2 v_b and 1 / v_b
        float ck[NB], lv[NB], rv[NB];
        uint32_t lit = 0;  // blocks with literal products
#pragma unroll
        for (int b = 0; b < NB; ++b) {
          const float4 v = scales[gj % Cfg::SCALES][half * NB + b];
          ck[b] = cq * v.x;
          lv[b] = v.y;
          rv[b] = v.z;
          lit |= v.w != 0.f ? 1u << b : 0u;
        }
        const float2 *raw = &literal[gj % Cfg::SCALES][half * NB];
        // (warp-uniform) the tree or a window's edge is in these columns
        const bool edge = kvh + SC > start || kvh < lo_all;
        if (edge || lit) {
          fix_scores(scol, edge ? tree_columns(mask, start, lo, kvh) : ~0ull, raw, lit);
          // hidden scores are -inf: a factor that left 32 bits (a tiny query on a tiny block
          // scale) would make them NaN.  (A NaN factor stays.)
#pragma unroll
          for (int b = 0; b < NB; ++b) ck[b] = ck[b] < 1.17549435e-38f ? 1.17549435e-38f : ck[b];
        }
        uint32_t s[SC];
#pragma unroll
        for (int q = 0; q < SC / 32; ++q)
          tc::ld32(scol + (uint32_t)(q * 32), *reinterpret_cast<uint32_t(*)[32]>(&s[q * 32]));
        float mx = -INFINITY;  // max of s c k_b + lv_b
#pragma unroll
        for (int b = 0; b < NB; ++b) {
          float mb = -INFINITY;
#pragma unroll
          for (int e = 0; e < kBlock; e += 2)
            mb = fmax3(mb, __uint_as_float(s[b * kBlock + e]), __uint_as_float(s[b * kBlock + e + 1]));
          mx = fmaxf(mx, fmaf(mb, ck[b], lv[b]));
        }
        // the row max over both halves (double-buffered exchange, bounded wait)
        const int par = xn & 1;
        red[par][half][row] = mx;
        __syncwarp();
        if (lane == 0) mbar_arrive(&xch[warp & 3][par]);
        ok = warp_wait(&xch[warp & 3][par], (uint32_t)(xn++ >> 1) & 1u, p.timeout_ns);
        if (!ok) break;
        mx = fmaxf(mx, red[par][half ^ 1][row]);
        const float m_new = fmaxf(m_run, mx);
        // warps w and w + 4 hold the same rows and the same m_new: same decision
        const bool rescale = __any_sync(kFull, m_new > m_run + 8.f);
        float alpha = 1.f;
        if (rescale) {
          alpha = m_new == -INFINITY ? 1.f : ex2(m_run - m_new);
          m_run = m_new;
        }
        const float mu = m_run == -INFINITY ? 0.f : m_run;
        uint32_t w[SC / 2];
        float sum = 0.f;
#pragma unroll
        for (int b = 0; b < NB; ++b) {
          const uint64_t cb = f2_pack(ck[b], ck[b]), nb = f2_pack(lv[b] - mu, lv[b] - mu);
          uint64_t sum2 = f2_pack(0.f, 0.f);
#pragma unroll
          for (int e = 0; e < kBlock / 2; ++e) {
            uint32_t unused;
            p_pair<false>(s[b * kBlock + 2 * e], s[b * kBlock + 2 * e + 1], cb, nb, sum2, w[b * 8 + e], unused);
          }
          const float2 sp = f2_unpack(sum2);
          sum = fmaf(sp.x + sp.y, rv[b], sum);
        }
        if (rescale && j > 0) {  // O must hold P . V of the item's previous tile before it is scaled
          ok = warp_wait(&pv_done[(gj - 1) % Cfg::SBUF], (uint32_t)((gj - 1) / Cfg::SBUF) & 1u, p.timeout_ns);
          if (!ok) break;
          tc::fence_after();
          rescale_o(tbase + lane_base + Cfg::COL_O + (uint32_t)(half * OC), alpha, OC);
        }
        l = l * alpha + sum;
        tc::st32(scol, w);  // P over this thread's own (already read) S columns
        tc::wait_st();
        if (lit) fix_weights(scol, raw, lit);
        tc::fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[sb]);
      }
      if (!ok) break;
      if (have) release_q();  // (the next item's)
      // ---- epilogue of the item: O / l, or a normalised partial and its lse ----
      const int gl = g + n - 1;
      ok = tile_wait(&pv_done[gl % Cfg::SBUF], (uint32_t)(gl / Cfg::SBUF) & 1u, p.timeout_ns);
      if (ok) {
        red_l[half][row] = l;
        __syncwarp();
        if (lane == 0) mbar_arrive(&xl);
        ok = tile_wait(&xl, (uint32_t)si & 1u, p.timeout_ns);
      }
      if (!ok) break;
      tc::fence_after();
      const float lt = l + red_l[half ^ 1][row];
      const float inv = lt == 0.f ? 0.f : 1.f / lt;  // a row that sees nothing gives 0 (and a NaN stays one)
      const ulonglong2 sp = *reinterpret_cast<const ulonglong2 *>(spoiled[si & 1]);
      if (sp.x | sp.y)
        add_spoiled<E4M3, Cfg::D>(tp, tbase + lane_base + Cfg::COL_O + (uint32_t)(half * OC), sg.b, sg.h, start, sg.first, sp.x,
                                                 sp.y, mask, lo, half * OC);
      uint32_t o[OC / 32][32];
#pragma unroll
      for (int q = 0; q < OC / 32; ++q)
        tc::ld32(tbase + lane_base + Cfg::COL_O + (uint32_t)(half * OC + q * 32), o[q]);
      tc::fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&o_free);
      if (live && sg.whole) {
        uint4 *dst = reinterpret_cast<uint4 *>(static_cast<uint16_t *>(p.out) +
                                               (((size_t)sg.b * p.q_len + node) * p.Hq + sg.h * p.G + gq) * Cfg::D + half * OC);
#pragma unroll
        for (int q = 0; q < OC / 32; ++q)
#pragma unroll
          for (int v = 0; v < 4; ++v) {
            uint32_t x[4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
              x[e] = pack2<Cfg::OUT_BF>(__uint_as_float(o[q][v * 8 + 2 * e]) * inv, __uint_as_float(o[q][v * 8 + 2 * e + 1]) * inv);
            dst[q * 4 + v] = make_uint4(x[0], x[1], x[2], x[3]);
          }
      } else if (live) {
        // partials lie as [D / 4][128 rows] groups of four: a warp's rows side by side
        const size_t part = ((size_t)blockIdx.x * 2 + sg.slot) * Cfg::M;
        float4 *po = reinterpret_cast<float4 *>(p.part_o + part * Cfg::D) + (size_t)(half * (OC / 4)) * Cfg::M + row;
#pragma unroll
        for (int q = 0; q < OC / 32; ++q)
#pragma unroll
          for (int v = 0; v < 8; ++v)
            po[(size_t)(q * 8 + v) * Cfg::M] =
                make_float4(__uint_as_float(o[q][4 * v]) * inv, __uint_as_float(o[q][4 * v + 1]) * inv,
                            __uint_as_float(o[q][4 * v + 2]) * inv, __uint_as_float(o[q][4 * v + 3]) * inv);
        if (half == 0) p.part_lse[part + row] = partial_lse(m_run, lt);
      }
      g += n;
      ++si;
      cq = cq_next;
    }
    if (ok) {  // sequences with rows but no tile (an empty context): zeros, sequence b by CTA b mod grid
      for (int b = blockIdx.x; b < p.B; b += gridDim.x) {
        const MqSeq s = mq_seq(p, b);
        if (s.T == 0) {
          uint4 *dst = reinterpret_cast<uint4 *>(static_cast<uint16_t *>(p.out) + (size_t)b * p.q_len * p.Hq * Cfg::D);
          for (size_t i = tid; i < (size_t)s.n * p.Hq * Cfg::D / 8; i += Cfg::SOFTMAX) dst[i] = make_uint4(0, 0, 0, 0);
        }
      }
    }
    if (!ok) fail();
  }

  // ---------------- drain, then free tensor memory ----------------
  tc::fence_before();
  __syncthreads();
  if (warp == Cfg::ISSUER || warp == Cfg::PV_ISSUER) {
    if (lane == 0) tc::commit(&fin);  // completes once every MMA either warp issued has
    __syncwarp();
    if (!mbar_wait_bounded(&fin, 0, p.timeout_ns) && lane == 0) atomicOr(&cta_flags, PKV_FLAG_TIMEOUT);
  } else if ((warp == Cfg::PRODUCER || warp == Cfg::V_PRODUCER) && lane == 0) {  // the copies last issued into each slot have landed
    const bool vw = warp == Cfg::V_PRODUCER;
    const int stages = vw ? Cfg::VRAW : Cfg::KSTAGES, n = vw ? r_issued : k_issued;
    for (int i = n > stages ? n - stages : 0; i < n; ++i)
      mbar_wait_bounded(vw ? &r_full[i % stages] : &k_full[i % stages], (uint32_t)(i / stages) & 1u, p.timeout_ns);
  }
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  if (warp == Cfg::ISSUER) tc::dealloc(tbase, Cfg::TMEM_COLS);
  if (tid == 0) write_status(tp, cta_flags);
}

template <class Cfg>
static cudaError_t launch_fp8_cfg(const TreeTileParams &p, const CUtensorMap &tmK, const CUtensorMap &tmV,
                                  cudaStream_t stream) {
  static int configured[64] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorNotSupported;
  if (!configured[dev]) {
    e = cudaFuncSetAttribute(tree_tile_fp8_kernel<Cfg>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)Cfg::SMEM);
    if (e != cudaSuccess) return e;
    configured[dev] = 1;
  }
  const int grid = p.RT * p.groups;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(Cfg::THREADS);
  cfg.dynamicSmemBytes = Cfg::SMEM;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, tree_tile_fp8_kernel<Cfg>, p, tmK, tmV);
  if (e != cudaSuccess) return e;
  return p.cta_status ? cudaSuccess : launch_tree_merge(p, grid, Cfg::OUT_BF ? 1 : 0, stream);
}

cudaError_t launch_tree_tiles_fp8(const TreeTileParams &p, int q_dtype, const CUtensorMap &tmK, const CUtensorMap &tmV,
                                  cudaStream_t stream) {
  if (q_dtype == PKV_BF16) {
    if (p.D == 128) return launch_fp8_cfg<TreeFp8Cfg<128, BF16>>(p, tmK, tmV, stream);
    if (p.D == 64) return launch_fp8_cfg<TreeFp8Cfg<64, BF16>>(p, tmK, tmV, stream);
  } else if (q_dtype == PKV_F16) {
    if (p.D == 128) return launch_fp8_cfg<TreeFp8Cfg<128, F16>>(p, tmK, tmV, stream);
    if (p.D == 64) return launch_fp8_cfg<TreeFp8Cfg<64, F16>>(p, tmK, tmV, stream);
  }
  return cudaErrorNotSupported;
}

}  // namespace pkv
