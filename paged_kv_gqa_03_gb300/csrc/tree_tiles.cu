// tree_tiles.cu — attention of a tree of drafted tokens over the paged cache on
// the tensor cores with the query rows on the M side.  A tile is 128 rows however
// few of them a call has: its K / V bytes bound it up to about 64 rows per kv
// head, so this kernel serves few rows too (tree_route in api.cpp).
//
// The tile pipeline is that of prefill_common.cuh (S = Q . K^T and O += P . V of
// 128 rows x 128 positions, tcgen05, S / P / O in tensor memory, TMA rings
// through the block table, eight softmax warps).  What differs from the
// prefill kernels is the schedule and the mask:
//  * a tree has at most 64 * G rows per kv head but any context, so the context
//    is split: the K / V tiles of all (sequence, kv head) items form one
//    sequence cut into `groups` equal ranges (stream-K, mq_walk.cuh), and the RT
//    row tiles of an item are RT CTAs of one group that walk the same range side
//    by side, so that each K / V tile comes from HBM once and from L2 for the
//    other row tiles.  Items cut between groups leave normalised partials and
//    their log-sum-exps, which tree_merge_kernel joins.
//  * a row sees the cached positions before the tree and the nodes its 64-bit
//    mask names.  A thread holds its row's mask in registers; a tile that
//    touches the tree turns it into a 64-bit word over the thread's 64 columns
//    with two shifts.  Tiles before the tree are not masked at all.
// Warp roles, rings and bounded waits as in prefill_tiles.cu; Q of the next
// item is copied into the one Q buffer while the current item's last tile is in
// the softmax (its last S has been read by then).
//
// Weights enter P . V as in the decode kernels: bf16 caches a high part plus residual (16
// bits), f16 caches as f16 (2^-11 each, 2.9e-4 of the outputs' size with their own rounding
// against 2.1e-4 by fp32 weights; a second f16 part would cost another product).
//
// What bounds it.  Up to about 64 rows per kv head, the K / V bytes: 64 / 8 heads,
// 16 x 8192, 1 - 8 nodes 98 - 100 us (5.4 TB/s with ~11 us of start, first tile and
// merge), 32 x 8192, 1 - 4 nodes 176 us (6.1 TB/s); DRAM reads are 1.002 - 1.005 times
// the bytes.  With full tiles about 2250 clocks a tile: its MMAs are 1536 (bf16: P's high parts
// and residuals are two products; f16 1024), its operands and copies 192 KiB of
// shared memory traffic, 1536 clocks too, and the eight softmax warps issue over 40% of the
// time (one sequence of 131072, 26 nodes: 150 - 159 us, tensor pipe 60% active; 32 x 8192, 64
// nodes: 562 - 609 us, 900 - 980 TFLOP/s as the formula counts them and 1350 - 1460 as issued, near
// the board's power limit).  The tile loop is short of registers: with every softmax thread walking the
// items by itself it spilled and these two took 159 and 604 us.  Measured against that
// version, at 157 and 591 us without the check of V, and slower or equal: a second group of
// softmax warps taking every other tile (152 and 563 - 600, but 106 against 97 for 24 x
// 512 - 2048 with 32 heads), two groups with S and O of their own (188 and 717), part of the
// 2^x as polynomials on the FMA pipes (153 and 581; f16 100 against 97), deeper rings at head
// dim 64 (equal).
#include "prefill_common.cuh"
#include "tree_tiles.cuh"

namespace pkv {

template <class T, int D_>
struct TreeCfg : PrefillCfg<T, D_> {
  using Cache = T;
  using Base = PrefillCfg<T, D_>;
  static constexpr int STAGE_BYTES = Base::SOFTMAX / 32 * 2048;  // output staging, 2 KiB per softmax warp
  static constexpr size_t SMEM = Base::SMEM + STAGE_BYTES;
  static_assert(SMEM + 6144 <= 232448, "shared memory");
};

// (tree_finite.cuh) The rows of a V tile, positions kv0 + r below ctx, that not every row of Q sees:
// what is not finite becomes 0, noted in `spoiled`.  Warp-wide, out of the issuing loop.
template <class Cfg>
static __device__ __noinline__ void clean_v_rows(uint8_t *vt, int kv0, int ctx, TreePartial t, unsigned long long *spoiled) {
  constexpr int CPR = 8 * Cfg::PANELS, U = 8;  // chunks per row, in flight
  const int lane = threadIdx.x & 31;
  auto at = [&](int i) {
    const int r = i / CPR, c = i % CPR;
    return smem_u32(vt + (c >> 3) * Cfg::PANEL_KV + r * 128 + (c & 7) * 16);
  };
#pragma unroll 1
  for (int part = 0; part < 2; ++part) {  // the tree's rows, a window's edge
    const int i0 = part ? lane : max(t.start - kv0, 0) * CPR + lane;
    const int i1 = min(part ? t.edge - kv0 : Cfg::N, min(ctx - kv0, Cfg::N)) * CPR;
#pragma unroll 1
    for (int i = i0; i < i1; i += 32 * U) {
      uint4 v[U];
#pragma unroll
      for (int u = 0; u < U; ++u) v[u] = lds128(at(min(i + 32 * u, i1 - 1)));  // (the last chunk again past the end)
      uint32_t bad = 0;
#pragma unroll
      for (int u = 0; u < U; ++u) bad |= nonfinite_any<typename Cfg::Cache>(v[u]);
      if (bad != 0) {
        TreeSpoiled s{0, 0};
#pragma unroll 1
        for (int u = 0; u < U; ++u) {
          const int k = i + 32 * u;
          if (k < i1 && clear_nonfinite<typename Cfg::Cache>(at(k))) s.note(t, kv0 + k / CPR);
        }
        if (s.nodes) atomicOr(&spoiled[0], (unsigned long long)s.nodes);
        if (s.edge) atomicOr(&spoiled[1], (unsigned long long)s.edge);
        fence_proxy_async();
      }
    }
  }
  __syncwarp();
}

template <class Cfg>
__global__ void __launch_bounds__(Cfg::THREADS, 1)
    tree_tile_kernel(const __grid_constant__ TreeTileParams tp, const __grid_constant__ CUtensorMap tmK,
                     const __grid_constant__ CUtensorMap tmV) {
  const MqParams &p = tp.m;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint8_t *sQ = smem;
  uint8_t *sK = sQ + Cfg::Q_BYTES;
  uint8_t *sV = sK + (size_t)Cfg::KSTAGES * Cfg::KV_BYTES;
  uint8_t *sOut = sV + (size_t)Cfg::VSTAGES * Cfg::KV_BYTES;
  __shared__ __align__(8) uint64_t k_full[Cfg::KSTAGES], k_empty[Cfg::KSTAGES];
  __shared__ __align__(8) uint64_t v_full[Cfg::VSTAGES], v_empty[Cfg::VSTAGES];
  __shared__ __align__(8) uint64_t s_full[Cfg::SBUF], p_full[Cfg::SBUF], pv_done[Cfg::SBUF];
  __shared__ __align__(8) uint64_t q_full, o_free, xl, fin;  // per item: Q staged, O read out, row sums exchanged
  __shared__ __align__(8) uint64_t xch[Cfg::SOFTMAX / 64][2];
  __shared__ float red[2][2][Cfg::M];
  __shared__ float red_l[2][Cfg::M];
  __shared__ TreeItem items[4];
  __shared__ __align__(8) uint64_t item_full[4];
  __shared__ __align__(16) unsigned long long spoiled[2][2];  // [item parity][nodes, window's edge]
  __shared__ TreeFind find;
  __shared__ uint32_t tmem_base;
  __shared__ int abort_flag, cta_flags, k_consumed, v_consumed, k_issued, v_issued;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rt = (int)blockIdx.x % tp.RT, group = (int)blockIdx.x / tp.RT;
  if (tid == 0) {
#pragma unroll
    for (int s = 0; s < Cfg::KSTAGES; ++s) {
      mbar_init(&k_full[s], 1);
      mbar_init(&k_empty[s], 1);
    }
#pragma unroll
    for (int s = 0; s < Cfg::VSTAGES; ++s) {
      mbar_init(&v_full[s], 1);
      mbar_init(&v_empty[s], 1);
    }
#pragma unroll
    for (int s = 0; s < Cfg::SBUF; ++s) {
      mbar_init(&s_full[s], 1);
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
    fence_barrier_init();
    abort_flag = 0;
    cta_flags = 0;
    k_consumed = v_consumed = k_issued = v_issued = 0;
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

  if (warp == Cfg::PRODUCER || warp == Cfg::V_PRODUCER) {
    // ---------------- TMA producers: K tiles (warp 8), V tiles (warp 10) ----------------
    // lane l fetches block (l % 8) of a tile, panel l / 8; block ids are
    // loaded three tiles ahead and first used when the tile's copies are issued
    const int slot = lane & (Cfg::BLOCKS - 1), panel = lane / Cfg::BLOCKS;
    MqWalk wk;
    wk.start(rg.b0, rg.base0, rg.t0, rg.t1);
    MqSeg cs{};
    int cj = 0;
    bool have = false;
    auto step = [&]() -> bool {  // to the cursor's next tile; false past the CTA's last
      if (have && ++cj < cs.j1) return true;
      have = next_item(wk, cs);
      if (have) cj = cs.j0;
      return have;
    };
    int bad = 0;
    struct Pend {
      int id, h;
      bool none;
    };
    auto fetch = [&]() -> Pend {
      Pend f;
      const int lb = (cs.j_first + cj) * Cfg::BLOCKS + slot;
      const int nblk = (cs.ctx + kBlock - 1) / kBlock;
      f.h = cs.h;
      f.none = lb >= nblk || (lb + 1) * kBlock <= cs.first;
      f.id = f.none ? 0 : __ldg(p.block_table + (size_t)cs.b * p.max_blocks + lb);
      return f;
    };
    // the box row of a fetched block; the box past the tensor (zeros) for none or a bad id
    auto row_of = [&](const Pend &f) -> int64_t {
      if (f.none) return p.num_blocks * p.Hkv;
      const bool good = f.id >= 0 && (int64_t)f.id < p.num_blocks;
      bad |= good ? 0 : 1;
      return good ? (int64_t)f.id * p.Hkv + f.h : p.num_blocks * p.Hkv;
    };
    const bool vw = warp == Cfg::V_PRODUCER;
    uint8_t *ring = vw ? sV : sK;
    uint64_t *full = vw ? v_full : k_full, *empty = vw ? v_empty : k_empty;
    const int stages = vw ? Cfg::VSTAGES : Cfg::KSTAGES;
    const CUtensorMap *tm = vw ? &tmV : &tmK;
    int *issued = vw ? &v_issued : &k_issued;
    bool ok = true;
    const Pend nil{0, 0, true};
    bool h0 = step();
    Pend f0 = h0 ? fetch() : nil;
    bool h1 = h0 && step();
    Pend f1 = h1 ? fetch() : nil;
    bool h2 = h1 && step();
    Pend f2 = h2 ? fetch() : nil;
    for (int g = 0; h0; ++g) {
      const bool h3 = h2 && step();
      const Pend f3 = h3 ? fetch() : nil;
      const int64_t trow = row_of(f0);
      const int s = g % stages;
      if (g >= stages) ok = tile_wait(&empty[s], (uint32_t)((g / stages) - 1) & 1u, p.timeout_ns);
      if (!ok || __any_sync(kFull, *(volatile int *)&abort_flag)) {
        ok = false;
        break;
      }
      if (lane == 0) mbar_arrive_expect_tx(&full[s], Cfg::KV_BYTES);
      __syncwarp();
      if (lane < Cfg::LOADS)
        tma_load_2d(ring + (size_t)s * Cfg::KV_BYTES + panel * Cfg::PANEL_KV + slot * 2048, tm, panel * 64,
                    (int)(trow * kBlock), &full[s]);
      if (lane == 0) *issued = g + 1;
      h0 = h1;
      f0 = f1;
      h1 = h2;
      f1 = f2;
      h2 = h3;
      f2 = f3;
    }
    if (__any_sync(kFull, bad) && lane == 0) atomicOr(&cta_flags, PKV_FLAG_BAD_BLOCK);
    if (!ok && lane == 0) {
      atomicOr(&cta_flags, PKV_FLAG_TIMEOUT);
      abort_flag = 1;
    }
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
      ok = tile_wait(&q_full, (uint32_t)si & 1u, p.timeout_ns);
      for (int j = sg.j0; ok && j < sg.j1; ++j, ++g) {
        const int ks = g % Cfg::KSTAGES, sb = g % Cfg::SBUF;
        ok = tile_wait(&k_full[ks], (uint32_t)(g / Cfg::KSTAGES) & 1u, p.timeout_ns);
        // S overwrites the buffer whose P . V of tile g - SBUF read P from it
        if (ok && g >= Cfg::SBUF)
          ok = tile_wait(&pv_done[sb], (uint32_t)((g / Cfg::SBUF) - 1) & 1u, p.timeout_ns);
        if (!ok) break;
        if (lane == 0) k_consumed = g + 1;
        tc::fence_after();
        if (lane == 0) {
          mma_s_tile<Cfg>(tbase + (uint32_t)(sb * Cfg::N), smem_u32(sQ), smem_u32(sK + (size_t)ks * Cfg::KV_BYTES));
          tc::commit(&s_full[sb]);
          tc::commit(&k_empty[ks]);
        }
        __syncwarp();
        if (__any_sync(kFull, *(volatile int *)&abort_flag)) ok = false;
      }
    }
    if (!ok && lane == 0) {
      atomicOr(&cta_flags, PKV_FLAG_TIMEOUT);
      abort_flag = 1;
    }
  } else if (warp == Cfg::PV_ISSUER) {
    // ---------------- P . V issue; an item's first waits until O was read out ----------------
    bool ok = true;
    MqWalk wk;
    wk.start(rg.b0, rg.base0, rg.t0, rg.t1);
    MqSeg sg{};
    int g = 0;
    for (int si = 0; ok && next_item(wk, sg); ++si) {
      if (si > 0) ok = tile_wait(&o_free, (uint32_t)(si - 1) & 1u, p.timeout_ns);
      if (lane < 2) spoiled[si & 1][lane] = 0;  // (last used two items ago, whose O was read out)
      __syncwarp();
      const PartialTiles part = partial_tiles(p, sg);
      const int nblk = (sg.ctx + kBlock - 1) / kBlock;
      for (int j = sg.j0; ok && j < sg.j1; ++j, ++g) {
        const int vs = g % Cfg::VSTAGES, sb = g % Cfg::SBUF;
        ok = tile_wait(&v_full[vs], (uint32_t)(g / Cfg::VSTAGES) & 1u, p.timeout_ns);
        uint8_t *vt = sV + (size_t)vs * Cfg::KV_BYTES;
        const int kv0 = (sg.j_first + j) * Cfg::N;  // first position of the tile
        if (ok && part.has(j)) clean_v_rows<Cfg>(vt, kv0, sg.ctx, tree_partial(p, sg), spoiled[si & 1]);
        if (ok) ok = tile_wait(&p_full[sb], (uint32_t)(g / Cfg::SBUF) & 1u, p.timeout_ns);
        if (!ok) break;
        if (lane == 0) v_consumed = g + 1;
        zero_v_rows<Cfg>(vt, sg.ctx - kv0, min(nblk * kBlock - kv0, Cfg::N), lane);
        __syncwarp();
        tc::fence_after();
        if (lane == 0) {
          mma_pv_tile<Cfg>(tbase + Cfg::COL_O, tbase + (uint32_t)(sb * Cfg::N), smem_u32(vt), j > sg.j0);
          tc::commit(&pv_done[sb]);
          tc::commit(&v_empty[vs]);
        }
        __syncwarp();
        if (__any_sync(kFull, *(volatile int *)&abort_flag)) ok = false;
      }
    }
    if (!ok && lane == 0) {
      atomicOr(&cta_flags, PKV_FLAG_TIMEOUT);
      abort_flag = 1;
    }
  } else {
    // ---------------- softmax + epilogue: thread (row, half) ----------------
    constexpr int SC = Cfg::N / 2;  // S columns of a thread (its half of the row)
    constexpr int OC = Cfg::D / 2;  // O columns of a thread
    const int row = tid & (Cfg::M - 1), half = tid / Cfg::M;
    const int r = rt * Cfg::M + row, node = r / p.G, gq = r - node * p.G;
    const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
    const float c = p.scale_log2;
    // half of this row of an item's Q (zeros for a row past the nodes)
    auto stage_q = [&](const MqSeg &s) {
      const bool live = node < s.n;
      const uint16_t *src = static_cast<const uint16_t *>(p.q) +
                            (((size_t)s.b * p.q_len + (live ? node : 0)) * p.Hq + s.h * p.G + gq) * Cfg::D;
#pragma unroll
      for (int k = 0; k < Cfg::D / 16; ++k) {
        const int ch = half * (Cfg::D / 16) + k;
        const uint32_t dst = smem_u32(sQ + (ch >> 3) * Cfg::PANEL_Q + row * 128 + (((ch & 7) ^ (row & 7)) << 4));
        if (live)
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src + ch * 8) : "memory");
        else
          sts128(dst, make_uint4(0, 0, 0, 0));
      }
    };
    auto release_q = [&]() {
      asm volatile("cp.async.wait_all;" ::: "memory");
      fence_proxy_async();
      __syncwarp();
      if (lane == 0) mbar_arrive(&q_full);
    };
    bool ok = true;
    auto next = [&](int k) -> bool {  // waits until item k is published; whether there is one
      ok = tile_wait(&item_full[k & 3], (uint32_t)(k >> 2) & 1u, p.timeout_ns);
      return ok && items[k & 3].have != 0;
    };
    bool have = next(0);
    if (have) stage_q(items[0].s);
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
      float m_run = -INFINITY, l = 0.f;
      for (int j = 0; j < n; ++j) {
        const int gj = g + j, sb = gj % Cfg::SBUF;
        ok = tile_wait(&s_full[sb], (uint32_t)(gj / Cfg::SBUF) & 1u, p.timeout_ns);
        if (!ok) break;
        tc::fence_after();
        // the item's last S has read Q: the next item's may come in
        if (j + 1 == n) {
          have = next(si + 1);
          if (!ok) break;
          if (have) stage_q(items[(si + 1) & 3].s);
        }
        if (dead) {  // (rows past the nodes: their P and O are never looked at)
          tc::fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&p_full[sb]);
          continue;
        }
        const uint32_t scol = tbase + lane_base + (uint32_t)(sb * Cfg::N + half * SC);
        const int kvh = (tile0 + j) * Cfg::N + half * SC;  // first position of this half
        if (kvh + SC > start || kvh < lo_all)  // (warp-uniform) the tree or a window's edge is in these columns
          fix_scores(scol, tree_columns(mask, start, lo, kvh), nullptr, 0);
        uint32_t s[SC];
#pragma unroll
        for (int q = 0; q < SC / 32; ++q)
          tc::ld32(scol + (uint32_t)(q * 32), *reinterpret_cast<uint32_t(*)[32]>(&s[q * 32]));
        float mx = -INFINITY;
#pragma unroll
        for (int e = 0; e < SC; e += 2) mx = fmax3(mx, __uint_as_float(s[e]), __uint_as_float(s[e + 1]));
        // the row max over both halves (double-buffered exchange, bounded wait)
        const int par = xn & 1;
        red[par][half][row] = mx;
        __syncwarp();
        if (lane == 0) mbar_arrive(&xch[warp & 3][par]);
        ok = warp_wait(&xch[warp & 3][par], (uint32_t)(xn++ >> 1) & 1u, p.timeout_ns);
        if (!ok) break;
        mx = fmaxf(mx, red[par][half ^ 1][row]);
        const float m_new = fmaxf(m_run, mx * c);
        // warps w and w + 4 hold the same rows and the same m_new: same decision
        const bool rescale = __any_sync(kFull, m_new > m_run + 8.f);
        float alpha = 1.f;
        if (rescale) {
          alpha = m_new == -INFINITY ? 1.f : ex2(m_run - m_new);
          m_run = m_new;
        }
        const float mu = m_run == -INFINITY ? 0.f : m_run;
        const uint64_t cmu = f2_pack(c, c), nmu = f2_pack(-mu, -mu);
        uint64_t sum2 = f2_pack(0.f, 0.f);
        uint32_t w[SC / 2], wl[Cfg::BF ? SC / 2 : 1];
#pragma unroll
        for (int e = 0; e < SC / 2; ++e) {
          uint32_t lo_;
          p_pair<Cfg::BF>(s[2 * e], s[2 * e + 1], cmu, nmu, sum2, w[e], lo_);
          if constexpr (Cfg::BF) wl[e] = lo_;
        }
        const float2 sp = f2_unpack(sum2);
        if (rescale && j > 0) {  // O must hold P . V of the item's previous tile before it is scaled
          ok = warp_wait(&pv_done[(gj - 1) % Cfg::SBUF], (uint32_t)((gj - 1) / Cfg::SBUF) & 1u, p.timeout_ns);
          if (!ok) break;
          tc::fence_after();
          rescale_o(tbase + lane_base + Cfg::COL_O + (uint32_t)(half * OC), alpha, OC);
        }
        l = l * alpha + (sp.x + sp.y);
        // P (bf16: high parts and residuals; f16: f16 pairs) over this thread's own (already read) S columns
        tc::st32(scol, w);
        if constexpr (Cfg::BF) tc::st32(scol + 32, wl);
        tc::wait_st();
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
        add_spoiled<typename Cfg::Cache, Cfg::D>(tp, tbase + lane_base + Cfg::COL_O + (uint32_t)(half * OC), sg.b, sg.h, start, sg.first, sp.x,
                                                 sp.y, mask, lo, half * OC);
      uint32_t o[OC / 32][32];
#pragma unroll
      for (int q = 0; q < OC / 32; ++q)
        tc::ld32(tbase + lane_base + Cfg::COL_O + (uint32_t)(half * OC + q * 32), o[q]);
      tc::fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&o_free);
      if (sg.whole) {
        uint4 *dst = live ? reinterpret_cast<uint4 *>(static_cast<uint16_t *>(p.out) +
                                                      (((size_t)sg.b * p.q_len + node) * p.Hq + sg.h * p.G + gq) * Cfg::D +
                                                      half * OC)
                          : nullptr;
        store_rows_staged<Cfg>(o, inv, dst, sOut + (size_t)(warp * 2048), lane);
      } else if (live) {
        // partials lie as [D / 4][128 rows] groups of four: a warp's rows side by side
        const size_t part = ((size_t)blockIdx.x * 2 + sg.slot) * Cfg::M;
        float4 *po = reinterpret_cast<float4 *>(p.part_o + part * Cfg::D) + (size_t)(half * (OC / 4)) * Cfg::M + row;
#pragma unroll
        for (int q = 0; q < OC / 32; ++q)
#pragma unroll
          for (int v = 0; v < 8; ++v)
            po[(size_t)(q * 8 + v) * Cfg::M] = make_float4(__uint_as_float(o[q][4 * v]) * inv, __uint_as_float(o[q][4 * v + 1]) * inv,
                                        __uint_as_float(o[q][4 * v + 2]) * inv, __uint_as_float(o[q][4 * v + 3]) * inv);
        if (half == 0) p.part_lse[part + row] = partial_lse(m_run, lt);
      }
      g += n;
      ++si;
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
    if (!ok && lane == 0) {
      atomicOr(&cta_flags, PKV_FLAG_TIMEOUT);
      abort_flag = 1;
    }
  }

  // ---------------- drain, then free tensor memory ----------------
  tc::fence_before();
  __syncthreads();
  if (warp == Cfg::ISSUER || warp == Cfg::PV_ISSUER) {
    if (lane == 0) tc::commit(&fin);  // completes once every MMA either warp issued has
    __syncwarp();
    if (!mbar_wait_bounded(&fin, 0, p.timeout_ns) && lane == 0) atomicOr(&cta_flags, PKV_FLAG_TIMEOUT);
  } else if (warp == Cfg::PRODUCER && lane == 0) {  // copies issued but never consumed (abort only)
    for (int j = k_consumed; j < k_issued; ++j)
      mbar_wait_bounded(&k_full[j % Cfg::KSTAGES], (uint32_t)(j / Cfg::KSTAGES) & 1u, p.timeout_ns);
    for (int j = v_consumed; j < v_issued; ++j)
      mbar_wait_bounded(&v_full[j % Cfg::VSTAGES], (uint32_t)(j / Cfg::VSTAGES) & 1u, p.timeout_ns);
  } else if (tid < Cfg::SOFTMAX) {
    asm volatile("cp.async.wait_all;" ::: "memory");  // a Q copy left in flight by an abort
  }
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  if (warp == Cfg::ISSUER) tc::dealloc(tbase, Cfg::TMEM_COLS);
  if (tid == 0) write_status(tp, cta_flags);
}

// Finishes the items cut between groups: block (x, y) takes row tile x % RT and
// the y-th 16 head-dim elements of the item that group c = x / RT + 1's range
// starts inside, if c's is the item's first cut: the partials of groups
// c - 1 .. (the item's last) are joined with weights 2^(lse - max lse) (rows
// every partial leaves empty give 0).  Thread (row, 8 elements).  Block (0, 0)
// publishes the status bits.
__global__ void __launch_bounds__(2 * kTreeTileRows)
    tree_merge_kernel(const __grid_constant__ TreeTileParams tp, int n_ctas, int out_bf16) {
  const MqParams &p = tp.m;
  __shared__ int s_last;
  const int tid = threadIdx.x, lane = tid & 31;
  grid_dep_wait();
  if (blockIdx.x == 0 && blockIdx.y == 0 && tid < 32) {
    int f = 0;
    for (int c = tid; c < n_ctas; c += 32) f |= p.cta_flags[c];
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) f |= __shfl_xor_sync(kFull, f, off);
    if (tid == 0) *p.status = f;
  }
  const int c = (int)blockIdx.x / tp.RT + 1, rt = (int)blockIdx.x % tp.RT;
  if (c >= tp.groups) return;
  const TreeCut cut = tp.cuts[c];
  const int first = tp.cuts[c - 1].t0;
  if (cut.e == 0 || first > cut.a) return;  // no item cut here, or an earlier cut merges it
  if (tid < 32) {  // the last group whose range starts inside the item
    int last = c;
    for (int w = c; w < tp.groups; w += 32) {
      const bool in = w + lane < tp.groups && tp.cuts[w + lane].t0 < cut.e;
      const unsigned m = __ballot_sync(kFull, in);
      if (m == 0) break;
      last = w + 31 - __clz(m);
      if (m != kFull) break;
    }
    if (lane == 0) s_last = last;
  }
  const int n = p.tree_lens != nullptr ? min(max(__ldg(p.tree_lens + cut.b), 0), p.q_len) : p.q_len;
  __syncthreads();
  const int last = s_last;
  const int row = tid & (kTreeTileRows - 1), r = rt * kTreeTileRows + row;
  if (r >= n * p.G) return;
  const int D = tp.D, d8 = (int)blockIdx.y * 2 + tid / kTreeTileRows;  // elements 8 d8 .. 8 d8 + 7
  constexpr int kBatch = 4;  // partials whose loads are in flight together
  float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  float M = -INFINITY, den = 0.f;
  for (int w0 = c - 1; w0 <= last; w0 += kBatch) {
    float4 x[kBatch], y[kBatch];
    float l[kBatch], cm = -INFINITY;
#pragma unroll
    for (int t = 0; t < kBatch; ++t) {
      l[t] = -INFINITY;
      x[t] = y[t] = make_float4(0.f, 0.f, 0.f, 0.f);
      const int w = w0 + t;
      if (w <= last) {
        // the item's part of group w: slot 0 if w's range starts in the item, else (c - 1, unless the item is its first) 1
        const int slot = w >= c || first == cut.a ? 0 : 1;
        const size_t part = (((size_t)w * tp.RT + rt) * 2 + slot) * kTreeTileRows;
        l[t] = p.part_lse[part + row];
        const float4 *po = reinterpret_cast<const float4 *>(p.part_o + part * D) + (size_t)(2 * d8) * kTreeTileRows + row;
        x[t] = po[0];
        y[t] = po[kTreeTileRows];
      }
    }
#pragma unroll
    for (int t = 0; t < kBatch; ++t) cm = fmaxf(cm, l[t]);
    if (cm == -INFINITY) continue;
    const float mn = fmaxf(M, cm), rescale = exp2f(M - mn);
#pragma unroll
    for (int e = 0; e < 8; ++e) acc[e] *= rescale;
    den *= rescale;
#pragma unroll
    for (int t = 0; t < kBatch; ++t) {
      const float wt = l[t] == -INFINITY ? 0.f : exp2f(l[t] - mn);
      const float v[8] = {x[t].x, x[t].y, x[t].z, x[t].w, y[t].x, y[t].y, y[t].z, y[t].w};
#pragma unroll
      for (int e = 0; e < 8; ++e) acc[e] = fmaf(wt, v[e], acc[e]);
      den += wt;
    }
    M = mn;
  }
  const float inv = den > 0.f ? 1.f / den : 0.f;
  const int node = r / p.G, gq = r - node * p.G;
  const size_t idx = (((size_t)cut.b * p.q_len + node) * p.Hq + cut.h * p.G + gq) * D + 8 * d8;
  uint32_t o[4];
#pragma unroll
  for (int e = 0; e < 4; ++e)
    o[e] = out_bf16 ? pack_bf16x2(acc[2 * e] * inv, acc[2 * e + 1] * inv) : pack_f16x2(acc[2 * e] * inv, acc[2 * e + 1] * inv);
  *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(p.out) + idx) = make_uint4(o[0], o[1], o[2], o[3]);
}

cudaError_t launch_tree_merge(const TreeTileParams &p, int grid, int out_bf16, cudaStream_t stream) {
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t mc = {};
  mc.gridDim = dim3((unsigned)(p.groups > 1 ? (p.groups - 1) * p.RT : 1), (unsigned)(p.D / 16));
  mc.blockDim = dim3(2 * kTreeTileRows);
  mc.stream = stream;
  mc.attrs = attr;
  mc.numAttrs = 1;
  return cudaLaunchKernelEx(&mc, tree_merge_kernel, p, grid, out_bf16);
}

void tree_tiles_grid(int R, int sms, int *RT, int *groups) {
  *RT = (R + kTreeTileRows - 1) / kTreeTileRows;
  *groups = *RT >= sms ? 1 : sms / *RT;
}

static inline size_t tt_align(size_t x) { return (x + 255) / 256 * 256; }

MqWsLayout tree_tiles_ws_layout(int D, int RT, int groups) {
  const size_t grid = (size_t)RT * groups;
  MqWsLayout L;
  size_t o = tt_align(sizeof(WsHeader));
  L.prefix = o;  // the groups' cuts
  o = tt_align(o + sizeof(TreeCut) * (size_t)groups);
  L.cta_flags = o;
  o = tt_align(o + sizeof(int32_t) * grid);
  L.part_o = o;
  o = tt_align(o + sizeof(float) * grid * 2 * kTreeTileRows * D);
  L.part_lse = o;
  o = tt_align(o + sizeof(float) * grid * 2 * kTreeTileRows);
  L.total = o;
  return L;
}

template <class Cfg>
static cudaError_t launch_tiles_cfg(const TreeTileParams &p, const CUtensorMap &tmK, const CUtensorMap &tmV,
                                    cudaStream_t stream) {
  static int configured[64] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorNotSupported;
  if (!configured[dev]) {
    e = cudaFuncSetAttribute(tree_tile_kernel<Cfg>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)Cfg::SMEM);
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
  e = cudaLaunchKernelEx(&cfg, tree_tile_kernel<Cfg>, p, tmK, tmV);
  if (e != cudaSuccess) return e;
  return p.cta_status ? cudaSuccess : launch_tree_merge(p, grid, Cfg::BF ? 1 : 0, stream);
}

cudaError_t launch_tree_tiles(const TreeTileParams &p, int cache_dtype, int q_dtype, const CUtensorMap &tmK, const CUtensorMap &tmV,
                              cudaStream_t stream) {
  if (p.m.B < 1 || p.m.B > kMqMaxBatch || p.RT < 1 || p.groups < 1) return cudaErrorNotSupported;
  if (cache_dtype == PKV_BF16) {
    if (p.D == 128) return launch_tiles_cfg<TreeCfg<BF16, 128>>(p, tmK, tmV, stream);
    if (p.D == 64) return launch_tiles_cfg<TreeCfg<BF16, 64>>(p, tmK, tmV, stream);
  } else if (cache_dtype == PKV_F16) {
    if (p.D == 128) return launch_tiles_cfg<TreeCfg<F16, 128>>(p, tmK, tmV, stream);
    if (p.D == 64) return launch_tiles_cfg<TreeCfg<F16, 64>>(p, tmK, tmV, stream);
  } else if (cache_dtype == PKV_FP8_E4M3) {
    return launch_tree_tiles_fp8(p, q_dtype, tmK, tmV, stream);
  }
  return cudaErrorNotSupported;
}

}  // namespace pkv
