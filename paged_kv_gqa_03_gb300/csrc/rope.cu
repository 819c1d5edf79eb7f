// rope.cu — rotary positions of the queries and keys of new tokens, and the
// rotated keys and the values written into their cache slots (the
// apply_rotary_emb in front of the cache update of "大模型推理加速——KV Cache篇"
// §3.1 Attention.forward, joined with the update itself).
//
// Pair i of a head's first `rot` elements is turned by position * f_i:
//   (a, b) -> m (a cos - b sin, b cos + a sin),
// a pair being elements (i, i + rot / 2), or (2 i, 2 i + 1) when interleaved.
//
// The angle.  f_i comes as turns a position in 2^-64 (uint64): position * turns
// mod 2^64 is then the fraction of a turn without a further rounding, whatever the position, with one
// integer product; as a float in half turns it goes to sincospi.  What is off is the table's entry,
// f_i / 2 pi in double: |position| (2^-52 f_i + 2^-61) radians, 2^-32 at 10^6.  (A 32-bit
// product position * f_i is off by 0.06 radians there.)  A token's
// rot / 2 sines are computed once a CTA and read by all heads.
//
// Split.  A CTA takes one token, or some heads of it; a thread turns 16 bytes of
// each half of a pair's run (interleaved: 32 bytes), U of them, and has them in flight
// before it waits for the sines.  Bound by HBM for prompts (each row read and
// written once: 16384 tokens, 64 + 8 + 8 heads of 128 in bf16, 671 MB in 107 us, 6.3 TB/s of the 6.8 that a
// copy reaches; 122 us with 256 threads of three items, 118 without the bound on registers), by
// latency for a decode step, whose heads are spread over more CTAs (64 tokens: 7 us).
// 4-bit caches: the rows, rounded to their type as a cache of that type would hold
// them, pass through shared memory to groups of 16; V's codes go out by exclusive ors, token by token.  16384
// tokens as above (623 MB) 116 us, 5.4 TB/s; 2048 21 us, 64 5 us; with a unit of 2^-4, by divisions, 131, 23 and 6.
#include "kv4.cuh"
#include "kv4.h"

namespace pkv {

namespace {

constexpr int kThreads = 128;
constexpr int kMaxPairs = 64;  // rot / 2, head dim 128

enum Dest { kRows, kCache, kCache4 };

template <class T>
struct RopeVec {
  static constexpr int VEC = 16 / T::kBytes;  // elements of a 16-byte access
};

template <class T>
__device__ __forceinline__ void unpack_vec(const uint4 &r, float *x) {
  const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (T::kBytes == 4) {
      x[i] = __uint_as_float(w[i]);
    } else {
      const float2 v = unpack2(T{}, w[i]);
      x[2 * i] = v.x;
      x[2 * i + 1] = v.y;
    }
  }
}
template <class T>
__device__ __forceinline__ uint4 pack_vec(const float *x) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (T::kBytes == 4)
      w[i] = __float_as_uint(x[i]);
    else
      w[i] = pack2(T{}, x[2 * i], x[2 * i + 1]);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// Which 16-byte chunks of a row item c of it holds, and whether they turn.
struct Chunks {
  int lo, hi;
  bool turn;
};
template <int VEC>
__device__ __forceinline__ Chunks chunks(const RopeParams &p, int c, bool value) {
  Chunks r;
  const int rc = p.rot / 2 / VEC;  // items of a row that turn
  r.turn = !value && c < rc;
  if (r.turn && !p.interleaved) {
    r.lo = c;
    r.hi = c + rc;
  } else {
    r.lo = 2 * c;
    r.hi = 2 * c + 1;
  }
  return r;
}

template <class T, int DEST, int U>
__global__ void __launch_bounds__(kThreads, 8) rope_kernel(const RopeParams p, int parts, int per_part) {
  using Type = T;
  constexpr int VEC = RopeVec<T>::VEC;
  __shared__ float s_cos[kMaxPairs], s_sin[kMaxPairs];
  extern __shared__ __align__(16) uint8_t s_rows[];  // (kCache4) this part's K and V rows
  grid_dep_launch();  // the next kernel of the chain may come up; it waits for this one
  grid_dep_wait();
  const int64_t t = blockIdx.x / parts;
  const int h0 = (int)(blockIdx.x - t * parts) * per_part;
  const int heads = p.Hq + (DEST == kRows ? 1 : 2) * p.Hkv;
  const int hn = min(per_part, heads - h0);
  const int items_row = p.D / (2 * VEC), items = hn * items_row;

  // the source row of head hh, and whether it is a value's
  auto source = [&](int hh, bool *value) -> const uint4 * {
    *value = hh >= p.Hq + p.Hkv;
    const void *base = hh < p.Hq ? p.q : (*value ? p.v : p.k);
    const int64_t ld = hh < p.Hq ? p.ld_q : (*value ? p.ld_v : p.ld_k);
    const int h = hh < p.Hq ? hh : (hh - p.Hq) % max(p.Hkv, 1);
    return reinterpret_cast<const uint4 *>(static_cast<const uint8_t *>(base) +
                                           (size_t)(t * ld + (int64_t)h * p.D) * T::kBytes);
  };

  uint4 lo[U], hi[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int i = threadIdx.x + u * kThreads;
    if (i < items) {
      bool value;
      const uint4 *src = source(h0 + i / items_row, &value);
      const Chunks c = chunks<VEC>(p, i % items_row, value);
      lo[u] = src[c.lo];
      hi[u] = src[c.hi];
    }
  }
  const int64_t slot = DEST == kRows ? 0 : p.slots[t];
  const bool keep = DEST == kRows || (slot >= 0 && slot / kBlock < p.num_blocks);
  if (threadIdx.x < p.rot / 2) {
    const uint64_t phase = (uint64_t)p.positions[t] * p.turns[threadIdx.x];
    float sn, cs;
    sincospif(__ll2float_rn((long long)phase) * 0x1p-63f, &sn, &cs);
    s_cos[threadIdx.x] = cs * p.magnitude;
    s_sin[threadIdx.x] = sn * p.magnitude;
  }
  __syncthreads();

#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int i = threadIdx.x + u * kThreads;
    if (i >= items) break;
    const int hh = h0 + i / items_row, ci = i % items_row;
    const bool value = hh >= p.Hq + p.Hkv;
    const Chunks c = chunks<VEC>(p, ci, value);
    if (c.turn) {
      float x[2 * VEC];
      unpack_vec<T>(lo[u], x);
      unpack_vec<T>(hi[u], x + VEC);
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        const float cs = s_cos[ci * VEC + e], sn = s_sin[ci * VEC + e];
        if (p.interleaved) {
          const float a = x[2 * e], b = x[2 * e + 1];
          x[2 * e] = a * cs - b * sn;
          x[2 * e + 1] = b * cs + a * sn;
        } else {
          const float a = x[e], b = x[VEC + e];
          x[e] = a * cs - b * sn;
          x[VEC + e] = b * cs + a * sn;
        }
      }
      lo[u] = pack_vec<T>(x);
      hi[u] = pack_vec<T>(x + VEC);
    }
    uint4 *dst;
    if (hh < p.Hq) {
      if (!c.turn && p.q_out == p.q) continue;  // in place: these stay
      dst = reinterpret_cast<uint4 *>(static_cast<uint8_t *>(p.q_out) +
                                      (size_t)(t * p.ld_q_out + (int64_t)hh * p.D) * T::kBytes);
    } else {
      const int h = value ? hh - p.Hq - p.Hkv : hh - p.Hq;
      if constexpr (DEST == kRows) {
        if (!c.turn && p.k_out == p.k) continue;
        dst = reinterpret_cast<uint4 *>(static_cast<uint8_t *>(p.k_out) +
                                        (size_t)(t * p.ld_k_out + (int64_t)h * p.D) * T::kBytes);
      } else if constexpr (DEST == kCache) {
        if (!keep) continue;
        dst = reinterpret_cast<uint4 *>(
            static_cast<uint8_t *>(value ? p.v_cache : p.k_cache) +
            ((size_t)(slot / kBlock * p.Hkv + h) * kBlock + slot % kBlock) * p.D * T::kBytes);
      } else {
        dst = reinterpret_cast<uint4 *>(s_rows + (size_t)(hh - max(h0, p.Hq)) * p.D * T::kBytes);
      }
    }
    dst[c.lo] = lo[u];
    dst[c.hi] = hi[u];
  }

  if constexpr (DEST == kCache4) {
    const int first = max(h0, p.Hq), rows = h0 + hn - first;  // this part's K and V rows
    if (rows <= 0 || !keep) return;                          // (the whole CTA alike)
    __syncthreads();
    const int G = p.D / 16;
    for (int i = threadIdx.x; i < rows * G; i += kThreads) {
      const int hh = first + i / G, g = i % G;
      const bool value = hh >= p.Hq + p.Hkv;
      const int h = value ? hh - p.Hq - p.Hkv : hh - p.Hq;
      const Kv4Group x = kv4_quantise_shared<Type>(s_rows, (size_t)(i / G) * p.D + 16 * g, value ? p.v_unit : p.k_unit);
      uint8_t *tile = p.kv4 + (size_t)(slot / kBlock * p.Hkv + h) * (18 * p.D);
      const int tok = (int)(slot % kBlock);
      if (p.D == 128)
        value ? kv4_store_v1<128>(tile, tok, g, x) : kv4_store_k<128>(tile, tok, g, x);
      else
        value ? kv4_store_v1<64>(tile, tok, g, x) : kv4_store_k<64>(tile, tok, g, x);
    }
  }
}

template <class T, int DEST>
cudaError_t launch(const RopeParams &p, cudaStream_t stream) {
  constexpr int VEC = RopeVec<T>::VEC;
  const int heads = p.Hq + (DEST == kRows ? 1 : 2) * p.Hkv;
  const int items_row = p.D / (2 * VEC);
  // few tokens: one item a thread, so that a step's rows are spread over as many CTAs as it
  // has; many: a token's rows in one CTA where five items a thread hold them
  const bool wide = p.T > 256;
  constexpr int kWide = 5;  // (kCache4: at most 20 KiB of rows)
  const int cap = kThreads * (wide ? kWide : 1) / items_row;  // heads a CTA holds
  const int parts = (heads + cap - 1) / cap, per = (heads + parts - 1) / parts;
  if ((double)p.T * parts > 2147483000.0) return cudaErrorNotSupported;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(p.T * parts));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = DEST == kCache4 ? (size_t)per * p.D * T::kBytes : 0;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = stream != nullptr ? 1 : 0;
  if (wide) return cudaLaunchKernelEx(&cfg, rope_kernel<T, DEST, kWide>, p, parts, per);
  return cudaLaunchKernelEx(&cfg, rope_kernel<T, DEST, 1>, p, parts, per);
}

template <class T>
cudaError_t launch_type(const RopeParams &p, cudaStream_t stream) {
  if (p.kv4) return launch<T, kCache4>(p, stream);
  if (p.k_cache) return launch<T, kCache>(p, stream);
  return launch<T, kRows>(p, stream);
}

}  // namespace

cudaError_t launch_rope(const RopeParams &p, int dtype, cudaStream_t stream) {
  if (dtype == PKV_F32) return launch_type<F32>(p, stream);
  if (dtype == PKV_F16) return launch_type<F16>(p, stream);
  return launch_type<BF16>(p, stream);
}

}  // namespace pkv
