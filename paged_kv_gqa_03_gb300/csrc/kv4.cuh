// kv4.cuh — the 4-bit cache's page format.
//
// 16 neighbouring elements of a row share a scale: with y = x / unit (fp32),
//   s = e4m3_rne(max|y| / 6), saturating at 448;  code = e2m1_rne(y / s), saturating at +-6;
//   value = code * s * unit        (E2M1: 0, 0.5, 1, 1.5, 2, 3, 4, 6 and their negatives)
// with the divisions in fp32.  Comparing fl(y / s) with the borders between two levels decides as
// the real quotient does: a border times s has 7 significant bits, so a y next to it is off by more
// than the quotient's rounding.  s = 0 (max|y| below 6 * 2^-10): every code 0.  A group with an
// element that is not finite has s = NaN: all its values read as NaN (E2M1 has no NaN of its own).
//
// A (block, kv head) tile is 18 D bytes, one contiguous run that one bulk copy fetches:
//   K codes [16 tokens][D / 2], the even element of a pair in the byte's lower half;
//   V codes [8 token pairs][D bytes]: byte d holds element d of both tokens, the even one in
//     the lower half: that is how the decode kernel's MMA operand pairs them.  Chunks c of 16 bytes (D = 128;
//     8 at D = 64) stand at c ^ 2 (u & 3) (D = 64: c ^ 4 (u / 2 & 1)) of pair u: the kernel's lanes then read
//     all of V without bank conflicts;
//   K scales [16 tokens][D / 16];
//   V scales [8 token pairs][D / 16][2 tokens]: the pair's two scales are one 16-bit load.
#pragma once

#include <cuda_fp4.h>

#include "common.cuh"

namespace pkv {

template <int D>
struct Kv4Tile {
  static constexpr int kGroups = D / 16;  // of a row
  static constexpr int kVCodes = 8 * D, kKScales = 16 * D, kVScales = 17 * D, kBytes = 18 * D;
  static __device__ __forceinline__ int k_code(int tok, int g) { return tok * (D / 2) + 8 * g; }
  static __device__ __forceinline__ int k_scale(int tok, int g) { return kKScales + tok * kGroups + g; }
  // 16 bytes: elements 16 g .. of the token pair u (D = 64: two chunks, which stay neighbours)
  static __device__ __forceinline__ int v_code(int u, int g) {
    if constexpr (D == 128)
      return kVCodes + u * 128 + ((g ^ (2 * (u & 3))) << 4);
    else
      return kVCodes + u * 64 + (((2 * g) ^ (4 * ((u >> 1) & 1))) << 3);
  }
  static __device__ __forceinline__ int v_scale(int tok, int g) {
    return kVScales + (tok >> 1) * (2 * kGroups) + 2 * g + (tok & 1);
  }
};

// 16 elements as the format holds them.
struct Kv4Group {
  uint2 codes;    // element i: bits 4 i .. 4 i + 3
  uint8_t scale;  // E4M3
};

__device__ __forceinline__ float e4m3_value(uint8_t s) {
  return __half2float(__half(__nv_cvt_fp8_to_halfraw(s, __NV_E4M3)));
}

// The codes of eight scaled elements, two a byte, the first of a pair in the lower half.
__device__ __forceinline__ uint32_t e2m1x8(const float *q) {
  uint32_t w;
  asm("{\n .reg .b8 a, b, c, d;\n"
      " cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n"
      " cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n"
      " cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n"
      " cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n"
      " mov.b32 %0, {a, b, c, d};\n}\n"
      : "=r"(w)
      : "f"(q[0]), "f"(q[1]), "f"(q[2]), "f"(q[3]), "f"(q[4]), "f"(q[5]), "f"(q[6]), "f"(q[7]));
  return w;
}
__device__ __forceinline__ uint2 e2m1_codes(const float (&q)[16]) { return make_uint2(e2m1x8(q), e2m1x8(q + 8)); }
// Packed |a| and the larger of each half, NaN if either is.
__device__ __forceinline__ uint32_t max_abs2(F16, uint32_t a, uint32_t b) {
  const uint32_t x = b & 0x7fff7fffu;
  const __half2 r = __hmax2_nan(*reinterpret_cast<const __half2 *>(&a), *reinterpret_cast<const __half2 *>(&x));
  return *reinterpret_cast<const uint32_t *>(&r);
}
__device__ __forceinline__ uint32_t max_abs2(BF16, uint32_t a, uint32_t b) {
  const uint32_t x = b & 0x7fff7fffu;
  const __nv_bfloat162 r =
      __hmax2_nan(*reinterpret_cast<const __nv_bfloat162 *>(&a), *reinterpret_cast<const __nv_bfloat162 *>(&x));
  return *reinterpret_cast<const uint32_t *>(&r);
}
__device__ __forceinline__ uint8_t e4m3_scale(float most) {
  return __nv_cvt_float_to_fp8(__fdiv_rn(most, 6.f), __NV_SATFINITE, __NV_E4M3);
}

__device__ __forceinline__ Kv4Group kv4_quantise(float (&y)[16], float unit) {
  float most = 0.f;
  bool finite = true;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    if (unit != 1.f) y[i] = __fdiv_rn(y[i], unit);
    finite &= fabsf(y[i]) < INFINITY;
    most = fmaxf(most, fabsf(y[i]));
  }
  Kv4Group r;
  r.codes = make_uint2(0, 0);
  r.scale = 0x7f;
  if (!finite) return r;
  r.scale = e4m3_scale(most);
  const float s = r.scale ? e4m3_value(r.scale) : INFINITY;
#pragma unroll
  for (int i = 0; i < 16; ++i) y[i] = __fdiv_rn(y[i], s);
  r.codes = e2m1_codes(y);
  return r;
}

// The same of 16-bit elements with unit = 1, without divisions (4096 pages packed and expanded: 186 us with them, 134 without).  An element y has
// at most 11 significant bits and a border m s between two codes at most 7, so that y / s either is m or
// is off by 2^-11 m or more, and m >= 1/4: y / s rounded to a multiple of 2^-14 falls on the same side of every border, or
// on it.  fmaf(y, r, 768) does that rounding (768's unit in the last place is 2^-14; r = 1 / s to 2^-23, |y r| <= 6.4;
// quotients beyond, where the scale saturates, saturate too).
template <class T>
__device__ __forceinline__ Kv4Group kv4_quantise16(const uint32_t (&w)[8]) {
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) top = max_abs2(T{}, top, w[i]);
  top = max(top & 0x7fffu, (top >> 16) & 0x7fffu);  // the largest magnitude's bits (NaN above all)
  Kv4Group r;
  r.codes = make_uint2(0, 0);
  r.scale = 0x7f;
  if (top >= (T::kCode == PKV_BF16 ? 0x7f80u : 0x7c00u)) return r;  // an element is not finite
  r.scale = e4m3_scale(unpack2(T{}, top).x);
  const float inv = r.scale ? __frcp_rn(e4m3_value(r.scale)) : 0.f;
  float q[16];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float2 v = unpack2(T{}, w[i]);
    q[2 * i] = fmaf(v.x, inv, 768.f) - 768.f;
    q[2 * i + 1] = fmaf(v.y, inv, 768.f) - 768.f;
  }
  r.codes = e2m1_codes(q);
  return r;
}

// The eight codes of w -> f16x2 of elements (0, 1), (2, 3), (4, 5), (6, 7).  One instruction each,
// which takes its byte of w itself (the conversion intrinsic on w >> 8 i costs two more).
__device__ __forceinline__ void e2m1x8_to_f16(uint32_t w, uint32_t (&h)[4]) {
  asm("{\n .reg .b8 a, b, c, d;\n"
      " mov.b32 {a, b, c, d}, %4;\n"
      " cvt.rn.f16x2.e2m1x2 %0, a;\n"
      " cvt.rn.f16x2.e2m1x2 %1, b;\n"
      " cvt.rn.f16x2.e2m1x2 %2, c;\n"
      " cvt.rn.f16x2.e2m1x2 %3, d;\n}\n"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(w));
}

__device__ __forceinline__ void kv4_values(const Kv4Group &g, float unit, float (&y)[16]) {
  const float s = e4m3_value(g.scale);
  uint32_t h[2][4];
  e2m1x8_to_f16(g.codes.x, h[0]);
  e2m1x8_to_f16(g.codes.y, h[1]);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float2 v = unpack2(F16{}, h[i / 4][i % 4]);
    y[2 * i] = v.x * s * unit;  // (code * s is exact)
    y[2 * i + 1] = v.y * s * unit;
  }
}

// Codes of 16 elements of two tokens <-> bytes that hold an element of both.
__device__ __forceinline__ uint32_t spread_nibbles(uint32_t w) {  // 4 nibbles (low half) -> the low halves of 4 bytes
  w = (w | (w << 8)) & 0x00ff00ffu;
  return (w | (w << 4)) & 0x0f0f0f0fu;
}
__device__ __forceinline__ uint32_t gather_nibbles(uint32_t w) {  // and back
  w &= 0x0f0f0f0fu;
  w = (w | (w >> 4)) & 0x00ff00ffu;
  return (w | (w >> 8)) & 0xffffu;
}
__device__ __forceinline__ uint4 spread16(uint2 c) {
  return make_uint4(spread_nibbles(c.x & 0xffffu), spread_nibbles(c.x >> 16), spread_nibbles(c.y & 0xffffu),
                    spread_nibbles(c.y >> 16));
}

template <int D>
__device__ __forceinline__ void kv4_store_k(uint8_t *tile, int tok, int g, const Kv4Group &x) {
  using Tile = Kv4Tile<D>;
  *reinterpret_cast<uint2 *>(tile + Tile::k_code(tok, g)) = x.codes;
  tile[Tile::k_scale(tok, g)] = x.scale;
}
// Both tokens of pair u.
template <int D>
__device__ __forceinline__ void kv4_store_v2(uint8_t *tile, int u, int g, const Kv4Group &a, const Kv4Group &b) {
  using Tile = Kv4Tile<D>;
  const uint4 x = spread16(a.codes), y = spread16(b.codes);
  *reinterpret_cast<uint4 *>(tile + Tile::v_code(u, g)) = make_uint4(x.x | y.x << 4, x.y | y.y << 4, x.z | y.z << 4, x.w | y.w << 4);
  *reinterpret_cast<uint16_t *>(tile + Tile::v_scale(2 * u, g)) = (uint16_t)(a.scale | b.scale << 8);
}
// One token, whose neighbour's nibbles another thread may be writing: the difference to what stands there
// in this token's own nibbles, which no one else writes, goes in by an exclusive or.
template <int D>
__device__ __forceinline__ void kv4_store_v1(uint8_t *tile, int tok, int g, const Kv4Group &a) {
  using Tile = Kv4Tile<D>;
  const int sh = 4 * (tok & 1);
  const uint4 x = spread16(a.codes);
  uint32_t *c = reinterpret_cast<uint32_t *>(tile + Tile::v_code(tok >> 1, g));
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t old = *reinterpret_cast<volatile uint32_t *>(c + i);
    atomicXor(c + i, (old ^ (w[i] << sh)) & (0x0f0f0f0fu << sh));
  }
  tile[Tile::v_scale(tok, g)] = a.scale;
}

template <int D>
__device__ __forceinline__ Kv4Group kv4_load_k(const uint8_t *tile, int tok, int g) {
  using Tile = Kv4Tile<D>;
  Kv4Group x;
  x.codes = *reinterpret_cast<const uint2 *>(tile + Tile::k_code(tok, g));
  x.scale = tile[Tile::k_scale(tok, g)];
  return x;
}
template <int D>
__device__ __forceinline__ void kv4_load_v2(const uint8_t *tile, int u, int g, Kv4Group &a, Kv4Group &b) {
  using Tile = Kv4Tile<D>;
  const uint4 c = *reinterpret_cast<const uint4 *>(tile + Tile::v_code(u, g));
  const uint16_t sc = *reinterpret_cast<const uint16_t *>(tile + Tile::v_scale(2 * u, g));
  a.codes = make_uint2(gather_nibbles(c.x) | gather_nibbles(c.y) << 16, gather_nibbles(c.z) | gather_nibbles(c.w) << 16);
  b.codes = make_uint2(gather_nibbles(c.x >> 4) | gather_nibbles(c.y >> 4) << 16,
                       gather_nibbles(c.z >> 4) | gather_nibbles(c.w >> 4) << 16);
  a.scale = (uint8_t)(sc & 0xff);
  b.scale = (uint8_t)(sc >> 8);
}

// 16 consecutive elements of a 16-bit type (16-byte aligned; one access where they are 32-byte aligned).
struct Half16 {
  uint32_t w[8];
};
__device__ __forceinline__ Half16 load_half16(const void *p) {
  Half16 r;
  if ((reinterpret_cast<uintptr_t>(p) & 31u) == 0) {
    asm volatile("ld.global.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(r.w[0]), "=r"(r.w[1]), "=r"(r.w[2]), "=r"(r.w[3]), "=r"(r.w[4]), "=r"(r.w[5]), "=r"(r.w[6]),
                   "=r"(r.w[7])
                 : "l"(__cvta_generic_to_global(p)));
  } else {
    const uint4 a = reinterpret_cast<const uint4 *>(p)[0], b = reinterpret_cast<const uint4 *>(p)[1];
    r = Half16{{a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w}};
  }
  return r;
}
__device__ __forceinline__ void store_half16(void *p, const Half16 &r) {
  if ((reinterpret_cast<uintptr_t>(p) & 31u) == 0) {
    asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(__cvta_generic_to_global(p)), "r"(r.w[0]),
                 "r"(r.w[1]), "r"(r.w[2]), "r"(r.w[3]), "r"(r.w[4]), "r"(r.w[5]), "r"(r.w[6]), "r"(r.w[7])
                 : "memory");
  } else {
    reinterpret_cast<uint4 *>(p)[0] = make_uint4(r.w[0], r.w[1], r.w[2], r.w[3]);
    reinterpret_cast<uint4 *>(p)[1] = make_uint4(r.w[4], r.w[5], r.w[6], r.w[7]);
  }
}

// 16 consecutive floats (16-byte aligned).
__device__ __forceinline__ void load16(const void *p, size_t i, float (&y)[16]) {
  const float4 *f = reinterpret_cast<const float4 *>(static_cast<const float *>(p) + i);
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float4 v = f[j];
    y[4 * j] = v.x; y[4 * j + 1] = v.y; y[4 * j + 2] = v.z; y[4 * j + 3] = v.w;
  }
}

__device__ __forceinline__ uint32_t pack2(F16, float lo, float hi) { return pack_f16x2(lo, hi); }
__device__ __forceinline__ uint32_t pack2(BF16, float lo, float hi) { return pack_bf16x2(lo, hi); }

__device__ __forceinline__ void store16(void *p, size_t i, const float (&y)[16]) {
  float4 *f = reinterpret_cast<float4 *>(static_cast<float *>(p) + i);
#pragma unroll
  for (int j = 0; j < 4; ++j) f[j] = make_float4(y[4 * j], y[4 * j + 1], y[4 * j + 2], y[4 * j + 3]);
}

// 16 elements of a 16-bit type as the format holds them: the one way for whole pages, appended rows and rotated rows, whose
// bytes are the same.  (Of an element that comes to 0 the sign depends on the unit: the divisions keep it.)
template <class T>
__device__ __forceinline__ Kv4Group kv4_quantise_half(const uint32_t (&w)[8], float unit) {
  if (unit == 1.f) return kv4_quantise16<T>(w);
  float y[16];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float2 v = unpack2(T{}, w[j]);
    y[2 * j] = v.x; y[2 * j + 1] = v.y;
  }
  return kv4_quantise(y, unit);
}
// 16 elements at p[i ..] of global memory.
template <class T>
__device__ __forceinline__ Kv4Group kv4_quantise_at(const void *p, size_t i, float unit) {
  if constexpr (T::kBytes == 2) {
    return kv4_quantise_half<T>(load_half16(static_cast<const uint16_t *>(p) + i).w, unit);
  } else {
    float y[16];
    load16(p, i, y);
    return kv4_quantise(y, unit);
  }
}
// The same of shared memory.
template <class T>
__device__ __forceinline__ Kv4Group kv4_quantise_shared(const void *p, size_t i, float unit) {
  if constexpr (T::kBytes == 2) {
    const uint4 *u = reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(p) + i);
    const uint4 a = u[0], b = u[1];
    return kv4_quantise_half<T>({a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w}, unit);
  } else {
    float y[16];
    load16(p, i, y);
    return kv4_quantise(y, unit);
  }
}
template <class T>
__device__ __forceinline__ void kv4_values_to(const Kv4Group &g, float unit, void *p, size_t i) {
  float y[16];
  kv4_values(g, unit, y);
  if constexpr (T::kBytes == 2) {
    Half16 h;
#pragma unroll
    for (int j = 0; j < 8; ++j) h.w[j] = pack2(T{}, y[2 * j], y[2 * j + 1]);
    store_half16(static_cast<uint16_t *>(p) + i, h);
  } else {
    store16(p, i, y);
  }
}

}  // namespace pkv
