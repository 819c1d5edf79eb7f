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
//   V codes [8 token pairs][128 or 64 bytes]: 16 bytes (D = 128: 16 elements of both tokens of
//     the pair, D = 64: 8 bytes, 8 elements of both) at chunk c ^ 2 (u & 3) (D = 64: c ^ 4 (u / 2 & 1))
//     of pair u: the decode kernel's lanes then read all of V without bank conflicts;
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
  // D = 128: 8 bytes.  D = 64: 4 bytes here and 4 bytes 8 further.
  static __device__ __forceinline__ int v_code(int tok, int g) {
    const int u = tok >> 1;
    if constexpr (D == 128)
      return kVCodes + u * 128 + ((g ^ (2 * (u & 3))) << 4) + (tok & 1) * 8;
    else
      return kVCodes + u * 64 + (((2 * g) ^ (4 * ((u >> 1) & 1))) << 3) + (tok & 1) * 4;
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
  r.scale = __nv_cvt_float_to_fp8(__fdiv_rn(most, 6.f), __NV_SATFINITE, __NV_E4M3);
  const float s = r.scale ? e4m3_value(r.scale) : INFINITY;
  uint32_t w[2] = {0, 0};
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float2 q = make_float2(__fdiv_rn(y[2 * i], s), __fdiv_rn(y[2 * i + 1], s));
    w[i / 4] |= (uint32_t)__nv_cvt_float2_to_fp4x2(q, __NV_E2M1, cudaRoundNearest) << (8 * (i % 4));
  }
  r.codes = make_uint2(w[0], w[1]);
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

template <int D>
__device__ __forceinline__ void kv4_store(uint8_t *tile, bool v, int tok, int g, const Kv4Group &x) {
  using Tile = Kv4Tile<D>;
  if (!v) {
    *reinterpret_cast<uint2 *>(tile + Tile::k_code(tok, g)) = x.codes;
    tile[Tile::k_scale(tok, g)] = x.scale;
  } else {
    uint8_t *c = tile + Tile::v_code(tok, g);
    if constexpr (D == 128) {
      *reinterpret_cast<uint2 *>(c) = x.codes;
    } else {
      *reinterpret_cast<uint32_t *>(c) = x.codes.x;
      *reinterpret_cast<uint32_t *>(c + 8) = x.codes.y;
    }
    tile[Tile::v_scale(tok, g)] = x.scale;
  }
}

template <int D>
__device__ __forceinline__ Kv4Group kv4_load(const uint8_t *tile, bool v, int tok, int g) {
  using Tile = Kv4Tile<D>;
  Kv4Group x;
  if (!v) {
    x.codes = *reinterpret_cast<const uint2 *>(tile + Tile::k_code(tok, g));
    x.scale = tile[Tile::k_scale(tok, g)];
  } else {
    const uint8_t *c = tile + Tile::v_code(tok, g);
    if constexpr (D == 128) {
      x.codes = *reinterpret_cast<const uint2 *>(c);
    } else {
      x.codes.x = *reinterpret_cast<const uint32_t *>(c);
      x.codes.y = *reinterpret_cast<const uint32_t *>(c + 8);
    }
    x.scale = tile[Tile::v_scale(tok, g)];
  }
  return x;
}

// 16 consecutive elements (16-byte aligned) <-> floats.
template <class T>
__device__ __forceinline__ void load16(const void *p, size_t i, float (&y)[16]) {
  if constexpr (T::kBytes == 4) {
    const float4 *f = reinterpret_cast<const float4 *>(static_cast<const float *>(p) + i);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float4 v = f[j];
      y[4 * j] = v.x; y[4 * j + 1] = v.y; y[4 * j + 2] = v.z; y[4 * j + 3] = v.w;
    }
  } else {
    const uint4 *u = reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(p) + i);
    const uint4 a = u[0], b = u[1];
    const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float2 v = unpack2(T{}, w[j]);
      y[2 * j] = v.x; y[2 * j + 1] = v.y;
    }
  }
}

__device__ __forceinline__ uint32_t pack2(F16, float lo, float hi) { return pack_f16x2(lo, hi); }
__device__ __forceinline__ uint32_t pack2(BF16, float lo, float hi) { return pack_bf16x2(lo, hi); }

template <class T>
__device__ __forceinline__ void store16(void *p, size_t i, const float (&y)[16]) {
  if constexpr (T::kBytes == 4) {
    float4 *f = reinterpret_cast<float4 *>(static_cast<float *>(p) + i);
#pragma unroll
    for (int j = 0; j < 4; ++j) f[j] = make_float4(y[4 * j], y[4 * j + 1], y[4 * j + 2], y[4 * j + 3]);
  } else {
    uint4 *u = reinterpret_cast<uint4 *>(static_cast<uint16_t *>(p) + i);
#pragma unroll
    for (int j = 0; j < 2; ++j)
      u[j] = make_uint4(pack2(T{}, y[8 * j], y[8 * j + 1]), pack2(T{}, y[8 * j + 2], y[8 * j + 3]),
                        pack2(T{}, y[8 * j + 4], y[8 * j + 5]), pack2(T{}, y[8 * j + 6], y[8 * j + 7]));
  }
}

}  // namespace pkv
