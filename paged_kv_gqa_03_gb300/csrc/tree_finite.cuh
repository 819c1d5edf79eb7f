// tree_finite.cuh — V rows of a tree's cache that are not finite (a drafted branch whose
// values overflowed, say).  A matrix instruction multiplies a hidden row by a
// weight of 0, and 0 times infinity is NaN: one branch would spoil the others.
// So in the few tiles with positions that not every row sees — the tree's nodes,
// and the positions at the edge of a window — elements that are not finite are
// set to 0 in shared memory and their positions noted, and the rows that do see such a
// position get those elements added at the end, read again from the cache: a weight is
// positive, so an infinity stays one and a NaN or opposite infinities give NaN.
#pragma once

#include "common.cuh"

namespace pkv {

// The bits of a word of cache elements that belong to elements that are not finite.
template <class T>
__device__ __forceinline__ uint32_t nonfinite_bits(uint32_t w) {
  if constexpr (T::kBytes == 2) {  // the exponent's bits all ones: adding its lowest carries into the sign's place
    const uint32_t e = T::kCode == PKV_BF16 ? 0x7f807f80u : 0x7c007c00u, one = T::kCode == PKV_BF16 ? 0x00800080u : 0x04000400u;
    return ((((w & e) + one) >> 15) & 0x00010001u) * 0xffffu;
  } else {  // E4M3: NaN is all ones
    return ((((w & 0x7f7f7f7fu) + 0x01010101u) >> 7) & 0x01010101u) * 0xffu;
  }
}
// 0x8000 (16-bit) or 0x80 (E4M3) bits of a chunk's words joined, set where an element is not finite.
template <class T>
__device__ __forceinline__ uint32_t nonfinite_any(uint4 v) {
  if constexpr (T::kBytes == 2) {
    const uint32_t e = T::kCode == PKV_BF16 ? 0x7f807f80u : 0x7c007c00u, one = T::kCode == PKV_BF16 ? 0x00800080u : 0x04000400u;
    return (((v.x & e) + one) | ((v.y & e) + one) | ((v.z & e) + one) | ((v.w & e) + one)) & 0x80008000u;
  } else {
    const uint32_t e = 0x7f7f7f7fu, one = 0x01010101u;
    return (((v.x & e) + one) | ((v.y & e) + one) | ((v.z & e) + one) | ((v.w & e) + one)) & 0x80808080u;
  }
}
// Zeroes such elements of the 16-byte chunk at shared address a; whether there were any.
template <class T>
__device__ __forceinline__ bool clear_nonfinite(uint32_t a) {
  const uint4 v = lds128(a);
  const uint4 b = make_uint4(nonfinite_bits<T>(v.x), nonfinite_bits<T>(v.y), nonfinite_bits<T>(v.z), nonfinite_bits<T>(v.w));
  if ((b.x | b.y | b.z | b.w) == 0) return false;
  sts128(a, make_uint4(v.x & ~b.x, v.y & ~b.y, v.z & ~b.z, v.w & ~b.w));
  return true;
}
// Element i of a cache if it is not finite, else 0.
template <class T>
__device__ __forceinline__ float nonfinite_value(const void *cache, size_t i) {
  if constexpr (T::kBytes == 2) {
    const float x = load_scalar(T{}, cache, i);
    return fabsf(x) < INFINITY ? 0.f : x;
  } else {
    return (static_cast<const uint8_t *>(cache)[i] & 0x7f) == 0x7f ? __int_as_float(0x7fc00000) : 0.f;
  }
}

// What not every row of a sequence sees: cached positions [first, edge) (those
// before `first` no row sees) and the tree's, from `start` on.
struct TreePartial {
  int first, edge, start;
  __device__ __forceinline__ bool holds(int pos) const { return pos >= start || pos < edge; }
};
// Such positions with elements that are not finite, as bits: node `bit`, or position
// first + bit (a window's edge is at most 63 positions wide).
struct TreeSpoiled {
  uint64_t nodes, edge;
  __device__ __forceinline__ bool any() const { return (nodes | edge) != 0; }
  __device__ __forceinline__ void note(const TreePartial &t, int pos) {
    if (pos >= t.start)
      nodes |= 1ull << (pos - t.start);
    else if (pos >= t.first)
      edge |= 1ull << (pos - t.first);
  }
};

}  // namespace pkv
