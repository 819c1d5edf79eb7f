// kv4_pages.cu — rows into and out of the 4-bit cache's pages (kv4.cuh): the
// append of new tokens, whole pages packed from 16 bits and expanded back, and
// the copy-on-write copy.
//
// A thread does 16 elements of K of two neighbouring tokens, or of V, whose codes share
// bytes: a scale needs nothing of another thread, a warp's loads and stores of codes are whole lines.  A new token
// whose neighbour is not beside it in the call is stored by an exclusive or into its own
// nibbles (kv4_store_v1).  A token and head read or write 4 D bytes in 16 bits and 18 D / 16 in 4.  4096 pages of 8
// heads of 128 in bf16 (344 MB): expanded in 55 us (6.2 TB/s: HBM), packed in 60 (5.7 TB/s, three issue slots of four
// taken: the conversions).  16384 tokens (86 MB) appended in 21 us: 4.1 TB/s, 0.6 of a copy's rate, DRAM busy for 39 %;
// issue slots again (0.73 a clock) and waits for the slots and rows, one load of a row in flight a thread, half of V's
// threads leaving at once.  Divisions (fp32 rows, units other than 1) cost more: packed in 111 us (fp32, 612 MB) and
// 136 (bf16, unit 2^-4), appended in 38 and 44.
#include "kv4.cuh"
#include "kv4.h"

namespace pkv {

constexpr int kThreads = kKv4PageThreads;
// Resident CTAs of the kernels that convert: whole occupancy (32 registers) is worth a few spilled registers, but for
// fp32 rows (bf16, 8 heads of 128 and of 64, with a bound of 8 and with this one: 4096 pages packed 69.9 -> 60.1 us and
// 37.8 -> 33.4, expanded 58.8 -> 55.1 and 31.7 -> 29.5; 16384 tokens appended 25.8 -> 21.1 and 14.7 -> 12.3).
template <class T>
constexpr int kResident = T::kBytes == 4 ? 8 : 16;

static cudaLaunchConfig_t config(int64_t threads, cudaLaunchAttribute *attr, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((threads + kThreads - 1) / kThreads));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  attr->id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr->val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = stream != nullptr ? 1 : 0;  // early launch on explicit streams only
  return cfg;
}

// Thread -> (token, K or V, head, group), the group fastest.
template <class T, int D>
__global__ void __launch_bounds__(kThreads, kResident<T>)
    kv4_append_kernel(const void *__restrict__ k_new, int64_t ld_k, const void *__restrict__ v_new, int64_t ld_v,
                      uint8_t *cache, const int64_t *__restrict__ slots, int T_, int Hkv, int64_t num_blocks,
                      float k_unit, float v_unit) {
  grid_dep_launch();  // the next kernel of the chain may come up; it waits for this one
  grid_dep_wait();
  constexpr int G = D / 16;
  const int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  const int g = (int)(i % G);
  const int64_t row = i / G;
  const int per = 2 * Hkv;
  const int64_t t = row / per;
  if (t >= T_) return;
  const int hv = (int)(row - t * per), h = hv < Hkv ? hv : hv - Hkv;
  const bool v = hv >= Hkv;
  const int64_t slot = slots[t];
  if (slot < 0 || slot / kBlock >= num_blocks) return;
  const int tok = (int)(slot % kBlock);
  uint8_t *tile = cache + (size_t)(slot / kBlock * Hkv + h) * Kv4Tile<D>::kBytes;
  const size_t at = (size_t)h * D + 16 * g;
  if (!v) {
    kv4_store_k<D>(tile, tok, g, kv4_quantise_at<T>(k_new, (size_t)(t * ld_k) + at, k_unit));
    return;
  }
  // a pair that stands together in the call: its even token's thread stores both
  if ((tok & 1) && t > 0 && slots[t - 1] == slot - 1) return;
  const bool two = !(tok & 1) && t + 1 < T_ && slots[t + 1] == slot + 1;
  const Kv4Group a = kv4_quantise_at<T>(v_new, (size_t)(t * ld_v) + at, v_unit);
  if (two) {
    kv4_store_v2<D>(tile, tok >> 1, g, a, kv4_quantise_at<T>(v_new, (size_t)((t + 1) * ld_v) + at, v_unit));
  } else {
    kv4_store_v1<D>(tile, tok, g, a);
  }
}

// Thread -> (pair, head, K or V, tokens 2 u and 2 u + 1, group), the group fastest.
struct PageThread {
  int64_t pair;
  int h, u, g;
  bool v;
};
template <int D>
__device__ __forceinline__ PageThread page_thread(int Hkv) {
  constexpr int G = D / 16, kTile = kBlock * G;
  const int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  const int in = (int)(i % kTile);
  const int64_t tile = i / kTile;
  PageThread p;
  p.g = in % G;
  p.u = in / G % (kBlock / 2);
  p.v = in >= kTile / 2;
  p.pair = tile / Hkv;
  p.h = (int)(tile - p.pair * Hkv);
  return p;
}

template <class T, int D>
__global__ void __launch_bounds__(kThreads, kResident<T>)
    kv4_pack_kernel(uint8_t *cache, int64_t num_blocks, const void *__restrict__ k, const void *__restrict__ vv,
                    int64_t num_src, const int32_t *__restrict__ pairs, int n, int Hkv, float k_unit, float v_unit) {
  grid_dep_launch();  // the next kernel of the chain may come up; it waits for this one
  grid_dep_wait();
  const PageThread p = page_thread<D>(Hkv);
  if (p.pair >= n) return;
  const int src = pairs[2 * p.pair], dst = pairs[2 * p.pair + 1];
  if (src < 0 || src >= num_src || dst < 0 || dst >= num_blocks) return;
  const size_t at = (((size_t)src * Hkv + p.h) * kBlock + 2 * p.u) * D + 16 * p.g;
  const void *rows = p.v ? vv : k;
  const float unit = p.v ? v_unit : k_unit;
  const Kv4Group a = kv4_quantise_at<T>(rows, at, unit), b = kv4_quantise_at<T>(rows, at + D, unit);
  uint8_t *tile = cache + ((size_t)dst * Hkv + p.h) * Kv4Tile<D>::kBytes;
  if (p.v) {
    kv4_store_v2<D>(tile, p.u, p.g, a, b);
  } else {
    kv4_store_k<D>(tile, 2 * p.u, p.g, a);
    kv4_store_k<D>(tile, 2 * p.u + 1, p.g, b);
  }
}

template <class T, int D>
__global__ void __launch_bounds__(kThreads, kResident<T>)
    kv4_expand_kernel(void *k, void *vv, int64_t num_dst, const uint8_t *__restrict__ cache, int64_t num_blocks,
                      const int32_t *__restrict__ pairs, int n, int Hkv, float k_unit, float v_unit) {
  grid_dep_launch();  // the next kernel of the chain may come up; it waits for this one
  grid_dep_wait();
  const PageThread p = page_thread<D>(Hkv);
  if (p.pair >= n) return;
  const int src = pairs[2 * p.pair], dst = pairs[2 * p.pair + 1];
  if (src < 0 || src >= num_blocks || dst < 0 || dst >= num_dst) return;
  const uint8_t *tile = cache + ((size_t)src * Hkv + p.h) * Kv4Tile<D>::kBytes;
  Kv4Group a, b;
  if (p.v) {
    kv4_load_v2<D>(tile, p.u, p.g, a, b);
  } else {
    a = kv4_load_k<D>(tile, 2 * p.u, p.g);
    b = kv4_load_k<D>(tile, 2 * p.u + 1, p.g);
  }
  const size_t at = (((size_t)dst * Hkv + p.h) * kBlock + 2 * p.u) * D + 16 * p.g;
  void *rows = p.v ? vv : k;
  const float unit = p.v ? v_unit : k_unit;
  kv4_values_to<T>(a, unit, rows, at);
  kv4_values_to<T>(b, unit, rows, at + D);
}

// A CTA a pair, four loads in flight a thread (one after another: a pair of 8 heads 1.6 -> 2.6 us, 256 pairs 3.1 -> 3.6).
__global__ void __launch_bounds__(kThreads)
    kv4_copy_kernel(uint8_t *cache, const int32_t *__restrict__ pairs, size_t block_bytes, int64_t num_blocks) {
  grid_dep_launch();  // the next kernel of the chain may come up; it waits for this one
  grid_dep_wait();
  const int src = pairs[2 * blockIdx.x], dst = pairs[2 * blockIdx.x + 1];
  if (src < 0 || dst < 0 || src >= num_blocks || dst >= num_blocks || src == dst) return;
  const uint4 *s = reinterpret_cast<const uint4 *>(cache + (size_t)src * block_bytes);
  uint4 *d = reinterpret_cast<uint4 *>(cache + (size_t)dst * block_bytes);
  const size_t n = block_bytes / 16;
  for (size_t i = threadIdx.x; i < n; i += 4 * kThreads) {
    uint4 x[4];
#pragma unroll
    for (int t = 0; t < 4; ++t)
      if (i + t * kThreads < n) x[t] = s[i + t * kThreads];
#pragma unroll
    for (int t = 0; t < 4; ++t)
      if (i + t * kThreads < n) d[i + t * kThreads] = x[t];
  }
}

// f(T{}, integral_constant<int, D>) of a (dtype, head dim).
template <class F>
static cudaError_t dispatch(int dtype, int D, F f) {
  if (dtype == PKV_F32) return D == 128 ? f(F32{}, Kv4Tile<128>{}) : f(F32{}, Kv4Tile<64>{});
  if (dtype == PKV_F16) return D == 128 ? f(F16{}, Kv4Tile<128>{}) : f(F16{}, Kv4Tile<64>{});
  return D == 128 ? f(BF16{}, Kv4Tile<128>{}) : f(BF16{}, Kv4Tile<64>{});
}

cudaError_t launch_kv4_append(const void *k_new, int64_t ld_k, const void *v_new, int64_t ld_v, int new_dtype,
                              uint8_t *cache, const int64_t *slots, int T, int Hkv, int D, int64_t num_blocks,
                              float k_unit, float v_unit, cudaStream_t stream) {
  return dispatch(new_dtype, D, [&](auto type, auto tile) {
    constexpr int DD = decltype(tile)::kGroups * 16;
    cudaLaunchAttribute attr[1];
    const cudaLaunchConfig_t cfg = config((int64_t)T * 2 * Hkv * (DD / 16), attr, stream);
    return cudaLaunchKernelEx(&cfg, kv4_append_kernel<decltype(type), DD>, k_new, ld_k, v_new, ld_v, cache, slots, T,
                              Hkv, num_blocks, k_unit, v_unit);
  });
}

cudaError_t launch_kv4_pack(uint8_t *cache, int64_t num_blocks, const void *k, const void *v, int dtype,
                            int64_t num_src, const int32_t *pairs, int n, int Hkv, int D, float k_unit, float v_unit,
                            cudaStream_t stream) {
  return dispatch(dtype, D, [&](auto type, auto tile) {
    constexpr int DD = decltype(tile)::kGroups * 16;
    cudaLaunchAttribute attr[1];
    const cudaLaunchConfig_t cfg = config((int64_t)n * Hkv * kBlock * (DD / 16), attr, stream);
    return cudaLaunchKernelEx(&cfg, kv4_pack_kernel<decltype(type), DD>, cache, num_blocks, k, v, num_src, pairs, n,
                              Hkv, k_unit, v_unit);
  });
}

cudaError_t launch_kv4_expand(void *k, void *v, int dtype, int64_t num_dst, const uint8_t *cache, int64_t num_blocks,
                              const int32_t *pairs, int n, int Hkv, int D, float k_unit, float v_unit,
                              cudaStream_t stream) {
  return dispatch(dtype, D, [&](auto type, auto tile) {
    constexpr int DD = decltype(tile)::kGroups * 16;
    cudaLaunchAttribute attr[1];
    const cudaLaunchConfig_t cfg = config((int64_t)n * Hkv * kBlock * (DD / 16), attr, stream);
    return cudaLaunchKernelEx(&cfg, kv4_expand_kernel<decltype(type), DD>, k, v, num_dst, cache, num_blocks, pairs, n,
                              Hkv, k_unit, v_unit);
  });
}

cudaError_t launch_kv4_copy(uint8_t *cache, const int32_t *pairs, int n, size_t block_bytes, int64_t num_blocks,
                            cudaStream_t stream) {
  cudaLaunchAttribute attr[1];
  const cudaLaunchConfig_t cfg = config((int64_t)n * kThreads, attr, stream);
  return cudaLaunchKernelEx(&cfg, kv4_copy_kernel, cache, pairs, block_bytes, num_blocks);
}

}  // namespace pkv
