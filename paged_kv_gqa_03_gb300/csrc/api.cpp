// api.cpp — the extern "C" boundary of libpagedkv.so: argument validation,
// kernel selection, TMA descriptor encoding, workspace layout and launches.
// Every check runs before the first launch, so a rejected call touches no
// memory.  No function here allocates device memory.
#include <cuda.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdlib>
#include <cstring>
#include <mutex>

#include "internal.h"
#include "kv4.h"
#include "pagedkv.h"
#include "mq_decode.h"
#include "prefill.h"
#include "tree.h"
#include "tree_tiles.h"

namespace pkv {

static thread_local int g_last_cuda_error = 0;

static int cuda_status(cudaError_t e) {
  if (e == cudaSuccess) return PKV_OK;
  g_last_cuda_error = static_cast<int>(e);
  return PKV_ECUDA;
}

void record_cuda_error(cudaError_t e) { g_last_cuda_error = static_cast<int>(e); }

static inline size_t align_up(size_t x, size_t a) { return (x + a - 1) / a * a; }

WsLayout ws_layout(int B, int P, int D, int GC) {
  WsLayout L;
  size_t o = 0;
  L.hdr = o;
  o = align_up(o + sizeof(WsHeader), 256);
  L.prefix = o;
  o = align_up(o + sizeof(int32_t) * (size_t)(B + 1), 256);
  L.starts = o;
  o = align_up(o + sizeof(int4) * (size_t)(P + 1), 256);
  L.part_o = o;
  o = align_up(o + sizeof(float) * (size_t)P * 2 * GC * D, 256);
  L.part_lse = o;
  o = align_up(o + sizeof(float) * (size_t)P * 2 * GC, 256);
  L.cta_flags = o;
  o = align_up(o + sizeof(int32_t) * (size_t)P, 256);
  L.total = o;
  return L;
}

Kv4WsLayout kv4_ws_layout(int B, int P, int D, int GC, int hg, int warps) {
  Kv4WsLayout L;
  size_t o = 0;
  L.hdr = o;
  o = align_up(o + sizeof(WsHeader), 256);
  L.prefix = o;
  o = align_up(o + sizeof(int32_t) * (size_t)(B + 1), 256);
  L.starts = o;
  o = align_up(o + sizeof(int4) * (size_t)(P + 1), 256);
  L.records = o;
  o = align_up(o + sizeof(int4) * (size_t)P, 256);
  L.part_o = o;  // [P][2][hg][GC][D]
  o = align_up(o + sizeof(float) * (size_t)P * 2 * hg * GC * D, 256);
  L.part_lse = o;  // [P][2][hg][GC] {largest raw score, sum of weights, the scores' factor}
  o = align_up(o + sizeof(float4) * (size_t)P * 2 * hg * GC, 256);
  L.first_o = o;
  o = align_up(o + sizeof(float) * (size_t)P * warps * GC * D, 256);
  L.total = o;
  return L;
}

// ---------------------------------------------------------------------------
// Kernel registry and per-device facts.
// ---------------------------------------------------------------------------
namespace {

constexpr int kMaxKernels = 64;
constexpr int kMaxDevices = 64;

struct Registry {
  DecodeKernel k[kMaxKernels];
  int n = 0;
  Kv4Kernel kv4[kKv4Kernels];
};

Registry &registry() {
  static Registry r;
  static std::once_flag once;
  std::call_once(once, [] {
    r.n += register_decode_bf16(r.k + r.n);
    r.n += register_decode_f16(r.k + r.n);
    r.n += register_decode_fp8(r.k + r.n);
    r.n += register_decode_f32(r.k + r.n);
    r.n += register_decode_tree(r.k + r.n);
    r.n += register_decode_tree_fp8(r.k + r.n);
    register_decode_kv4(r.kv4);
  });
  return r;
}

// Route overrides set by pkv_set_route (PKV_ROUTE_AUTO = the rule of shapes).
std::atomic<int> g_route[3];

// Limit of every bounded in-kernel wait (a wait that runs out sets
// PKV_FLAG_TIMEOUT instead of hanging).
constexpr uint64_t kWaitLimitNs = 4000000000ull;

// Pending failure-path test requests (pkv_test_stall_next), one per kernel
// family, consumed by the next call that launches that family: the wait
// limit of that call, or 0.
std::atomic<uint64_t> g_stall[2];

// Sets the wait limit and the test hook of a launch from a pending request.
template <class Params>
void take_stall(Params &p, int which) {
  const uint64_t st = g_stall[which].exchange(0, std::memory_order_relaxed);
  p.stall_ns = st;
  p.timeout_ns = st ? st : kWaitLimitNs;
}

struct DeviceFacts {
  int sm_count = 0;
  int ctas_per_sm[kMaxKernels + kKv4Kernels] = {};  // 0 = not yet configured (the 4-bit kernels' at the end)
};
std::mutex g_dev_mu;
DeviceFacts g_dev[kMaxDevices];

// Configures a kernel on the current device (opt-in shared memory) and
// returns its resident CTAs per SM, kept at `at`, and the SM count.
int occupancy(int at, const void *fn, int threads, size_t smem_bytes, int *ctas_per_sm, int *sm_count) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return cuda_status(e);
  if (dev < 0 || dev >= kMaxDevices) return PKV_EUNSUPPORTED;
  std::lock_guard<std::mutex> lock(g_dev_mu);
  DeviceFacts &f = g_dev[dev];
  if (f.sm_count == 0) {
    e = cudaDeviceGetAttribute(&f.sm_count, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return cuda_status(e);
  }
  if (f.ctas_per_sm[at] == 0) {
    e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem_bytes);
    if (e != cudaSuccess) return cuda_status(e);
    int nb = 0;
    e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&nb, fn, threads, smem_bytes);
    if (e != cudaSuccess) return cuda_status(e);
    if (nb <= 0) return PKV_EUNSUPPORTED;
    f.ctas_per_sm[at] = nb;
  }
  *ctas_per_sm = f.ctas_per_sm[at];
  *sm_count = f.sm_count;
  return PKV_OK;
}
int kernel_occupancy(int ki, int *ctas_per_sm, int *sm_count) {
  const DecodeKernel &k = registry().k[ki];
  return occupancy(ki, k.fn, k.warps * 32, k.smem_bytes, ctas_per_sm, sm_count);
}

// The current device's SM count (cached).
int device_sm_count(int *out) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return cuda_status(e);
  if (dev < 0 || dev >= kMaxDevices) return PKV_EUNSUPPORTED;
  std::lock_guard<std::mutex> lock(g_dev_mu);
  DeviceFacts &f = g_dev[dev];
  if (f.sm_count == 0) {
    e = cudaDeviceGetAttribute(&f.sm_count, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return cuda_status(e);
  }
  *out = f.sm_count;
  return PKV_OK;
}

PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void *p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) ==
            cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
  });
  return fn;
}

int esize_of(int dtype) {
  switch (dtype) {
    case PKV_F32: return 4;
    case PKV_F16: return 2;
    case PKV_BF16: return 2;
    case PKV_FP8_E4M3: return 1;
  }
  return 0;
}

// [a, a + na) and [b, b + nb) share a byte (null: no memory).
bool overlap(const void *a, size_t na, const void *b, size_t nb) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return a && b && x < y + nb && y < x + na;
}

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Tensor map over a [num_blocks][Hkv][16][D] cache as 2-D rows of 128 bytes
// wide boxes with the 128-byte swizzle; one box is 16 token rows x 128 bytes
// (or 8 lines of two 64-byte tokens).
// rows64: 64-byte rows as 16 x 64-byte boxes with the 64-byte swizzle instead (the
// K-major operand layout of an 8-bit tile of head dim 64).
int encode_cache_map(CUtensorMap *map, const void *base, int dtype, int64_t num_blocks, int Hkv, int D, bool rows64) {
  auto fn = encode_fn();
  if (!fn) return cuda_status(cudaErrorNotSupported);
  const int es = esize_of(dtype);
  const int rowb = D * es;
  cuuint64_t dims[2], strides[1];
  cuuint32_t box[2], estr[2] = {1, 1};
  const cuuint64_t tiles = (cuuint64_t)num_blocks * Hkv;
  if (rowb >= 128 || rows64) {
    dims[0] = (cuuint64_t)D;
    dims[1] = tiles * kBlock;
    strides[0] = (cuuint64_t)rowb;
    box[0] = rows64 ? D : 128 / es;
    box[1] = kBlock;
  } else {
    dims[0] = 128 / es;
    dims[1] = tiles * kBlock * rowb / 128;
    strides[0] = 128;
    box[0] = 128 / es;
    box[1] = kBlock * rowb / 128;
  }
  const CUtensorMapDataType dt = es == 1   ? CU_TENSOR_MAP_DATA_TYPE_UINT8
                                 : es == 2 ? CU_TENSOR_MAP_DATA_TYPE_UINT16
                                           : CU_TENSOR_MAP_DATA_TYPE_FLOAT32;
  CUresult r = fn(map, dt, 2, const_cast<void *>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  rows64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return cuda_status(cudaErrorInvalidValue);
  return PKV_OK;
}

// Encoded tensor maps of recently used caches.  A map depends only on the
// cache's base address, element type and dimensions, which make up the key,
// so a hit is always the map the encoder would produce; decode calls on the
// same cache (every layer step of a serving loop) skip the encoder.  Small
// and fixed in size, replaced round-robin; no allocation.
struct MapKey {
  const void *base;
  int64_t num_blocks;
  int dtype, Hkv, D;
  bool rows64;
  bool operator==(const MapKey &o) const {
    return base == o.base && num_blocks == o.num_blocks && dtype == o.dtype && Hkv == o.Hkv && D == o.D &&
           rows64 == o.rows64;
  }
};
struct MapCache {
  static constexpr int kEntries = 64;
  MapKey key[kEntries] = {};
  CUtensorMap map[kEntries];
  int used = 0, next = 0;
  std::mutex mu;
};
MapCache g_maps;

int cache_map(CUtensorMap *map, const void *base, int dtype, int64_t num_blocks, int Hkv, int D, bool rows64 = false) {
  const MapKey k{base, num_blocks, dtype, Hkv, D, rows64};
  {
    std::lock_guard<std::mutex> lock(g_maps.mu);
    for (int i = 0; i < g_maps.used; ++i)
      if (g_maps.key[i] == k) {
        *map = g_maps.map[i];
        return PKV_OK;
      }
  }
  const int rc = encode_cache_map(map, base, dtype, num_blocks, Hkv, D, rows64);
  if (rc != PKV_OK) return rc;
  std::lock_guard<std::mutex> lock(g_maps.mu);
  const int slot = g_maps.used < MapCache::kEntries ? g_maps.used++ : g_maps.next;
  if (g_maps.used == MapCache::kEntries) g_maps.next = (slot + 1) % MapCache::kEntries;
  g_maps.key[slot] = k;
  g_maps.map[slot] = *map;
  return PKV_OK;
}

struct Choice {
  int ki;   // registry index
  int GC;   // query rows per unit
  int NC;   // units per kv head
};

// Picks the kernel for a shape: tensor cores (8-row units, unused columns
// padded; 16-row units on fp8 caches past 8 rows) for every group size on
// 16-bit and fp8 caches — even for
// MHA the mma.sync block step measured faster on GB300 than the CUDA-core one
// (5.83 vs 5.56 TB/s, fp16 MHA layer) — and CUDA cores for fp32 caches.  The
// first compiled match is the default pipeline shape.  A build with
// PKV_SWEEP_SHAPES defined (pipeline-shape sweeps, not the product build)
// also compiles alternative shapes and lets PKV_PATH=mma|simt,
// PKV_DECODE_WARPS, PKV_DECODE_STAGES and PKV_DECODE_GC=8 in the environment
// pick among them.
int choose_kernel(int cache_dtype, int q_dtype, int D, int R, Choice *c, bool tree) {
#ifdef PKV_SWEEP_SHAPES
  static const int force = [] {
    const char *v = std::getenv("PKV_PATH");
    if (v && std::strcmp(v, "simt") == 0) return 1;
    if (v && std::strcmp(v, "mma") == 0) return 2;
    return 0;
  }();
  static const int want_warps = [] {
    const char *v = std::getenv("PKV_DECODE_WARPS");
    return v ? std::atoi(v) : 0;
  }();
  static const int want_stages = [] {
    const char *v = std::getenv("PKV_DECODE_STAGES");
    return v ? std::atoi(v) : 0;
  }();
  static const int want_gc = [] {
    const char *v = std::getenv("PKV_DECODE_GC");
    return v ? std::atoi(v) : 0;
  }();
#else
  constexpr int force = 0, want_warps = 0, want_stages = 0, want_gc = 0;
#endif
  const bool mma = cache_dtype != PKV_F32 && force != 1;
  // fp8 caches serve a kv head with more than 8 rows in 16-row units: each
  // E4M3 element is widened once per 16 rows instead of once per 8 (on the
  // 32K fp8 layer at 16 rows, one 16-row unit per kv head against two 8-row
  // units streaming the same blocks)
  int GC = mma ? 8 : (R >= 2 ? 2 : 1);
  if (mma && cache_dtype == PKV_FP8_E4M3 && R > 8 && want_gc != 8) GC = 16;
  Registry &r = registry();
  int first = -1;
  for (int pass = 0; pass < 2 && first < 0; ++pass) {
    if (pass == 1) {
      if (GC != 16) break;
      GC = 8;  // no 16-row kernel for this (q dtype, D): 8-row units
    }
    for (int i = 0; i < r.n; ++i) {
      const DecodeKernel &k = r.k[i];
      if (k.mma == (mma ? 1 : 0) && k.cache_dtype == cache_dtype && k.q_dtype == q_dtype && k.D == D && k.GC == GC &&
          k.tree == (tree ? 1 : 0)) {
        if (first < 0) first = i;
        if ((want_warps == 0 || k.warps == want_warps) && (want_stages == 0 || k.stages == want_stages)) {
          first = i;
          break;
        }
      }
    }
  }
  if (first < 0) return PKV_EUNSUPPORTED;
  c->ki = first;
  c->GC = GC;
  c->NC = (R + GC - 1) / GC;
  return PKV_OK;
}

constexpr double kCountLimit = 2147483000.0;  // 32-bit counts

int validate_shapes(int q_dtype, int cache_dtype, int B, int q_len, int Hq, int Hkv, int D, int64_t num_blocks,
                    int max_blocks) {
  if (B < 0 || Hq <= 0 || Hkv <= 0 || D <= 0 || num_blocks <= 0 || max_blocks <= 0) return PKV_EINVAL;
  if (q_len < 1 || q_len > PKV_MAX_Q_LEN) return PKV_EINVAL;
  if (max_blocks > (1 << 26)) return PKV_EUNSUPPORTED;  // 16 * max_blocks stays below 2^30
  if (Hq % Hkv != 0) return PKV_EINVAL;
  if (esize_of(cache_dtype) == 0 || esize_of(q_dtype) == 0 || q_dtype == PKV_FP8_E4M3) return PKV_EINVAL;
  if (D != 64 && D != 128) return PKV_EUNSUPPORTED;
  if (cache_dtype == PKV_F32 && q_dtype != PKV_F32) return PKV_EUNSUPPORTED;
  if ((cache_dtype == PKV_F16 || cache_dtype == PKV_BF16) && q_dtype != cache_dtype) return PKV_EUNSUPPORTED;
  if (cache_dtype == PKV_FP8_E4M3 && q_dtype == PKV_F32) return PKV_EUNSUPPORTED;
  // TMA row coordinates are 32-bit
  if ((double)num_blocks * Hkv * kBlock >= kCountLimit) return PKV_EUNSUPPORTED;
  return PKV_OK;
}

int validate_decode_shapes(int q_dtype, int cache_dtype, int B, int q_len, int Hq, int Hkv, int D,
                           int64_t num_blocks, int max_blocks) {
  const int rc = validate_shapes(q_dtype, cache_dtype, B, q_len, Hq, Hkv, D, num_blocks, max_blocks);
  if (rc != PKV_OK) return rc;
  // the work-item count is 32-bit
  const int R = q_len * (Hq / Hkv);  // query rows per kv head; units per kv head <= R
  if ((double)B * max_blocks * Hkv * R >= kCountLimit) return PKV_EUNSUPPORTED;
  return PKV_OK;
}

// Resolves the kernel and the partition count for a call.
int plan_call(int cache_dtype, int q_dtype, int B, int q_len, int Hq, int Hkv, int D, int num_splits, Choice *c,
              int *P, bool tree = false) {
  int rc = choose_kernel(cache_dtype, q_dtype, D, q_len * (Hq / Hkv), c, tree);
  if (rc != PKV_OK) return rc;
  if (num_splits < 0) return PKV_EINVAL;
  if (num_splits > 0) {
    *P = num_splits;
  } else {
    int ctas = 0, sms = 0;
    rc = kernel_occupancy(c->ki, &ctas, &sms);
    if (rc != PKV_OK) return rc;
    *P = sms * ctas * registry().k[c->ki].warps;
  }
  if (*P > (1 << 24)) return PKV_EINVAL;
  (void)B;
  return PKV_OK;
}

// The same of the 4-bit attention: units of 8 rows, 16 past 8 rows a kv head; P ranges, one per CTA: num_splits, or one
// per SM.
int plan_kv4(int q_dtype, int q_len, int Hq, int Hkv, int D, int num_splits, Choice *c, int *P) {
  const int R = q_len * (Hq / Hkv), GC = R > 8 ? 16 : 8;
  const Kv4Kernel *k = registry().kv4;
  for (c->ki = 0; c->ki < kKv4Kernels; ++c->ki)
    if (k[c->ki].q_dtype == q_dtype && k[c->ki].D == D && k[c->ki].GC == GC) break;
  if (c->ki == kKv4Kernels) return PKV_EUNSUPPORTED;
  c->GC = GC;
  c->NC = (R + GC - 1) / GC;
  if (num_splits < 0 || num_splits > (1 << 24)) return PKV_EINVAL;
  *P = num_splits;
  if (num_splits == 0) {
    const int rc = device_sm_count(P);
    if (rc != PKV_OK) return rc;
  }
  *P = std::min(*P, kKv4MaxRanges);
  return PKV_OK;
}

}  // namespace
}  // namespace pkv

using namespace pkv;

extern "C" {

int pkv_version(void) { return 10100; }

int pkv_set_route(int which, int choice) {
  if (which == PKV_ROUTE_MULTI_QUERY) {
    if (choice < PKV_ROUTE_AUTO || choice > PKV_MQ_UNITS) return PKV_EINVAL;
  } else if (which == PKV_ROUTE_PREFILL) {
    if (choice < PKV_ROUTE_AUTO || choice > PKV_PREFILL_PER_ITEM) return PKV_EINVAL;
  } else if (which == PKV_ROUTE_TREE) {
    if (choice < PKV_ROUTE_AUTO || choice > PKV_TREE_UNITS) return PKV_EINVAL;
  } else {
    return PKV_EINVAL;
  }
  g_route[which].store(choice, std::memory_order_relaxed);
  return PKV_OK;
}

int pkv_test_stall_next(int which, uint64_t limit_ns) {
  if (which != PKV_STALL_DECODE && which != PKV_STALL_PREFILL) return PKV_EINVAL;
  if (limit_ns != 0 && (limit_ns < 1000000ull || limit_ns > 10000000000ull)) return PKV_EINVAL;
  g_stall[which].store(limit_ns, std::memory_order_relaxed);
  return PKV_OK;
}

int pkv_get_route(int which) {
  if (which != PKV_ROUTE_MULTI_QUERY && which != PKV_ROUTE_PREFILL && which != PKV_ROUTE_TREE) return PKV_EINVAL;
  return g_route[which].load(std::memory_order_relaxed);
}

int pkv_last_cuda_error(void) { return g_last_cuda_error; }

const char *pkv_status_string(int status) {
  switch (status) {
    case PKV_OK: return "ok";
    case PKV_EINVAL: return "invalid argument";
    case PKV_EUNSUPPORTED: return "unsupported shape or dtype combination";
    case PKV_EWORKSPACE: return "workspace missing, misaligned or too small";
    case PKV_ECUDA: return "CUDA runtime error";
    case PKV_ETIMEOUT: return "an in-kernel wait timed out";
    case PKV_EOOM: return "no free physical block";
    case PKV_ERANGE: return "value out of range";
    case PKV_ENOTFOUND: return "unknown sequence id";
  }
  return "unknown status";
}

int paged_kv_append(const void *k_new, const void *v_new, int new_dtype, void *k_cache, void *v_cache,
                    int cache_dtype, float *k_scale, float *v_scale, const int64_t *slot_mapping, int B, int Hkv,
                    int D, int64_t num_blocks, pkv_stream_t stream) {
  if (B < 0 || Hkv <= 0 || num_blocks <= 0) return PKV_EINVAL;
  if (esize_of(cache_dtype) == 0 || esize_of(new_dtype) == 0) return PKV_EINVAL;
  if (D != 64 && D != 128) return PKV_EUNSUPPORTED;
  if (B == 0) return PKV_OK;
  if (!k_new || !v_new || !k_cache || !v_cache || !slot_mapping) return PKV_EINVAL;
  if (cache_dtype == PKV_FP8_E4M3) {
    if (new_dtype == PKV_FP8_E4M3) return PKV_EUNSUPPORTED;
    if (!k_scale || !v_scale) return PKV_EINVAL;
  } else {
    if (new_dtype != cache_dtype) return PKV_EUNSUPPORTED;
    if (!aligned16(k_new) || !aligned16(v_new)) return PKV_EINVAL;
  }
  if (!aligned16(k_cache) || !aligned16(v_cache)) return PKV_EINVAL;
  return cuda_status(launch_append(k_new, v_new, new_dtype, k_cache, v_cache, cache_dtype, k_scale, v_scale,
                                   slot_mapping, B, Hkv, D, num_blocks, reinterpret_cast<cudaStream_t>(stream)));
}

int paged_decode_multi_workspace_bytes(int B, int q_len, int Hq, int Hkv, int D, int cache_dtype, int q_dtype,
                                       int num_splits, size_t *bytes_out) {
  if (!bytes_out) return PKV_EINVAL;
  int rc = validate_decode_shapes(q_dtype, cache_dtype, B, q_len, Hq, Hkv, D, 1, 1);
  if (rc != PKV_OK) return rc;
  Choice c;
  int P = 0;
  rc = plan_call(cache_dtype, q_dtype, B, q_len, Hq, Hkv, D, num_splits, &c, &P);
  if (rc != PKV_OK) return rc;
  size_t total = ws_layout(B, P, D, c.GC).total;
  if (q_len >= 2 && num_splits == 0 && D == kMqHeadDim && q_len * (Hq / Hkv) <= kMqRows && B <= kMqMaxBatch &&
      (cache_dtype == PKV_BF16 || cache_dtype == PKV_F16 ||
       (cache_dtype == PKV_FP8_E4M3 && q_len * (Hq / Hkv) <= kMqRowsFp8))) {
    int sms = 0;
    rc = device_sm_count(&sms);
    if (rc != PKV_OK) return rc;
    const size_t mq = mq_ws_layout(B, sms).total;  // the transposed kernel's partials
    if (mq > total) total = mq;
  }
  *bytes_out = total;
  return PKV_OK;
}

int paged_kv_append_calibrated(const void *k_new, const void *v_new, int new_dtype, void *k_cache, void *v_cache,
                               int cache_dtype, float *k_scale, float *v_scale, const int64_t *slot_mapping, int B,
                               int Hkv, int D, int64_t num_blocks, pkv_stream_t stream) {
  if (cache_dtype != PKV_FP8_E4M3)
    return paged_kv_append(k_new, v_new, new_dtype, k_cache, v_cache, cache_dtype, k_scale, v_scale, slot_mapping, B,
                           Hkv, D, num_blocks, stream);
  if (B < 0 || Hkv <= 0 || num_blocks <= 0) return PKV_EINVAL;
  if (esize_of(new_dtype) == 0) return PKV_EINVAL;
  if (new_dtype == PKV_FP8_E4M3) return PKV_EUNSUPPORTED;
  if (D != 64 && D != 128) return PKV_EUNSUPPORTED;
  if (B == 0) return PKV_OK;
  if (!k_new || !v_new || !k_cache || !v_cache || !slot_mapping || !k_scale || !v_scale) return PKV_EINVAL;
  if (!aligned16(k_cache) || !aligned16(v_cache)) return PKV_EINVAL;
  return cuda_status(launch_append_calibrated(k_new, v_new, new_dtype, k_cache, v_cache, k_scale, v_scale,
                                              slot_mapping, B, Hkv, D, num_blocks,
                                              reinterpret_cast<cudaStream_t>(stream)));
}

int paged_decode_workspace_bytes(int B, int Hq, int Hkv, int D, int cache_dtype, int q_dtype, int num_splits,
                                 size_t *bytes_out) {
  return paged_decode_multi_workspace_bytes(B, 1, Hq, Hkv, D, cache_dtype, q_dtype, num_splits, bytes_out);
}

int paged_decode_attention(void *out, const void *q, int q_dtype, const void *k_cache, const void *v_cache,
                           int cache_dtype, const float *k_scale, const float *v_scale, const int32_t *block_table,
                           int max_blocks_per_seq, const int32_t *context_lens, int B, int Hq, int Hkv, int D,
                           int64_t num_blocks, float scale, int num_splits, void *workspace, size_t workspace_bytes,
                           pkv_stream_t stream) {
  return paged_decode_attention_multi(out, q, q_dtype, k_cache, v_cache, cache_dtype, k_scale, v_scale, block_table,
                                      max_blocks_per_seq, context_lens, B, 1, 0, Hq, Hkv, D, num_blocks, scale,
                                      num_splits, workspace, workspace_bytes, stream);
}

// The two prefill kernels run one tile pipeline and differ in scheduling.
// One CTA per work item (row tile x kv head x sequence) runs the per-tile
// loop fastest and suits long items: new tokens after a cached prefix of
// thousands of positions.  The persistent kernel (one CTA per SM walking its
// items) saves each item's start-up and balances short items of unequal
// length: prompts without a long prefix.  The longest context the block
// table can describe (max_blocks * block size) less the new tokens bounds
// the prefix; a bound of 2048 positions or more picks one CTA per item, or
// 1024 for items of at most 64 rows (a few new tokens of one group), which
// that kernel serves with row replicas (measured on 70B-layer shapes: at
// 1024 positions the two kernels tie, at 1500 one CTA per item is 11 %
// faster, at 300-512 the persistent kernel is 14-15 % faster).
// pkv_set_route(PKV_ROUTE_PREFILL, ...) overrides the choice.
static cudaError_t launch_prefill_auto(const PrefillParams &p, int cache_dtype, const CUtensorMap &tmK,
                                       const CUtensorMap &tmV, cudaStream_t s) {
  const int64_t bound = (int64_t)p.max_q_len * p.G <= 64 ? 1024 : 2048;
  bool tiles = (int64_t)p.max_blocks * kBlock - p.max_q_len >= bound;
  const int force = g_route[PKV_ROUTE_PREFILL].load(std::memory_order_relaxed);
  if (force == PKV_PREFILL_PER_ITEM) tiles = true;
  if (force == PKV_PREFILL_PERSISTENT) tiles = false;
  return tiles ? launch_prefill_tiles(p, cache_dtype, tmK, tmV, s) : launch_prefill(p, cache_dtype, tmK, tmV, s);
}

// A call's parameters for the decode kernels that stream units (decode.cuh,
// kv4_decode.cu) and for their merge.
static DecodeParams unit_params(const Choice &c, int P, void *out, const void *q, int q_dtype, const float *k_scale,
                                const float *v_scale, const int32_t *block_table, int max_blocks_per_seq,
                                const int32_t *context_lens, int B, int q_len, int window, int Hq, int Hkv, int D,
                                int64_t num_blocks, float scale, void *workspace) {
  const WsLayout L = ws_layout(B, P, D, c.GC);
  uint8_t *ws = static_cast<uint8_t *>(workspace);
  DecodeParams p;
  std::memset(&p, 0, sizeof(p));
  p.out = out;
  p.q = q;
  p.k_scale = k_scale;
  p.v_scale = v_scale;
  p.block_table = block_table;
  p.context_lens = context_lens;
  p.hdr = reinterpret_cast<WsHeader *>(ws + L.hdr);
  p.prefix = reinterpret_cast<int32_t *>(ws + L.prefix);
  p.starts = reinterpret_cast<int4 *>(ws + L.starts);
  p.part_o = reinterpret_cast<float *>(ws + L.part_o);
  p.part_lse = reinterpret_cast<float *>(ws + L.part_lse);
  p.cta_flags = reinterpret_cast<int32_t *>(ws + L.cta_flags);
  p.num_blocks = num_blocks;
  p.B = B;
  p.Hq = Hq;
  p.Hkv = Hkv;
  p.D = D;
  p.G = Hq / Hkv;
  p.GC = c.GC;
  p.NC = c.NC;
  p.HU = Hkv * c.NC;
  p.q_len = q_len;
  p.R = q_len * p.G;
  // a window of 2^30 positions or more covers any context this call accepts
  p.window = window < (1 << 30) ? window : 0;
  p.wlen = p.window > 0 ? p.window : (1 << 30);
  p.P = P;
  p.max_blocks = max_blocks_per_seq;
  p.out_dtype = q_dtype;
  p.scale_log2 = scale * 1.4426950408889634f;
  p.inline_plan = B + 1 <= kInlinePrefix ? 1 : 0;
  take_stall(p, PKV_STALL_DECODE);
  return p;
}

// Plan (large batches) and decode kernel.
static cudaError_t launch_units(const void *fn, int threads, size_t smem_bytes, const DecodeParams &p, void **args,
                                cudaStream_t s) {
  const bool pdl = s != nullptr;  // programmatic launch on explicit streams only
  cudaError_t e = cudaSuccess;
  if (!p.inline_plan) {
    e = launch_plan(p, s);
    if (e != cudaSuccess) return e;
  }

  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(p.n_ctas);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem_bytes;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pdl ? 1 : 0;
  return cudaLaunchKernelExC(&cfg, fn, args);
}

// The decode kernel (8- or 16-row units, one partition per warp) and its
// split-KV merge: single-token decode, and several new tokens per sequence on
// the unit route, causal or (tree) under per-node masks.
struct TreeArgs {
  const uint64_t *mask;
  const int32_t *lens;
  int mask_stride;
};
static int run_units(const Choice &c, int P, void *out, const void *q, int q_dtype, const void *k_cache,
                     const void *v_cache, int cache_dtype, const float *k_scale, const float *v_scale,
                     const int32_t *block_table, int max_blocks_per_seq, const int32_t *context_lens, int B, int q_len,
                     int window, int Hq, int Hkv, int D, int64_t num_blocks, float scale, void *workspace,
                     pkv_stream_t stream, const TreeArgs *tree) {
  int ctas = 0, sms = 0;
  int rc = kernel_occupancy(c.ki, &ctas, &sms);  // also opts the kernel into its shared memory
  if (rc != PKV_OK) return rc;

  CUtensorMap tmK, tmV;
  rc = cache_map(&tmK, k_cache, cache_dtype, num_blocks, Hkv, D);
  if (rc != PKV_OK) return rc;
  rc = cache_map(&tmV, v_cache, cache_dtype, num_blocks, Hkv, D);
  if (rc != PKV_OK) return rc;

  DecodeParams p = unit_params(c, P, out, q, q_dtype, k_scale, v_scale, block_table, max_blocks_per_seq, context_lens, B,
                               q_len, window, Hq, Hkv, D, num_blocks, scale, workspace);
  const DecodeKernel &k = registry().k[c.ki];
  p.n_ctas = (P + k.warps - 1) / k.warps;
  if (tree) {
    p.tree_mask = tree->mask;
    p.tree_lens = tree->lens;
    p.mask_stride = tree->mask_stride;
    p.v_cache = v_cache;
  }
  void *args[3] = {&p, &tmK, &tmV};
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t e = launch_units(k.fn, k.warps * 32, k.smem_bytes, p, args, s);
  if (e == cudaSuccess) e = launch_splitk_merge(p, s, s != nullptr);
  return cuda_status(e);
}

// The call's parameters for the kernels that share the stream-K schedule
// (mq_walk.cuh), on a workspace laid out as M.
static MqParams mq_params(const MqWsLayout &M, void *out, const void *q, const float *k_scale, const float *v_scale,
                          const int32_t *block_table, int max_blocks_per_seq, const int32_t *context_lens, int B,
                          int q_len, int window, int Hq, int Hkv, int64_t num_blocks, float scale, void *workspace,
                          const TreeArgs *tree) {
  uint8_t *ws = static_cast<uint8_t *>(workspace);
  MqParams mp;
  std::memset(&mp, 0, sizeof(mp));
  mp.out = out;
  mp.q = q;
  mp.k_scale = k_scale;
  mp.v_scale = v_scale;
  mp.block_table = block_table;
  mp.context_lens = context_lens;
  mp.status = &reinterpret_cast<WsHeader *>(ws)->status;
  mp.cta_flags = reinterpret_cast<int32_t *>(ws + M.cta_flags);
  mp.prefix = reinterpret_cast<int32_t *>(ws + M.prefix);
  mp.part_o = reinterpret_cast<float *>(ws + M.part_o);
  mp.part_lse = reinterpret_cast<float *>(ws + M.part_lse);
  mp.num_blocks = num_blocks;
  mp.B = B;
  mp.q_len = q_len;
  mp.Hq = Hq;
  mp.Hkv = Hkv;
  mp.G = Hq / Hkv;
  mp.R = q_len * mp.G;
  mp.max_blocks = max_blocks_per_seq;
  mp.window = window < (1 << 30) ? window : 0;
  mp.scale_log2 = scale * 1.4426950408889634f;
  mp.timeout_ns = kWaitLimitNs;
  if (tree) {
    mp.tree_mask = tree->mask;
    mp.tree_lens = tree->lens;
    mp.mask_stride = tree->mask_stride;
  }
  return mp;
}

// The transposed tensor-core kernel (head dim 128) and its merge, on the
// workspace mq_ws_layout(B, sms) describes.
static int run_mq(void *out, const void *q, int q_dtype, const void *k_cache, const void *v_cache, int cache_dtype,
                  const float *k_scale, const float *v_scale, const int32_t *block_table, int max_blocks_per_seq,
                  const int32_t *context_lens, int B, int q_len, int window, int Hq, int Hkv, int64_t num_blocks,
                  float scale, void *workspace, int sms, pkv_stream_t stream) {
  const MqWsLayout M = mq_ws_layout(B, sms);
  CUtensorMap tmK, tmV;
  int rc = cache_map(&tmK, k_cache, cache_dtype, num_blocks, Hkv, kMqHeadDim);
  if (rc != PKV_OK) return rc;
  rc = cache_map(&tmV, v_cache, cache_dtype, num_blocks, Hkv, kMqHeadDim);
  if (rc != PKV_OK) return rc;
  const MqParams mp = mq_params(M, out, q, k_scale, v_scale, block_table, max_blocks_per_seq, context_lens, B, q_len,
                                window, Hq, Hkv, num_blocks, scale, workspace, nullptr);
  return cuda_status(launch_mq_decode(mp, cache_dtype, q_dtype, tmK, tmV, sms, reinterpret_cast<cudaStream_t>(stream)));
}

int paged_decode_attention_multi(void *out, const void *q, int q_dtype, const void *k_cache, const void *v_cache,
                                 int cache_dtype, const float *k_scale, const float *v_scale,
                                 const int32_t *block_table, int max_blocks_per_seq, const int32_t *context_lens,
                                 int B, int q_len, int window, int Hq, int Hkv, int D, int64_t num_blocks,
                                 float scale, int num_splits, void *workspace, size_t workspace_bytes,
                                 pkv_stream_t stream) {
  int rc = validate_decode_shapes(q_dtype, cache_dtype, B, q_len, Hq, Hkv, D, num_blocks, max_blocks_per_seq);
  if (rc != PKV_OK) return rc;
  if (window < 0) return PKV_EINVAL;
  if (!std::isfinite(scale)) return PKV_EINVAL;
  if (B == 0) return PKV_OK;
  if (!out || !q || !k_cache || !v_cache || !block_table || !context_lens) return PKV_EINVAL;
  if (cache_dtype == PKV_FP8_E4M3 && (!k_scale || !v_scale)) return PKV_EINVAL;
  if (!aligned16(out) || !aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache)) return PKV_EINVAL;
  Choice c;
  int P = 0;
  rc = plan_call(cache_dtype, q_dtype, B, q_len, Hq, Hkv, D, num_splits, &c, &P);
  if (rc != PKV_OK) return rc;
  const WsLayout L = ws_layout(B, P, D, c.GC);
  if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255u) != 0 || workspace_bytes < L.total)
    return PKV_EWORKSPACE;
  if (q_len >= 2 && num_splits == 0) {
    // Several new tokens per sequence on a 16-bit cache: a tensor-core
    // kernel streams each (sequence, kv head)'s K/V once for all of its
    // q_len * G rows (the decode kernel's units below stream it once per
    // unit).
    //  * up to 32 rows and head dim 128: the transposed kernel (positions on
    //    the tensor core's M side, stream-K over every item's tiles, so any
    //    batch fills the GPU);
    //  * otherwise the prefill kernel with 128-row tiles, when its grid of
    //    (sequence, kv head, row tile) items fills the GPU (no context split;
    //    on the 70B layer at 64 rows it is faster than the transposed kernel,
    //    whose softmax work grows with the rows);
    //  * the transposed kernel for 33-64 rows on grids the prefill kernel
    //    cannot fill.
    // pkv_set_route(PKV_ROUTE_MULTI_QUERY, ...) forces one route where it
    // applies (for measurement and tests).
    int sms = 0;
    rc = device_sm_count(&sms);
    if (rc != PKV_OK) return rc;
    const int force = g_route[PKV_ROUTE_MULTI_QUERY].load(std::memory_order_relaxed);
    const bool units = force == PKV_MQ_UNITS;
    const bool no_mq = units || force == PKV_MQ_PREFILL;
    const bool want_mq = force == PKV_MQ_TRANSPOSED;
    const int G = Hq / Hkv;
    const int R = q_len * G;
    const int64_t tiles = ((int64_t)q_len * G + 127) / 128;
    const bool prefill_fills = (int64_t)B * Hkv * tiles >= sms && B <= 65535;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    // FP8 caches take the decode kernel's units (16 rows each past 8 rows):
    // the transposed kernel widens each tile to f16 in shared memory, which
    // on 32 KiB fp8 tiles costs more than the tile's HBM time (~2.1 TB/s
    // whatever the rows, against the units' 6.1 / 4.6 / 2.4 TB/s at 8 / 16 /
    // 32 rows on the 32K fp8 layer); it runs only when forced.  FP8 caches
    // have no prefill route.
    const bool fp8 = cache_dtype == PKV_FP8_E4M3;
    const bool fp8_mq = fp8 && R <= kMqRowsFp8 && want_mq;
    if (!no_mq && (cache_dtype == PKV_BF16 || cache_dtype == PKV_F16 || fp8_mq) && scale > 0.f &&
        D == kMqHeadDim && R <= kMqRows && B <= kMqMaxBatch && (R <= 32 || !prefill_fills || want_mq)) {
      if (workspace_bytes >= mq_ws_layout(B, sms).total)
        return run_mq(out, q, q_dtype, k_cache, v_cache, cache_dtype, k_scale, v_scale, block_table,
                      max_blocks_per_seq, context_lens, B, q_len, window, Hq, Hkv, num_blocks, scale, workspace, sms,
                      stream);
    }
    if (!units && (cache_dtype == PKV_BF16 || cache_dtype == PKV_F16) && scale > 0.f && prefill_fills) {
      CUtensorMap tmK, tmV;
      rc = cache_map(&tmK, k_cache, cache_dtype, num_blocks, Hkv, D);
      if (rc != PKV_OK) return rc;
      rc = cache_map(&tmV, v_cache, cache_dtype, num_blocks, Hkv, D);
      if (rc != PKV_OK) return rc;
      WsHeader *hdr = reinterpret_cast<WsHeader *>(static_cast<uint8_t *>(workspace) + L.hdr);
      cudaError_t e = cudaMemsetAsync(&hdr->status, 0, sizeof(int32_t), s);
      if (e != cudaSuccess) return cuda_status(e);
      PrefillParams pp;
      std::memset(&pp, 0, sizeof(pp));
      pp.out = out;
      pp.q = q;
      pp.block_table = block_table;
      pp.context_lens = context_lens;
      pp.q_start = nullptr;
      pp.uniform_q_len = q_len;
      pp.status = &hdr->status;
      pp.num_blocks = num_blocks;
      pp.B = B;
      pp.Hq = Hq;
      pp.Hkv = Hkv;
      pp.D = D;
      pp.G = G;
      pp.max_blocks = max_blocks_per_seq;
      pp.max_q_len = q_len;
      pp.max_tiles = (int)tiles;
      pp.window = window < (1 << 30) ? window : 0;
      pp.scale_log2 = scale * 1.4426950408889634f;
      take_stall(pp, PKV_STALL_PREFILL);
      return cuda_status(launch_prefill_auto(pp, cache_dtype, tmK, tmV, s));
    }
  }
  return run_units(c, P, out, q, q_dtype, k_cache, v_cache, cache_dtype, k_scale, v_scale, block_table,
                   max_blocks_per_seq, context_lens, B, q_len, window, Hq, Hkv, D, num_blocks, scale, workspace, stream,
                   nullptr);
}

// Kernels of paged_tree_attention (PKV_TREE_*): which one a shape takes, or the
// forced one (pkv_set_route) where it applies.  The row tiles read an item's
// cache once for 128 rows and split it anywhere; the units read it once per 8
// rows or fewer.  Up to 8 rows per kv head (fp8: 16) both read it once (or
// twice, from L2) and the choice is by what the table can hold.  Units / tiles, us, out of a cold L2:
//   16-bit, D = 128: the tiles, but for many items (a range then holds the ends
//     of several), where both are equal: 1 x 16384, 8 heads of 8 rows 60 / 34,
//     16 x 8192 115 / 113, 64 x 500 47 / 46, 16 x 1000, 32 heads of 8 71 / 70, 64 x
//     500, 32 heads of 4 122 / 122;
//   D = 64 and fp8 (half the bytes a tile, or V to widen for 128 rows): the
//     tiles for small work: bf16 D = 64, 8 rows, 1 x 16384 53 / 28, 16 x 1000
//     25 / 22, 64 x 500 31 / 36, 16 x 4096 46 / 52; fp8 D = 128, 8 heads of 4 /
//     16 rows, 1 x 500 23, 29 / 19, 19, 16 x 1000 31, 42 / 25, 25, 4 x 8192 42, 52 /
//     41, 42, 8 x 8192 53, 62 / 59, 60, 64 x 500 36, 58 / 53, 53, 32 x 2000 50, 67 /
//     70, 71, 16 x 8192 74, 90 / 94, 94; fp8 D = 64, 16 rows, 16 x 1000 31 / 22,
//     64 x 500 40 / 44, 16 x 2000 38 / 36, 64 x 4096 123 / 150.
// Above, the tiles everywhere: 16-bit D = 128, 16 x 8192, 16 rows 128 / 113; D =
// 64, 16 x 4096, 16 rows 59 / 52; fp8 16 x 8192, 32 rows 145 / 95.
static bool tree_tiles_apply(int cache_dtype, int B) {
  return cache_dtype != PKV_F32 && B <= kMqMaxBatch;
}
static int tree_route(int cache_dtype, int B, int R, int Hkv, int D, int max_blocks) {
  const int force = g_route[PKV_ROUTE_TREE].load(std::memory_order_relaxed);
  const bool fp8 = cache_dtype == PKV_FP8_E4M3;
  if (!tree_tiles_apply(cache_dtype, B) || force == PKV_TREE_UNITS) return PKV_TREE_UNITS;
  if (force == PKV_TREE_TILES || R > (fp8 ? 16 : 8)) return PKV_TREE_TILES;
  const int64_t items = (int64_t)B * Hkv;
  if (!fp8 && D == 128) return items < 512 ? PKV_TREE_TILES : PKV_TREE_UNITS;
  const int64_t rows = items * max_blocks * kBlock;  // K rows, at most
  return rows <= (items <= 32 ? 1 << 18 : 1 << 17) ? PKV_TREE_TILES : PKV_TREE_UNITS;
}

// Shapes of a tree call: a tree has up to 64 nodes' rows, so the decode kernel's limit
// (a unit per row at worst) would refuse long tables of wide batches that either kernel
// serves.  Query rows are counted in 32 bits, ...
static int validate_tree_shapes(int q_dtype, int cache_dtype, int B, int q_len, int Hq, int Hkv, int D,
                                int64_t num_blocks, int max_blocks) {
  const int rc = validate_shapes(q_dtype, cache_dtype, B, q_len, Hq, Hkv, D, num_blocks, max_blocks);
  if (rc != PKV_OK) return rc;
  return (double)std::max(B, 1) * q_len * Hq < kCountLimit ? PKV_OK : PKV_EUNSUPPORTED;
}
// ... and so are the route's work items: K / V tiles of 128 positions, or (unit, block) pairs.
static int tree_items(int route, const Choice &c, int B, int Hkv, int max_blocks) {
  const double items = route == PKV_TREE_TILES ? (double)B * Hkv * ((max_blocks + 7) / 8) : (double)B * Hkv * c.NC * max_blocks;
  return items < kCountLimit ? PKV_OK : PKV_EUNSUPPORTED;
}

int paged_tree_workspace_bytes(int B, int q_len, int Hq, int Hkv, int D, int cache_dtype, int q_dtype,
                               size_t *bytes_out) {
  if (!bytes_out) return PKV_EINVAL;
  int rc = validate_tree_shapes(q_dtype, cache_dtype, B, q_len, Hq, Hkv, D, 1, 1);
  if (rc != PKV_OK) return rc;
  Choice c;
  int P = 0;
  rc = plan_call(cache_dtype, q_dtype, B, q_len, Hq, Hkv, D, 0, &c, &P, true);
  if (rc != PKV_OK) return rc;
  size_t total = ws_layout(B, P, D, c.GC).total;
  int sms = 0;
  rc = device_sm_count(&sms);
  if (rc != PKV_OK) return rc;
  const int R = q_len * (Hq / Hkv);
  if (tree_tiles_apply(cache_dtype, B)) {
    int RT = 0, groups = 0;
    tree_tiles_grid(R, sms, &RT, &groups);
    total = std::max(total, tree_tiles_ws_layout(D, RT, groups).total);
  }
  *bytes_out = total;
  return PKV_OK;
}

int paged_tree_attention(void *out, const void *q, int q_dtype, const void *k_cache, const void *v_cache,
                         int cache_dtype, const float *k_scale, const float *v_scale, const int32_t *block_table,
                         int max_blocks_per_seq, const int32_t *context_lens, const uint64_t *tree_mask,
                         int mask_per_seq, const int32_t *tree_lens, int B, int q_len, int window, int Hq, int Hkv,
                         int D, int64_t num_blocks, float scale, void *workspace, size_t workspace_bytes,
                         pkv_stream_t stream) {
  int rc = validate_tree_shapes(q_dtype, cache_dtype, B, q_len, Hq, Hkv, D, num_blocks, max_blocks_per_seq);
  if (rc != PKV_OK) return rc;
  const int R = q_len * (Hq / Hkv), route = tree_route(cache_dtype, B, R, Hkv, D, max_blocks_per_seq);
  Choice c;
  rc = choose_kernel(cache_dtype, q_dtype, D, R, &c, true);
  if (rc == PKV_OK) rc = tree_items(route, c, B, Hkv, max_blocks_per_seq);
  if (rc != PKV_OK) return rc;
  if (window < 0 || (mask_per_seq != 0 && mask_per_seq != 1)) return PKV_EINVAL;
  if (!(scale > 0.f) || !std::isfinite(scale)) return PKV_EINVAL;
  if (B == 0) return PKV_OK;
  if (!out || !q || !k_cache || !v_cache || !block_table || !context_lens || !tree_mask) return PKV_EINVAL;
  if (cache_dtype == PKV_FP8_E4M3 && (!k_scale || !v_scale)) return PKV_EINVAL;
  if (!aligned16(out) || !aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache)) return PKV_EINVAL;
  if ((reinterpret_cast<uintptr_t>(tree_mask) & 7u) != 0) return PKV_EINVAL;
  if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255u) != 0) return PKV_EWORKSPACE;
  const TreeArgs tree{tree_mask, tree_lens, mask_per_seq ? q_len : 0};
  int sms = 0;
  rc = device_sm_count(&sms);
  if (rc != PKV_OK) return rc;
  if (route == PKV_TREE_TILES) {
    CUtensorMap tmK, tmV;
    rc = cache_map(&tmK, k_cache, cache_dtype, num_blocks, Hkv, D, cache_dtype == PKV_FP8_E4M3 && D == 64);
    if (rc != PKV_OK) return rc;
    rc = cache_map(&tmV, v_cache, cache_dtype, num_blocks, Hkv, D);
    if (rc != PKV_OK) return rc;
    TreeTileParams tp;
    std::memset(&tp, 0, sizeof(tp));
    tree_tiles_grid(R, sms, &tp.RT, &tp.groups);
    tp.D = D;
    const MqWsLayout M = tree_tiles_ws_layout(D, tp.RT, tp.groups);
    if (workspace_bytes < M.total) return PKV_EWORKSPACE;
    tp.m = mq_params(M, out, q, k_scale, v_scale, block_table,
                     max_blocks_per_seq, context_lens, B, q_len, window, Hq, Hkv, num_blocks, scale, workspace, &tree);
    tp.cuts = reinterpret_cast<TreeCut *>(tp.m.prefix);
    tp.v_cache = v_cache;
    // a table too short for an item to be cut: the merge's launch would join nothing
    // (1 sequence of 333, 7 nodes: 14.8 us with it, 12.1 without)
    WsHeader *hdr = static_cast<WsHeader *>(workspace);
    if ((int64_t)max_blocks_per_seq * kBlock <= kUncutTiles * 128 && tp.RT * tp.groups <= (int)sizeof(hdr->cta_status))
      tp.cta_status = hdr->cta_status;
    return cuda_status(launch_tree_tiles(tp, cache_dtype, q_dtype, tmK, tmV, reinterpret_cast<cudaStream_t>(stream)));
  }
  int P = 0;
  rc = plan_call(cache_dtype, q_dtype, B, q_len, Hq, Hkv, D, 0, &c, &P, true);
  if (rc != PKV_OK) return rc;
  if (workspace_bytes < ws_layout(B, P, D, c.GC).total) return PKV_EWORKSPACE;
  return run_units(c, P, out, q, q_dtype, k_cache, v_cache, cache_dtype, k_scale, v_scale, block_table,
                   max_blocks_per_seq, context_lens, B, q_len, window, Hq, Hkv, D, num_blocks, scale, workspace, stream,
                   &tree);
}

int paged_tree_verify(int32_t *path, int32_t *path_len, int64_t *next_token, const int64_t *draft_tokens,
                      const uint64_t *tree_mask, int mask_per_seq, const int32_t *tree_lens, const void *target_probs,
                      int64_t ld_target, const void *draft_probs, int64_t ld_draft, int prob_dtype,
                      const float *uniforms, int B, int q_len, int V, pkv_stream_t stream) {
  if (B < 0 || V <= 0 || q_len < 1 || q_len > PKV_MAX_Q_LEN) return PKV_EINVAL;
  if (prob_dtype != PKV_F32 && prob_dtype != PKV_F16 && prob_dtype != PKV_BF16)
    return esize_of(prob_dtype) == 0 ? PKV_EINVAL : PKV_EUNSUPPORTED;
  if (mask_per_seq != 0 && mask_per_seq != 1) return PKV_EINVAL;
  if (V > (1 << 30) || B > (1 << 24)) return PKV_EUNSUPPORTED;
  if (ld_target < V || (draft_probs && ld_draft < V) || (draft_probs && !uniforms)) return PKV_EINVAL;
  if (B == 0) return PKV_OK;
  if (!path || !path_len || !next_token || !draft_tokens || !tree_mask || !target_probs) return PKV_EINVAL;
  const uintptr_t es = (uintptr_t)esize_of(prob_dtype);
  if (reinterpret_cast<uintptr_t>(target_probs) % es != 0 || reinterpret_cast<uintptr_t>(draft_probs) % es != 0 ||
      (reinterpret_cast<uintptr_t>(tree_mask) & 7u) != 0)
    return PKV_EINVAL;
  VerifyParams p;
  std::memset(&p, 0, sizeof(p));
  p.path = path;
  p.path_len = path_len;
  p.next_token = next_token;
  p.tokens = draft_tokens;
  p.mask = tree_mask;
  p.lens = tree_lens;
  p.target = target_probs;
  p.draft = draft_probs;
  p.u = uniforms;
  p.ld_target = ld_target;
  p.ld_draft = ld_draft;
  p.n = q_len;
  p.mask_stride = mask_per_seq ? q_len : 0;
  p.V = V;
  int sms = 0;
  const int rc = device_sm_count(&sms);
  if (rc != PKV_OK) return rc;
  return cuda_status(launch_tree_verify(p, prob_dtype, B, sms, reinterpret_cast<cudaStream_t>(stream)));
}

static int run_commit(void *k_cache, void *v_cache, int cache_dtype, float *k_scale, float *v_scale,
                      const int32_t *path, const int32_t *path_len, const int32_t *block_table,
                      int max_blocks_per_seq, const int32_t *context_lens, const int32_t *tree_lens,
                      int32_t *new_lens, int B, int q_len, int Hkv, int D, int64_t num_blocks, bool calibrated,
                      pkv_stream_t stream) {
  if (B < 0 || Hkv <= 0 || num_blocks <= 0 || max_blocks_per_seq <= 0) return PKV_EINVAL;
  if (q_len < 1 || q_len > PKV_MAX_Q_LEN) return PKV_EINVAL;
  if (esize_of(cache_dtype) == 0) return PKV_EINVAL;
  if (D != 64 && D != 128) return PKV_EUNSUPPORTED;
  if (max_blocks_per_seq > (1 << 26) || (double)B * Hkv >= 1073741000.0) return PKV_EUNSUPPORTED;
  if (B == 0) return PKV_OK;
  if (!k_cache || !v_cache || !path || !path_len || !block_table || !context_lens) return PKV_EINVAL;
  if (cache_dtype == PKV_FP8_E4M3 && (!k_scale || !v_scale)) return PKV_EINVAL;
  if (!aligned16(k_cache) || !aligned16(v_cache)) return PKV_EINVAL;
  // a sequence's new length is written while other warps still read what it comes from
  const size_t per = sizeof(int32_t) * (size_t)B;
  if (overlap(new_lens, per, context_lens, per) || overlap(new_lens, per, tree_lens, per) ||
      overlap(new_lens, per, path_len, per) || overlap(new_lens, per, path, per * q_len) ||
      overlap(new_lens, per, block_table, per * max_blocks_per_seq))
    return PKV_EINVAL;
  CommitParams p;
  std::memset(&p, 0, sizeof(p));
  p.k_cache = static_cast<uint8_t *>(k_cache);
  p.v_cache = static_cast<uint8_t *>(v_cache);
  if (cache_dtype == PKV_FP8_E4M3) {
    p.k_scale = k_scale;
    p.v_scale = v_scale;
  }
  p.path = path;
  p.path_len = path_len;
  p.block_table = block_table;
  p.context_lens = context_lens;
  p.tree_lens = tree_lens;
  p.new_lens = new_lens;
  p.num_blocks = num_blocks;
  p.B = B;
  p.n = q_len;
  p.Hkv = Hkv;
  p.max_blocks = max_blocks_per_seq;
  p.row_bytes = D * esize_of(cache_dtype);
  p.calibrated = calibrated ? 1 : 0;
  return cuda_status(launch_tree_commit(p, reinterpret_cast<cudaStream_t>(stream)));
}

int paged_tree_commit(void *k_cache, void *v_cache, int cache_dtype, const float *k_scale, const float *v_scale,
                      const int32_t *path, const int32_t *path_len, const int32_t *block_table,
                      int max_blocks_per_seq, const int32_t *context_lens, const int32_t *tree_lens,
                      int32_t *new_lens, int B, int q_len, int Hkv, int D, int64_t num_blocks, pkv_stream_t stream) {
  return run_commit(k_cache, v_cache, cache_dtype, const_cast<float *>(k_scale), const_cast<float *>(v_scale), path, path_len,
                    block_table, max_blocks_per_seq, context_lens, tree_lens, new_lens, B, q_len, Hkv, D, num_blocks, false,
                    stream);
}

int paged_tree_commit_calibrated(void *k_cache, void *v_cache, int cache_dtype, float *k_scale, float *v_scale,
                                 const int32_t *path, const int32_t *path_len, const int32_t *block_table,
                                 int max_blocks_per_seq, const int32_t *context_lens, const int32_t *tree_lens,
                                 int32_t *new_lens, int B, int q_len, int Hkv, int D, int64_t num_blocks,
                                 pkv_stream_t stream) {
  return run_commit(k_cache, v_cache, cache_dtype, k_scale, v_scale, path, path_len, block_table, max_blocks_per_seq,
                    context_lens, tree_lens, new_lens, B, q_len, Hkv, D, num_blocks, true, stream);
}

int paged_prefill_attention(void *out, const void *q, int q_dtype, const void *k_cache, const void *v_cache,
                            int cache_dtype, const int32_t *block_table, int max_blocks_per_seq,
                            const int32_t *context_lens, const int32_t *q_start, int B, int max_q_len, int Hq,
                            int Hkv, int D, int64_t num_blocks, float scale, int window, int32_t *status,
                            pkv_stream_t stream) {
  int rc = validate_decode_shapes(q_dtype, cache_dtype, B, 1, Hq, Hkv, D, num_blocks, max_blocks_per_seq);
  if (rc != PKV_OK) return rc;
  if (cache_dtype != PKV_F16 && cache_dtype != PKV_BF16) return PKV_EUNSUPPORTED;
  if (!(scale > 0.f) || !std::isfinite(scale) || window < 0 || max_q_len < 0) return PKV_EINVAL;
  if (B > 65535 || Hkv > 65535) return PKV_EUNSUPPORTED;
  const int G = Hq / Hkv;
  const int64_t tiles = ((int64_t)max_q_len * G + 127) / 128;
  if (tiles > INT32_MAX) return PKV_EUNSUPPORTED;
  if (B == 0 || tiles == 0) return PKV_OK;
  if (!out || !q || !k_cache || !v_cache || !block_table || !context_lens || !q_start) return PKV_EINVAL;
  if (!aligned16(out) || !aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache)) return PKV_EINVAL;
  CUtensorMap tmK, tmV;
  rc = cache_map(&tmK, k_cache, cache_dtype, num_blocks, Hkv, D);
  if (rc != PKV_OK) return rc;
  rc = cache_map(&tmV, v_cache, cache_dtype, num_blocks, Hkv, D);
  if (rc != PKV_OK) return rc;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (status) {
    cudaError_t e = cudaMemsetAsync(status, 0, sizeof(int32_t), s);
    if (e != cudaSuccess) return cuda_status(e);
  }
  PrefillParams p;
  std::memset(&p, 0, sizeof(p));
  p.out = out;
  p.q = q;
  p.block_table = block_table;
  p.context_lens = context_lens;
  p.q_start = q_start;
  p.status = status;
  p.num_blocks = num_blocks;
  p.B = B;
  p.Hq = Hq;
  p.Hkv = Hkv;
  p.D = D;
  p.G = G;
  p.max_blocks = max_blocks_per_seq;
  p.max_q_len = max_q_len;
  p.max_tiles = (int)tiles;
  p.window = window < (1 << 30) ? window : 0;
  p.scale_log2 = scale * 1.4426950408889634f;
  take_stall(p, PKV_STALL_PREFILL);
  return cuda_status(launch_prefill_auto(p, cache_dtype, tmK, tmV, s));
}

int paged_decode_status(const void *workspace, size_t workspace_bytes, pkv_stream_t stream, int *flags_out) {
  if (!workspace || workspace_bytes < sizeof(WsHeader)) return PKV_EWORKSPACE;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  WsHeader hdr;
  cudaError_t e = cudaMemcpyAsync(&hdr, workspace, sizeof(hdr), cudaMemcpyDeviceToHost, s);
  if (e == cudaSuccess) e = cudaStreamSynchronize(s);
  if (e != cudaSuccess) return cuda_status(e);
  int32_t status = hdr.status;
  if (status & kStatusPerCta) {
    const int n = std::min<int>(status & ~kStatusPerCta, sizeof(hdr.cta_status));
    status = 0;
    for (int i = 0; i < n; ++i) status |= hdr.cta_status[i];
  }
  if (flags_out) *flags_out = status;
  if (status & PKV_FLAG_TIMEOUT) return PKV_ETIMEOUT;
  if (status & (PKV_FLAG_BAD_LEN | PKV_FLAG_BAD_BLOCK | PKV_FLAG_RANGE)) return PKV_ERANGE;
  return PKV_OK;
}

int paged_decode_merge(void *out, int out_dtype, const float *o_partial, const float *lse, int B, int Hq, int D,
                       int S, pkv_stream_t stream) {
  if (B < 0 || Hq <= 0 || D <= 0 || S <= 0) return PKV_EINVAL;
  if (out_dtype != PKV_F32 && out_dtype != PKV_F16 && out_dtype != PKV_BF16) return PKV_EINVAL;
  if (B == 0) return PKV_OK;
  if (!out || !o_partial || !lse) return PKV_EINVAL;
  return cuda_status(launch_merge(out, out_dtype, o_partial, lse, B, Hq, D, S, reinterpret_cast<cudaStream_t>(stream)));
}

int paged_kv_copy_blocks(void *k_cache, void *v_cache, int cache_dtype, float *k_scale, float *v_scale,
                         const int32_t *src_dst_pairs, int n_pairs, int Hkv, int D, int64_t num_blocks,
                         pkv_stream_t stream) {
  if (n_pairs < 0 || Hkv <= 0 || num_blocks <= 0) return PKV_EINVAL;
  if (esize_of(cache_dtype) == 0) return PKV_EINVAL;
  if (D != 64 && D != 128) return PKV_EUNSUPPORTED;
  if (n_pairs == 0) return PKV_OK;
  if (!k_cache || !v_cache || !src_dst_pairs) return PKV_EINVAL;
  if (cache_dtype == PKV_FP8_E4M3 && (!k_scale || !v_scale)) return PKV_EINVAL;
  if (!aligned16(k_cache) || !aligned16(v_cache)) return PKV_EINVAL;
  return cuda_status(launch_copy_blocks(k_cache, v_cache, cache_dtype, k_scale, v_scale, src_dst_pairs, n_pairs,
                                        Hkv, D, num_blocks, reinterpret_cast<cudaStream_t>(stream)));
}

int pkv_copy(void *dst, const void *src, size_t bytes, pkv_stream_t stream) {
  if (bytes == 0) return PKV_OK;
  if (!dst || !src || (bytes & 15u) != 0 || !aligned16(dst) || !aligned16(src)) return PKV_EINVAL;
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return cuda_status(e);
  return cuda_status(launch_copy(dst, src, bytes, sms, reinterpret_cast<cudaStream_t>(stream)));
}

int paged_kv4_decode_workspace_bytes(int B, int q_len, int Hq, int Hkv, int D, int q_dtype, int num_splits,
                                     size_t *bytes_out) {
  if (!bytes_out) return PKV_EINVAL;
  if (q_dtype == PKV_F32) return PKV_EUNSUPPORTED;
  int rc = validate_decode_shapes(q_dtype, q_dtype, B, q_len, Hq, Hkv, D, 1, 1);
  if (rc != PKV_OK) return rc;
  Choice c;
  int P = 0;
  rc = plan_kv4(q_dtype, q_len, Hq, Hkv, D, num_splits, &c, &P);
  if (rc != PKV_OK) return rc;
  *bytes_out = kv4_ws_layout(B, P, D, c.GC, kv4_heads(Hkv), registry().kv4[c.ki].warps).total;
  return PKV_OK;
}

int paged_kv4_decode_attention(void *out, const void *q, int q_dtype, const void *cache, const int32_t *block_table,
                               int max_blocks_per_seq, const int32_t *context_lens, int B, int q_len, int window,
                               int Hq, int Hkv, int D, int64_t num_blocks, float scale, float k_unit, float v_unit,
                               int num_splits, void *workspace, size_t workspace_bytes, pkv_stream_t stream) {
  if (q_dtype == PKV_F32) return PKV_EUNSUPPORTED;
  int rc = validate_decode_shapes(q_dtype, q_dtype, B, q_len, Hq, Hkv, D, num_blocks, max_blocks_per_seq);
  if (rc != PKV_OK) return rc;
  if (window < 0 || !kv4_unit_ok(k_unit) || !kv4_unit_ok(v_unit)) return PKV_EINVAL;
  const float s = scale * k_unit;
  if (!std::isfinite(scale) || !std::isfinite(s * 1.4426950408889634f)) return PKV_EINVAL;
  if (B == 0) return PKV_OK;
  if (!out || !q || !cache || !block_table || !context_lens) return PKV_EINVAL;
  if (!aligned16(out) || !aligned16(q) || !aligned16(cache)) return PKV_EINVAL;
  Choice c;
  int P = 0;
  rc = plan_kv4(q_dtype, q_len, Hq, Hkv, D, num_splits, &c, &P);
  if (rc != PKV_OK) return rc;
  const Kv4Kernel &k = registry().kv4[c.ki];
  const Kv4WsLayout L = kv4_ws_layout(B, P, D, c.GC, kv4_heads(Hkv), k.warps);
  if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255u) != 0 || workspace_bytes < L.total)
    return PKV_EWORKSPACE;
  int ctas = 0, sms = 0;
  rc = occupancy(kMaxKernels + c.ki, k.fn, k.threads, k.smem_bytes, &ctas, &sms);  // opts into its shared memory
  if (rc != PKV_OK) return rc;
  uint8_t *ws = static_cast<uint8_t *>(workspace);
  Kv4Params p;
  p.d = unit_params(c, P, out, q, q_dtype, nullptr, nullptr, block_table, max_blocks_per_seq, context_lens, B, q_len,
                    window, Hq, Hkv, D, num_blocks, s, workspace);
  p.d.hdr = reinterpret_cast<WsHeader *>(ws + L.hdr);
  p.d.prefix = reinterpret_cast<int32_t *>(ws + L.prefix);
  p.d.starts = reinterpret_cast<int4 *>(ws + L.starts);
  p.d.part_o = reinterpret_cast<float *>(ws + L.part_o);
  p.d.part_lse = reinterpret_cast<float *>(ws + L.part_lse);
  p.d.cta_flags = nullptr;
  p.d.n_ctas = P;
  p.d.inline_plan = B + 1 <= kKv4Prefix ? 1 : 0;
  p.cache = static_cast<const uint8_t *>(cache);
  // the most blocks that a unit reads
  const int64_t most = window > 0 ? std::min((int64_t)max_blocks_per_seq, ((int64_t)window + q_len + 14) / kBlock + 1)
                                  : max_blocks_per_seq;
  // Heads a unit takes together.  Short tables' units are not cut between CTAs: two heads where that spreads few units
  // over more rings (us a call, 4 / 2 heads: 1 x 333 12.3 / 11.0, 1 x 700 17.0 / 13.3, 1 x 333 with 4 new tokens
  // 16.8 / 13.1; but for a few blocks, 1 x 100 9.6 / 11.5).
  p.hg = kv4_heads(Hkv);
  if (p.hg == 4 && most > 12 && most <= kv4_whole(D) && (int64_t)B * (Hkv / 4) * c.NC < P) p.hg = 2;
  p.hg_log2 = p.hg / 2;  // (of 1, 2 and 4)
  p.d.HU = Hkv / p.hg * c.NC;
  p.records = reinterpret_cast<int4 *>(ws + L.records);
  p.first_o = reinterpret_cast<float *>(ws + L.first_o);
  p.v_unit = v_unit;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  void *args[1] = {&p};
  cudaError_t e = launch_units(k.fn, k.threads, k.smem_bytes, p.d, args, st);
  // units of no more blocks: none is cut between CTAs
  if (e == cudaSuccess && most > kv4_whole(D) && P > 1) e = launch_kv4_merge(p, st, st != nullptr);
  return cuda_status(e);
}

}  // extern "C"
