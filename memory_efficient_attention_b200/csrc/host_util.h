// host_util.h — host-side helpers shared by the translation units of libmea: device attributes,
// TMA descriptor encoding (with its cache), one-time kernel attributes and the split-KV layout.
// Inline, so that all units share one timeout, one device table and one descriptor cache.
#pragma once

#include <cudaTypedefs.h>
#include <cuda.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>
#include <mutex>

#include "../../include/mea.h"

namespace mea_host {

inline std::atomic<unsigned long long> g_timeout_ns{2000000000ull};

struct DeviceInfo {
  bool init = false;
  bool ok = false;
  int sms = 0;
};
constexpr int kMaxDevices = 64;
inline DeviceInfo g_dev[kMaxDevices];
inline std::mutex g_dev_mu;

inline int current_device_info(DeviceInfo& out) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return MEA_ERR_CUDA;
  std::lock_guard<std::mutex> lk(g_dev_mu);
  DeviceInfo& d = g_dev[dev];
  if (!d.init) {
    int major = 0, sms = 0;
    if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
      return MEA_ERR_CUDA;
    d.ok = (major == 10);
    d.sms = sms;
    d.init = true;
  }
  out = d;
  return d.ok ? MEA_OK : MEA_ERR_DEVICE;
}

inline PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
    void* ptr = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &ptr, cudaEnableDefault, &q) !=
            cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      return static_cast<PFN_cuTensorMapEncodeTiled_v12000>(nullptr);
    return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(ptr);
  }();
  return fn;
}

// 3-D tiled map over a row-major [d2, d1, d0] tensor of 16-bit elements, 128-byte swizzle.
constexpr int kDtypeE4M3 = 2;  // internal: 8-bit e4m3 tensor (mea_forward_fp8)

inline bool encode_3d_uncached(CUtensorMap* map, const void* base, int dtype, uint64_t d0,
                        uint64_t d1, uint64_t d2, uint32_t b0, uint32_t b1, uint32_t b2) {
  auto fn = encode_fn();
  if (!fn) return false;
  const uint64_t es = dtype == kDtypeE4M3 ? 1 : 2;
  cuuint64_t dims[3] = {d0, d1, d2};
  cuuint64_t strides[2] = {d0 * es, d0 * d1 * es};
  cuuint32_t box[3] = {b0, b1, b2};
  cuuint32_t estr[3] = {1, 1, 1};
  CUresult r = fn(map, dtype == kDtypeE4M3 ? CU_TENSOR_MAP_DATA_TYPE_UINT8
                       : dtype == MEA_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                           : CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
                  3, const_cast<void*>(base), dims, strides, box, estr,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS;
}

// ------------------------------------------------------------------------------------------
// Cache of encoded tensor maps. A map only describes (address, sizes, strides, box, element
// type, swizzle), so one encoded for the same arguments is the same 128 bytes; serving calls
// that reuse their buffers (every decode step of a KV cache, for instance) skip the encoding.
// The cache is the library's only state besides per-device attributes: kMapCache entries,
// least recently used replaced first, guarded by a mutex.
// ------------------------------------------------------------------------------------------
struct MapKey {
  const void* base;
  int dtype, rank;
  uint64_t dims[5];
  uint32_t box[5];
  bool operator==(const MapKey& o) const {
    if (base != o.base || dtype != o.dtype || rank != o.rank) return false;
    for (int i = 0; i < 5; ++i)
      if (dims[i] != o.dims[i] || box[i] != o.box[i]) return false;
    return true;
  }
};
constexpr int kMapCache = 64;
struct MapCache {
  MapKey key[kMapCache];
  CUtensorMap map[kMapCache];
  uint64_t used[kMapCache] = {};  // 0 = empty slot
  uint64_t tick = 0;
  std::mutex mu;
};
inline MapCache g_maps;

// Copies the cached map for `k` into *out; false when it is not cached.
inline bool map_lookup(const MapKey& k, CUtensorMap* out) {
  std::lock_guard<std::mutex> lk(g_maps.mu);
  for (int i = 0; i < kMapCache; ++i)
    if (g_maps.used[i] && g_maps.key[i] == k) {
      g_maps.used[i] = ++g_maps.tick;
      *out = g_maps.map[i];
      return true;
    }
  return false;
}

inline void map_insert(const MapKey& k, const CUtensorMap& m) {
  std::lock_guard<std::mutex> lk(g_maps.mu);
  int victim = 0;
  for (int i = 0; i < kMapCache; ++i) {
    if (g_maps.used[i] == 0) {
      victim = i;
      break;
    }
    if (g_maps.used[i] < g_maps.used[victim]) victim = i;
  }
  g_maps.key[victim] = k;
  g_maps.map[victim] = m;
  g_maps.used[victim] = ++g_maps.tick;
}

inline bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// cudaFuncSetAttribute(max dynamic shared memory) once per (kernel, device); the result of that
// one call is kept and returned on every later call, so a failure is never forgotten. The kernel
// is a template argument so that every kernel (not every kernel signature) has its own state.
template <auto kern>
cudaError_t smem_attr_once(uint32_t smem) {
  static std::once_flag once[kMaxDevices];
  static cudaError_t result[kMaxDevices];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices)
    return cudaErrorInvalidDevice;
  std::call_once(once[dev], [&] {
    result[dev] = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  });
  return result[dev];
}

// Drops a launch error left by an earlier, unrelated call, so that the check after this
// call's launches reports only their own failures.
inline void clear_stale_launch_error() { (void)cudaGetLastError(); }

// Launches `kern` as the dependent of the stream's previous kernel: it may start before that one
// has ended and calls pdl_wait before it touches anything that one reads or writes. What that one
// writes is read by ld_after_wait or a plain load, never by __ldg, which stays for buffers that were
// complete before that one was launched.
template <class... Params, class... Args>
cudaError_t launch_dependent(void (*kern)(Params...), dim3 grid, dim3 block, size_t smem,
                             cudaStream_t stream, Args&&... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, static_cast<Params>(args)...);
}

// 3-D / 4-D maps through the cache (same arguments as the uncached encoders).
inline bool encode_3d(CUtensorMap* map, const void* base, int dtype, uint64_t d0, uint64_t d1,
               uint64_t d2, uint32_t b0, uint32_t b1, uint32_t b2) {
  const MapKey k{base, dtype, 3, {d0, d1, d2, 0}, {b0, b1, b2, 0}};
  if (map_lookup(k, map)) return true;
  if (!encode_3d_uncached(map, base, dtype, d0, d1, d2, b0, b1, b2)) return false;
  map_insert(k, *map);
  return true;
}

// 4-D tiled map over a paged cache [d3 blocks, d2 slots, d1 heads, d0] of 16-bit elements.
inline bool encode_4d_uncached(CUtensorMap* map, const void* base, int dtype, uint64_t d0,
                        uint64_t d1, uint64_t d2, uint64_t d3, uint32_t b0, uint32_t b1,
                        uint32_t b2, uint32_t b3) {
  auto fn = encode_fn();
  if (!fn) return false;
  cuuint64_t dims[4] = {d0, d1, d2, d3};
  cuuint64_t strides[3] = {d0 * 2, d0 * d1 * 2, d0 * d1 * d2 * 2};
  cuuint32_t box[4] = {b0, b1, b2, b3};
  cuuint32_t estr[4] = {1, 1, 1, 1};
  CUresult r = fn(map, dtype == MEA_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                         : CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
                  4, const_cast<void*>(base), dims, strides, box, estr,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS;
}

inline bool encode_4d(CUtensorMap* map, const void* base, int dtype, uint64_t d0, uint64_t d1,
               uint64_t d2, uint64_t d3, uint32_t b0, uint32_t b1, uint32_t b2, uint32_t b3) {
  const MapKey k{base, dtype, 4, {d0, d1, d2, d3}, {b0, b1, b2, b3}};
  if (map_lookup(k, map)) return true;
  if (!encode_4d_uncached(map, base, dtype, d0, d1, d2, d3, b0, b1, b2, b3)) return false;
  map_insert(k, *map);
  return true;
}

// 5-D tiled map over a paged cache [blocks, slots, heads, head_dim] of 16-bit elements with
// head_dim = 64 * atoms, seen as (64 columns, slot, atom, head, block): one box {64, rows, atoms,
// 1, 1} brings `rows` slots of one head and block with every 64-column atom, landing as
// [atom][rows][128 B] (the 128-byte swizzle per 128-byte row).
inline bool encode_paged5(CUtensorMap* map, const void* base, int dtype, uint64_t head_dim,
                   uint64_t heads, uint64_t slots, uint64_t blocks, uint32_t rows) {
  const uint64_t atoms = head_dim / 64;
  const MapKey k{base, dtype, 5, {64, slots, atoms, heads, blocks}, {64, rows, uint32_t(atoms), 1, 1}};
  if (map_lookup(k, map)) return true;
  auto fn = encode_fn();
  if (!fn) return false;
  cuuint64_t dims[5] = {64, slots, atoms, heads, blocks};
  cuuint64_t strides[4] = {heads * head_dim * 2, 128, head_dim * 2, slots * heads * head_dim * 2};
  cuuint32_t box[5] = {64, rows, static_cast<cuuint32_t>(atoms), 1, 1};
  cuuint32_t estr[5] = {1, 1, 1, 1, 1};
  CUresult r = fn(map, dtype == MEA_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                         : CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
                  5, const_cast<void*>(base), dims, strides, box, estr,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return false;
  map_insert(k, *map);
  return true;
}

// Keys per chunk when the caller leaves it to the library: the largest power of two from 128 to
// 2048 that still gives about half a work item (chunk, head block) per SM or more. Every item
// costs a fixed ~1.4 us (its four warps' merge and partial write) beside streaming its keys, so
// few long items beat many short ones: on 64 requests of U[512, 32768] keys 2048-key chunks
// stream at the HBM copy rate where 1024 reach 0.95 of it, and one 32768-key request is 3.4x
// faster at 2048 than at 128, although 2048 leaves 20 of 148 SMs without an item.
inline int auto_split_keys(int total_k, int n_hb, int sms) {
  long long work = static_cast<long long>(total_k) * n_hb;
  long long target = 2 * work / static_cast<long long>(sms > 0 ? sms : 148);
  int c = 128;
  while (c < 2048 && c * 2 <= target) c *= 2;
  return c;
}

inline int decode_rb(int R) {
  int rb = 1;
  for (int d = 1; d <= 16; ++d)
    if (R % d == 0) rb = d;
  return rb;
}

inline size_t align_up(size_t x, size_t a) { return (x + a - 1) / a * a; }

struct DecLayout {
  int chunk = 0, n_slots = 0;
  size_t o_bytes = 0, lse_off = 0, total = 0;
};

// Head dims of the decode: a multiple of 8 from 8 to 256; the kernels run 64, 128 or 256 wide.
inline bool dec_head_dim_ok(int d) { return d >= 8 && d <= 256 && d % 8 == 0; }
inline int padded_head_dim(int d) { return d <= 64 ? 64 : d <= 128 ? 128 : 256; }

inline bool dec_layout(int n_seqs, int total_k, int hq, int hkv, int d, int split_keys, int sms,
                DecLayout& L) {
  if (n_seqs < 1 || total_k < 0 || hq < 1 || hkv < 1 || hq % hkv || !dec_head_dim_ok(d))
    return false;
  d = padded_head_dim(d);  // the partials are kept at the kernel's width
  if (split_keys < 0 || split_keys % 64) return false;
  const int R = hq / hkv;
  const int n_hb = hq / decode_rb(R);
  L.chunk = split_keys ? split_keys : auto_split_keys(total_k, n_hb, sms);
  const long long slots = (static_cast<long long>(total_k) + L.chunk - 1) / L.chunk + n_seqs;
  if (slots > (1ll << 30)) return false;
  L.n_slots = static_cast<int>(slots);
  L.o_bytes = static_cast<size_t>(slots) * hq * d * sizeof(float);
  L.lse_off = align_up(L.o_bytes, 256);
  L.total = L.lse_off + align_up(static_cast<size_t>(slots) * hq * sizeof(float), 256);
  return true;
}

}  // namespace mea_host
