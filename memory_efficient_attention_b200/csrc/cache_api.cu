// cache_api.cu — C ABI of the operators on a paged K/V cache (declared in include/mea.h): the
// blocks' key ranges, block choice and the decode over chosen blocks, the decode that also gives
// the keys' attention weights, and eviction. Argument checks, TMA descriptors and launches; no
// device memory is allocated and no call synchronises the host.
#include <cuda.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "../../include/mea.h"
#include "cache_sm100.cuh"
#include "decode_sm100.cuh"
#include "host_util.h"

using namespace mea_host;

namespace mea_cache {
// This translation unit's device error word (see mea_device_error).
__attribute__((visibility("hidden"))) int device_error(unsigned int* code, bool clear) {
  if (cudaMemcpyFromSymbol(code, mea::g_mea_error, sizeof(*code)) != cudaSuccess)
    return MEA_ERR_CUDA;
  const unsigned int z = 0;
  if (clear && cudaMemcpyToSymbol(mea::g_mea_error, &z, sizeof(z)) != cudaSuccess)
    return MEA_ERR_CUDA;
  return MEA_OK;
}
}  // namespace mea_cache

namespace {

// Whether two buffers of 32-bit elements share a byte.
bool overlap(const void* a, long long na, const void* b, long long nb) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x < y + 4 * static_cast<uintptr_t>(nb) && y < x + 4 * static_cast<uintptr_t>(na);
}

bool block_size_ok(int bs) { return bs == 16 || bs == 32 || (bs >= 64 && bs % 64 == 0); }

// The checks that every operator on the cache shares, in the order of the statuses' documentation.
int check_cache(int n_seqs, int num_blocks, int block_size, int max_blocks, int n_heads_kv,
                int head_dim, int dtype) {
  if (n_seqs < 1 || num_blocks < 1 || max_blocks < 1 || !block_size_ok(block_size))
    return MEA_ERR_SHAPE;
  if (n_heads_kv < 1) return MEA_ERR_HEADS;
  if (!dec_head_dim_ok(head_dim)) return MEA_ERR_HEAD_DIM;
  if (dtype != MEA_F16 && dtype != MEA_BF16) return MEA_ERR_DTYPE;
  return MEA_OK;
}

// K and V maps of a paged cache for the decode's split kernel (boxes of one block's rows).
bool decode_maps(CUtensorMap* tk, CUtensorMap* tv, const void* k, const void* v, int dtype,
                 int head_dim, int n_heads_kv, int block_size, int num_blocks,
                 mea::DecParams& p) {
  const uint32_t rows = block_size < 64 ? static_cast<uint32_t>(block_size) : 64u;
  p.box5 = (head_dim == 64 || head_dim == 128 || head_dim == 256) ? 1 : 0;
  p.lay_log2 = p.box5 ? (rows == 16 ? 4 : rows == 32 ? 5 : 6) : 6;
  if (p.box5)
    return encode_paged5(tk, k, dtype, head_dim, n_heads_kv, block_size, num_blocks, rows) &&
           encode_paged5(tv, v, dtype, head_dim, n_heads_kv, block_size, num_blocks, rows);
  return encode_4d(tk, k, dtype, head_dim, n_heads_kv, block_size, num_blocks, 64, 1, rows, 1) &&
         encode_4d(tv, v, dtype, head_dim, n_heads_kv, block_size, num_blocks, 64, 1, rows, 1);
}

// The split kernel and what completes it. max_seqlen_k sizes the grid of the weights (DEC_WEIGHTS).
template <int D, bool BF16, bool ALIBI, int MODE>
int launch_split(const CUtensorMap& tk, const CUtensorMap& tv, const mea::DecParams& p, int grid,
                 int max_seqlen_k, cudaStream_t stream) {
  constexpr auto kern = mea::mea_decode_split_kernel<D, BF16, ALIBI, true, MODE>;
  constexpr uint32_t smem = mea::DecCfg<D, true>::SMEM_TOTAL;
  constexpr int threads = mea::DecCfg<D, true>::THREADS;
  if (smem_attr_once<kern>(smem) != cudaSuccess) return MEA_ERR_CUDA;
  clear_stale_launch_error();
  if constexpr (MODE == mea::DEC_SELECTED) {
    if (launch_dependent(kern, grid, threads, smem, stream, tk, tv, p) != cudaSuccess)
      return MEA_ERR_CUDA;
    if (grid > 1 && launch_dependent(mea::mea_selected_merge_kernel<D, BF16>, grid - 1, 256, 0,
                                     stream, p, grid) != cudaSuccess)
      return MEA_ERR_CUDA;
    return MEA_OK;
  } else {
    const dim3 wgrid(1 + (max_seqlen_k + 1023) / 1024, p.hq / p.R, p.n_seqs);
    if (grid == 0) {  // no keys at all: nothing of ours runs before the merge
      mea::mea_decode_weights_kernel<D, BF16><<<wgrid, 256, 0, stream>>>(p);
      return cudaGetLastError() == cudaSuccess ? MEA_OK : MEA_ERR_CUDA;
    }
    kern<<<grid, threads, smem, stream>>>(tk, tv, p);
    if (cudaGetLastError() != cudaSuccess) return MEA_ERR_CUDA;
    return launch_dependent(mea::mea_decode_weights_kernel<D, BF16>, wgrid, 256, 0, stream, p) ==
                   cudaSuccess
               ? MEA_OK
               : MEA_ERR_CUDA;
  }
}

template <int MODE>
int launch_split_any(int head_dim, int dtype, const CUtensorMap& tk, const CUtensorMap& tv,
                     const mea::DecParams& p, int grid, int max_k, cudaStream_t s) {
  const bool bf = dtype == MEA_BF16, al = p.slopes != nullptr;
#define MEA_SPLIT(DD)                                                                     \
  return bf ? (al ? launch_split<DD, true, true, MODE>(tk, tv, p, grid, max_k, s)                \
                  : launch_split<DD, true, false, MODE>(tk, tv, p, grid, max_k, s))              \
            : (al ? launch_split<DD, false, true, MODE>(tk, tv, p, grid, max_k, s)               \
                  : launch_split<DD, false, false, MODE>(tk, tv, p, grid, max_k, s))
  if (head_dim > 128) MEA_SPLIT(256);
  if (head_dim > 64) MEA_SPLIT(128);
  MEA_SPLIT(64);
#undef MEA_SPLIT
}

void fill_decode(mea::DecParams& p, const void* q, void* out, float* lse, const int32_t* cu_k,
                 const int32_t* block_table, const float* slopes, int n_seqs, int num_blocks,
                 int block_size, int max_blocks, int hq, int hkv, int head_dim, float scale) {
  p.q = q;
  p.out = out;
  p.lse = lse;
  p.cu_k = cu_k;
  p.slopes = slopes;
  p.block_table = block_table;
  p.block_size = block_size;
  p.max_blocks = max_blocks;
  p.num_blocks = num_blocks;
  p.n_seqs = n_seqs;
  p.hq = hq;
  p.dh = head_dim;
  p.R = hq / hkv;
  p.RB = decode_rb(p.R);
  p.n_hb = hq / p.RB;
  p.c1 = scale * 1.4426950408889634f;
  p.timeout_ns = g_timeout_ns.load();
}

// Decode over chosen blocks: two partial ranges per CTA, the heads of one item each.
size_t selected_ws_lse(int hq, int hkv, int d, int sms) {
  return align_up(2 * static_cast<size_t>(sms) * decode_rb(hq / hkv) * padded_head_dim(d) *
                      sizeof(float), 256);
}
size_t selected_ws(int hq, int hkv, int d, int sms) {
  return selected_ws_lse(hq, hkv, d, sms) +
         align_up(2 * static_cast<size_t>(sms) * decode_rb(hq / hkv) * sizeof(float), 256);
}

}  // namespace

extern "C" {

int mea_block_key_bounds(const void* k_cache, const int32_t* block_table,
                         const int32_t* cu_seqlens_k, const int32_t* first_key, void* bounds,
                         int n_seqs, int num_blocks, int block_size, int max_blocks,
                         int max_seqlen_k, int n_heads_kv, int head_dim, int dtype,
                         void* stream) {
  if (!k_cache || !block_table || !cu_seqlens_k || !bounds) return MEA_ERR_NULL;
  if (int rc = check_cache(n_seqs, num_blocks, block_size, max_blocks, n_heads_kv, head_dim, dtype))
    return rc;
  if (n_seqs > 65535 || max_seqlen_k < 0 ||
      static_cast<long long>(max_blocks) * block_size < max_seqlen_k)
    return MEA_ERR_SHAPE;
  if (!aligned(k_cache, 16) || !aligned(bounds, 16) || !aligned(block_table, 4) ||
      !aligned(cu_seqlens_k, 4) || (first_key && !aligned(first_key, 4)))
    return MEA_ERR_ALIGN;
  DeviceInfo di;
  if (int rc = current_device_info(di); rc != MEA_OK) return rc;
  if (max_seqlen_k == 0) return MEA_OK;
  mea::BoundsParams p{};
  p.k = k_cache;
  p.bounds = bounds;
  p.block_table = block_table;
  p.cu_k = cu_seqlens_k;
  p.first_key = first_key;
  p.num_blocks = num_blocks;
  p.block_size = block_size;
  p.max_blocks = max_blocks;
  p.hkv = n_heads_kv;
  p.dh = head_dim;
  // One unit (16 bytes of a block's rows) per thread over the longest request. With first_key few
  // of a request's blocks change as a rule, and CTAs without one only cost their launch: then the
  // grid is held to about two per SM and the threads walk.
  const long long units = (static_cast<long long>(max_seqlen_k) + block_size - 1) / block_size *
                          (static_cast<long long>(n_heads_kv) * head_dim / 8);
  long long gx = (units + 255) / 256;
  const long long cap = first_key ? (2ll * di.sms + n_seqs - 1) / n_seqs : 0x7fffffffll;
  if (gx > cap) gx = cap;
  const dim3 grid(static_cast<unsigned>(gx), static_cast<unsigned>(n_seqs));
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  clear_stale_launch_error();
  if (dtype == MEA_BF16)
    mea::mea_key_bounds_kernel<true><<<grid, 256, 0, s>>>(p);
  else
    mea::mea_key_bounds_kernel<false><<<grid, 256, 0, s>>>(p);
  return cudaGetLastError() == cudaSuccess ? MEA_OK : MEA_ERR_CUDA;
}

int mea_select_blocks(const void* q, const void* bounds, const int32_t* block_table,
                      const int32_t* cu_seqlens_k, int32_t* selected, int n_seqs, int num_blocks,
                      int block_size, int max_blocks, int max_seqlen_k, int n_heads_q,
                      int n_heads_kv, int head_dim, int n_select, int n_first, int n_last,
                      int dtype, void* stream) {
  if (!q || !bounds || !block_table || !cu_seqlens_k || !selected) return MEA_ERR_NULL;
  if (int rc = check_cache(n_seqs, num_blocks, block_size, max_blocks, n_heads_kv, head_dim, dtype))
    return rc;
  if (n_heads_q < 1 || n_heads_q % n_heads_kv != 0) return MEA_ERR_HEADS;
  const long long live = (static_cast<long long>(max_seqlen_k) + block_size - 1) / block_size;
  if (max_seqlen_k < 0 || live > max_blocks || live > MEA_SELECT_MAX_BLOCKS || n_select < 1 ||
      n_first < 0 || n_last < 0 ||
      static_cast<long long>(n_seqs) * n_heads_kv * 8 > 0x7fffffffll)
    return MEA_ERR_SHAPE;
  if (!aligned(q, 16) || !aligned(bounds, 16) || !aligned(block_table, 4) ||
      !aligned(cu_seqlens_k, 4) || !aligned(selected, 4))
    return MEA_ERR_ALIGN;
  DeviceInfo di;
  if (int rc = current_device_info(di); rc != MEA_OK) return rc;
  mea::SelectParams p{};
  p.q = q;
  p.bounds = bounds;
  p.block_table = block_table;
  p.cu_k = cu_seqlens_k;
  p.selected = selected;
  p.num_blocks = num_blocks;
  p.block_size = block_size;
  p.max_blocks = max_blocks;
  p.hq = n_heads_q;
  p.hkv = n_heads_kv;
  p.dh = head_dim;
  p.n_select = n_select;
  p.n_first = n_first;
  p.n_last = n_last;
  p.n_seqs = n_seqs;
  p.max_live = static_cast<int>(live);
  p.longest_first = n_seqs > 1 && n_seqs <= mea::kRankedSeqs && live >= 256;
  // CTAs per (request, head): as many as fill the SMs about twice, and no more than have a round of
  // 128 blocks to score.
  const long long pairs = static_cast<long long>(n_seqs) * n_heads_kv;
  int cs = 1;
  while (cs < 8 && pairs * cs <= di.sms && live > 128ll * cs) cs *= 2;
  constexpr uint32_t max_smem = MEA_SELECT_MAX_BLOCKS * 4u;
  const uint32_t smem = static_cast<uint32_t>(live > 0 ? live : 1) * 4u;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(pairs * cs));
  cfg.blockDim = dim3(mea::kSelThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = static_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = static_cast<unsigned>(cs);
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  auto go = [&](auto tag, auto chunks) {
    constexpr auto kern = mea::mea_select_blocks_kernel<decltype(tag)::value,
                                                        decltype(chunks)::value>;
    if (smem_attr_once<kern>(max_smem) != cudaSuccess) return MEA_ERR_CUDA;
    clear_stale_launch_error();
    return cudaLaunchKernelEx(&cfg, kern, p) == cudaSuccess ? MEA_OK : MEA_ERR_CUDA;
  };
  using C4 = std::integral_constant<int, 4>;
  using C8 = std::integral_constant<int, 8>;
  using C16 = std::integral_constant<int, 16>;
  if (dtype == MEA_BF16)
    return head_dim > 128  ? go(std::true_type{}, C16{})
           : head_dim > 64 ? go(std::true_type{}, C8{})
                           : go(std::true_type{}, C4{});
  return head_dim > 128  ? go(std::false_type{}, C16{})
         : head_dim > 64 ? go(std::false_type{}, C8{})
                         : go(std::false_type{}, C4{});
}

size_t mea_decode_selected_workspace_size(int n_seqs, int n_select, int block_size, int n_heads_q,
                                          int n_heads_kv, int head_dim) {
  if (n_seqs < 1 || n_select < 1 || !block_size_ok(block_size) || n_heads_q < 1 ||
      n_heads_kv < 1 || n_heads_q % n_heads_kv || !dec_head_dim_ok(head_dim))
    return 0;
  DeviceInfo di;
  return selected_ws(n_heads_q, n_heads_kv, head_dim,
                     current_device_info(di) == MEA_OK ? di.sms : 148);
}

int mea_decode_selected(const void* q, const void* k_cache, const void* v_cache,
                        const int32_t* block_table, const int32_t* cu_seqlens_k,
                        const int32_t* selected, void* out, float* lse, int n_seqs, int num_blocks,
                        int block_size, int max_blocks, int n_select, int n_heads_q,
                        int n_heads_kv, int head_dim, float scale, const float* alibi_slopes,
                        int dtype, void* workspace, size_t workspace_bytes, void* stream) {
  if (!q || !k_cache || !v_cache || !block_table || !cu_seqlens_k || !selected || !out)
    return MEA_ERR_NULL;
  if (int rc = check_cache(n_seqs, num_blocks, block_size, max_blocks, n_heads_kv, head_dim, dtype))
    return rc;
  if (n_heads_q < 1 || n_heads_q % n_heads_kv != 0) return MEA_ERR_HEADS;
  const long long keys = static_cast<long long>(n_select) * block_size;
  if (n_select < 1 || keys > (1ll << 30)) return MEA_ERR_SHAPE;
  if (!std::isfinite(scale)) return MEA_ERR_SCALE;
  if (!aligned(q, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(out, 16) ||
      (lse && !aligned(lse, 4)) || !aligned(cu_seqlens_k, 4) || !aligned(block_table, 4) ||
      !aligned(selected, 4) || (alibi_slopes && !aligned(alibi_slopes, 4)))
    return MEA_ERR_ALIGN;
  if (!workspace || !aligned(workspace, 256)) return MEA_ERR_WORKSPACE;
  DeviceInfo di;
  if (int rc = current_device_info(di); rc != MEA_OK) return rc;
  if (workspace_bytes < selected_ws(n_heads_q, n_heads_kv, head_dim, di.sms))
    return MEA_ERR_WORKSPACE;
  mea::DecParams p{};
  fill_decode(p, q, out, lse, cu_seqlens_k, block_table, alibi_slopes, n_seqs, num_blocks,
              block_size, max_blocks, n_heads_q, n_heads_kv, head_dim, scale);
  p.selected = selected;
  p.n_select = n_select;
  p.item_tiles = static_cast<int>((keys + 63) / 64);
  p.n_items = static_cast<long long>(n_seqs) * p.n_hb;
  p.ws_o = static_cast<float*>(workspace);
  p.ws_lse = reinterpret_cast<float*>(static_cast<char*>(workspace) +
                                      selected_ws_lse(n_heads_q, n_heads_kv, head_dim, di.sms));
  CUtensorMap tk, tv;
  if (!decode_maps(&tk, &tv, k_cache, v_cache, dtype, head_dim, n_heads_kv, block_size, num_blocks,
                   p))
    return MEA_ERR_CUDA;
  // At least two tiles a CTA: a CTA costs about as much as streaming two.
  const long long half = (p.n_items * p.item_tiles + 1) / 2;
  const int grid = static_cast<int>(half < di.sms ? half : di.sms);
  return launch_split_any<mea::DEC_SELECTED>(head_dim, dtype, tk, tv, p, grid, 0,
                                             static_cast<cudaStream_t>(stream));
}

size_t mea_decode_weights_workspace_size(int n_seqs, int total_k, int n_heads_q, int n_heads_kv,
                                         int head_dim, int split_keys) {
  DeviceInfo di;
  const int sms = (current_device_info(di) == MEA_OK) ? di.sms : 148;
  DecLayout L;
  if (!dec_layout(n_seqs, total_k, n_heads_q, n_heads_kv, head_dim, split_keys, sms, L)) return 0;
  return L.total + static_cast<size_t>(L.n_slots) * n_heads_q * L.chunk * sizeof(float);
}

int mea_decode_weights(const void* q, const void* k_cache, const void* v_cache,
                       const int32_t* block_table, const int32_t* cu_seqlens_k, void* out,
                       float* lse, float* weights, const float* prev_weights,
                       long long weights_stride, int n_seqs, int num_blocks, int block_size,
                       int max_blocks, int total_k, int max_seqlen_k, int n_heads_q,
                       int n_heads_kv, int head_dim, float scale, const float* alibi_slopes,
                       int dtype, void* workspace, size_t workspace_bytes, int split_keys,
                       void* stream) {
  if (!q || !k_cache || !v_cache || !block_table || !cu_seqlens_k || !out ||
      (max_seqlen_k > 0 && !weights))
    return MEA_ERR_NULL;
  if (int rc = check_cache(n_seqs, num_blocks, block_size, max_blocks, n_heads_kv, head_dim, dtype))
    return rc;
  if (n_heads_q < 1 || n_heads_q % n_heads_kv != 0) return MEA_ERR_HEADS;
  if (n_seqs > 65535 || n_heads_kv > 65535 || total_k < 0 || max_seqlen_k < 0 ||
      max_seqlen_k > total_k || weights_stride < max_seqlen_k ||
      static_cast<long long>(max_blocks) * block_size < max_seqlen_k || split_keys < 0 ||
      split_keys % 64)
    return MEA_ERR_SHAPE;
  if (!std::isfinite(scale)) return MEA_ERR_SCALE;
  if (!aligned(q, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(out, 16) ||
      (lse && !aligned(lse, 4)) || !aligned(cu_seqlens_k, 4) || !aligned(block_table, 4) ||
      !aligned(weights, 4) || (prev_weights && !aligned(prev_weights, 4)) ||
      (alibi_slopes && !aligned(alibi_slopes, 4)))
    return MEA_ERR_ALIGN;
  // (The same tensor is read and written element by element; a shifted one would be read too late.)
  const long long n_weights = static_cast<long long>(n_seqs) * n_heads_kv * weights_stride;
  if (prev_weights && prev_weights != weights &&
      overlap(prev_weights, n_weights, weights, n_weights))
    return MEA_ERR_SHAPE;
  if (!workspace || !aligned(workspace, 256)) return MEA_ERR_WORKSPACE;
  DeviceInfo di;
  if (int rc = current_device_info(di); rc != MEA_OK) return rc;
  DecLayout L;
  if (!dec_layout(n_seqs, total_k, n_heads_q, n_heads_kv, head_dim, split_keys, di.sms, L))
    return MEA_ERR_SHAPE;
  const size_t need =
      L.total + static_cast<size_t>(L.n_slots) * n_heads_q * L.chunk * sizeof(float);
  if (workspace_bytes < need) return MEA_ERR_WORKSPACE;
  mea::DecParams p{};
  fill_decode(p, q, out, lse, cu_seqlens_k, block_table, alibi_slopes, n_seqs, num_blocks,
              block_size, max_blocks, n_heads_q, n_heads_kv, head_dim, scale);
  p.chunk = L.chunk;
  p.n_slots = L.n_slots;
  p.n_items = static_cast<long long>(L.n_slots) * p.n_hb;
  p.ws_o = static_cast<float*>(workspace);
  p.ws_lse = reinterpret_cast<float*>(static_cast<char*>(workspace) + L.lse_off);
  p.ws_s = reinterpret_cast<float*>(static_cast<char*>(workspace) + L.total);
  p.weights = weights;
  p.prev = prev_weights;
  p.w_stride = weights_stride;
  CUtensorMap tk, tv;
  if (!decode_maps(&tk, &tv, k_cache, v_cache, dtype, head_dim, n_heads_kv, block_size, num_blocks,
                   p))
    return MEA_ERR_CUDA;
  const int grid = total_k > 0 ? static_cast<int>(p.n_items < di.sms ? p.n_items : di.sms) : 0;
  return launch_split_any<mea::DEC_WEIGHTS>(head_dim, dtype, tk, tv, p, grid, max_seqlen_k,
                                            static_cast<cudaStream_t>(stream));
}

int mea_evict_paged(const void* k_cache, const void* v_cache, const int32_t* block_table,
                    const int32_t* cu_seqlens_k, const float* weights, long long weights_stride,
                    void* out_k_cache, void* out_v_cache, const int32_t* out_table, int32_t* kept,
                    float* out_weights, int32_t* out_cu_seqlens_k, int n_seqs, int num_blocks,
                    int num_out_blocks, int block_size, int max_blocks, int max_out_blocks,
                    int max_seqlen_k, int n_heads_kv, int head_dim, int n_keep, int n_recent,
                    int dtype, void* stream) {
  if (!k_cache || !v_cache || !block_table || !cu_seqlens_k || (max_seqlen_k > 0 && !weights) ||
      !out_k_cache || !out_v_cache || !out_table || !kept || !out_weights || !out_cu_seqlens_k)
    return MEA_ERR_NULL;
  if (int rc = check_cache(n_seqs, num_blocks, block_size, max_blocks, n_heads_kv, head_dim, dtype))
    return rc;
  const long long left = n_keep < max_seqlen_k ? n_keep : max_seqlen_k;
  if (num_out_blocks < 1 || max_out_blocks < 1 || max_seqlen_k < 0 ||
      weights_stride < max_seqlen_k || n_keep < 1 || n_recent < 0 || n_recent > n_keep ||
      static_cast<long long>(max_blocks) * block_size < max_seqlen_k ||
      static_cast<long long>(max_out_blocks) * block_size < left)
    return MEA_ERR_SHAPE;
  const long long pairs = static_cast<long long>(n_seqs) * n_heads_kv;
  const long long copies = pairs * ((static_cast<long long>(n_keep) + mea::kEvictRows - 1) /
                                    mea::kEvictRows);
  if (copies > 0x7fffffffll) return MEA_ERR_SHAPE;
  if (!aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(out_k_cache, 16) ||
      !aligned(out_v_cache, 16) || !aligned(block_table, 4) || !aligned(out_table, 4) ||
      !aligned(cu_seqlens_k, 4) || !aligned(weights, 4) || !aligned(out_weights, 4) ||
      !aligned(kept, 4) || !aligned(out_cu_seqlens_k, 4))
    return MEA_ERR_ALIGN;
  // CTAs read lengths, weights and tables while others write the new ones: no updates in place.
  {
    struct Span {
      const void* at;
      long long n;
    };
    const Span outs[] = {
        {kept, pairs * n_keep}, {out_weights, pairs * n_keep}, {out_cu_seqlens_k, n_seqs + 1ll}};
    const Span ins[] = {{weights, pairs * weights_stride},
                        {cu_seqlens_k, n_seqs + 1ll},
                        {block_table, static_cast<long long>(n_seqs) * max_blocks},
                        {out_table, static_cast<long long>(n_seqs) * max_out_blocks}};
    for (int i = 0; i < 3; ++i) {
      for (const Span& in : ins)
        if (overlap(outs[i].at, outs[i].n, in.at, in.n)) return MEA_ERR_SHAPE;
      for (int j = 0; j < i; ++j)
        if (overlap(outs[i].at, outs[i].n, outs[j].at, outs[j].n)) return MEA_ERR_SHAPE;
    }
  }
  DeviceInfo di;
  if (int rc = current_device_info(di); rc != MEA_OK) return rc;
  mea::EvictParams p{};
  p.k = k_cache;
  p.v = v_cache;
  p.k_out = out_k_cache;
  p.v_out = out_v_cache;
  p.block_table = block_table;
  p.out_table = out_table;
  p.cu_k = cu_seqlens_k;
  p.weights = weights;
  p.w_stride = weights_stride;
  p.out_weights = out_weights;
  p.kept = kept;
  p.out_cu = out_cu_seqlens_k;
  p.num_blocks = num_blocks;
  p.num_out_blocks = num_out_blocks;
  p.block_size = block_size;
  p.max_blocks = max_blocks;
  p.max_out_blocks = max_out_blocks;
  p.n_seqs = n_seqs;
  p.hkv = n_heads_kv;
  p.dh = head_dim;
  p.n_keep = n_keep;
  p.n_recent = n_recent;
  // Rank keys in shared memory for up to 48 Ki keys; longer rows are read again in every pass.
  constexpr int max_keys = 48 * 1024;
  p.smem_keys = max_seqlen_k < max_keys ? max_seqlen_k : max_keys;
  p.longest_first = pairs > di.sms && n_seqs > 1 && n_seqs <= mea::kRankedSeqs &&
                    max_seqlen_k >= 4096;
  constexpr auto sel = mea::mea_evict_select_kernel;
  if (smem_attr_once<sel>(max_keys * 4) != cudaSuccess) return MEA_ERR_CUDA;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  clear_stale_launch_error();
  sel<<<static_cast<unsigned>(pairs), mea::kEvictThreads, static_cast<size_t>(p.smem_keys) * 4,
        s>>>(p);
  if (cudaGetLastError() != cudaSuccess) return MEA_ERR_CUDA;
  return launch_dependent(mea::mea_evict_copy_kernel, static_cast<unsigned>(copies), 256, 0, s,
                          p) == cudaSuccess
             ? MEA_OK
             : MEA_ERR_CUDA;
}

}  // extern "C"
