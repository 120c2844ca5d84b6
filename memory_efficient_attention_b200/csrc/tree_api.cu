// tree_api.cu — C ABI of the tree attention over a paged cache and of a prompt's attention weights
// (declared in include/mea.h): argument checks, TMA descriptors and launches. No device memory is
// allocated and no call synchronises the host.
#include <cuda.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>
#include <cstring>

#include "../../include/mea.h"
#include "host_util.h"
#include "tree_sm100.cuh"
#include "weights_sm100.cuh"

using namespace mea_host;

namespace mea_tree {
// This translation unit's device error word (see mea_device_error).
__attribute__((visibility("hidden"))) int device_error(unsigned int* code, bool clear) {
  if (cudaMemcpyFromSymbol(code, mea::g_mea_error, sizeof(*code)) != cudaSuccess)
    return MEA_ERR_CUDA;
  const unsigned int z = 0;
  if (clear && cudaMemcpyToSymbol(mea::g_mea_error, &z, sizeof(z)) != cudaSuccess)
    return MEA_ERR_CUDA;
  return MEA_OK;
}
}  // namespace mea_tree

namespace {

template <int D, bool BF16, bool ALIBI>
int launch_tree(const CUtensorMap& tk, const CUtensorMap& tv, const mea::TreeParams& p, int grid,
                int rows, cudaStream_t s) {
  constexpr auto kern = mea::mea_tree_sm100_kernel<D, BF16, ALIBI>;
  using C = mea::TreeCfg<D>;
  if (smem_attr_once<kern>(C::SMEM_TOTAL) != cudaSuccess) return MEA_ERR_CUDA;
  clear_stale_launch_error();
  kern<<<grid, C::THREADS, C::SMEM_TOTAL, s>>>(tk, tv, p);
  if (cudaGetLastError() != cudaSuccess) return MEA_ERR_CUDA;
  if (grid > 1 && launch_dependent(mea::mea_tree_merge_kernel<D, BF16>,
                                   dim3(static_cast<unsigned>(grid - 1),
                                        static_cast<unsigned>((rows + 15) / 16)),
                                   256, 0, s,
                                   p, grid) != cudaSuccess)
    return MEA_ERR_CUDA;
  return MEA_OK;
}

template <int D, bool BF16, bool CAUSAL, bool ALIBI>
int launch_weights(const CUtensorMap& tq, const CUtensorMap& tk, const mea::WeightsParams& p,
                   int grid, cudaStream_t s) {
  constexpr auto kern = mea::mea_weights_sm100_kernel<D, BF16, CAUSAL, ALIBI>;
  using C = mea::WeightsCfg<D>;
  if (smem_attr_once<kern>(C::SMEM_TOTAL) != cudaSuccess) return MEA_ERR_CUDA;
  clear_stale_launch_error();
  kern<<<grid, C::THREADS, C::SMEM_TOTAL, s>>>(tq, tk, p);
  if (cudaGetLastError() != cudaSuccess) return MEA_ERR_CUDA;
  if (grid > 1 && launch_dependent(mea::mea_weights_merge_kernel<D, CAUSAL>, grid - 1, C::KT, 0,
                                   s, p, grid) != cudaSuccess)
    return MEA_ERR_CUDA;
  return MEA_OK;
}

template <int D, bool BF16>
int launch_weights_d(bool causal, const CUtensorMap& tq, const CUtensorMap& tk,
                     const mea::WeightsParams& p, int grid, cudaStream_t s) {
  const bool al = p.slopes != nullptr;
  if (causal)
    return al ? launch_weights<D, BF16, true, true>(tq, tk, p, grid, s)
              : launch_weights<D, BF16, true, false>(tq, tk, p, grid, s);
  return al ? launch_weights<D, BF16, false, true>(tq, tk, p, grid, s)
            : launch_weights<D, BF16, false, false>(tq, tk, p, grid, s);
}

size_t tree_rows(int d) { return d > 128 ? mea::TreeCfg<256>::ROWS : mea::TreeCfg<128>::ROWS; }
// Two partial ranges per CTA: ROWS rows of the kernel's width, then ROWS log-sum-exps, in fp32.
size_t tree_ws_lse(int d, int sms) {
  return 2 * static_cast<size_t>(sms) * tree_rows(d) * padded_head_dim(d) * sizeof(float);
}
size_t tree_ws(int d, int sms) {
  return tree_ws_lse(d, sms) + 2 * static_cast<size_t>(sms) * tree_rows(d) * sizeof(float);
}

// Keys per item of the prompt's weights, and two ranges of them per CTA.
int weights_keys(int d) { return d > 128 ? mea::WeightsCfg<256>::KT : mea::WeightsCfg<128>::KT; }
size_t weights_ws(int d, int sms) {
  return 2 * static_cast<size_t>(sms) * weights_keys(d) * sizeof(float);
}

// Words of mea_call. An integer that does not fit an int becomes -1, which every count refuses.
struct Words {
  const long long* v;
  int i(int k) const {
    return v[k] >= -0x7fffffffll && v[k] <= 0x7fffffffll ? static_cast<int>(v[k]) : -1;
  }
  float f(int k) const {
    double d;
    std::memcpy(&d, v + k, sizeof(d));
    return static_cast<float>(d);
  }
  template <class T>
  T* p(int k) const {
    return reinterpret_cast<T*>(v[k]);
  }
};

}  // namespace

extern "C" {

int mea_call(int entry, const void* words) {
  if (!words) return MEA_ERR_NULL;
  const Words w{static_cast<const long long*>(words)};
  switch (entry) {
    case MEA_CALL_BLOCK_KEY_BOUNDS:
      return mea_block_key_bounds(w.p<const void>(0), w.p<const int32_t>(1),
                                  w.p<const int32_t>(2), w.p<const int32_t>(3), w.p<void>(4),
                                  w.i(5), w.i(6), w.i(7), w.i(8), w.i(9), w.i(10), w.i(11),
                                  w.i(12), w.p<void>(13));
    case MEA_CALL_SELECT_BLOCKS:
      return mea_select_blocks(w.p<const void>(0), w.p<const void>(1), w.p<const int32_t>(2),
                               w.p<const int32_t>(3), w.p<int32_t>(4), w.i(5), w.i(6), w.i(7),
                               w.i(8), w.i(9), w.i(10), w.i(11), w.i(12), w.i(13), w.i(14),
                               w.i(15), w.i(16), w.p<void>(17));
    case MEA_CALL_DECODE_SELECTED:
      return mea_decode_selected(w.p<const void>(0), w.p<const void>(1), w.p<const void>(2),
                                 w.p<const int32_t>(3), w.p<const int32_t>(4),
                                 w.p<const int32_t>(5), w.p<void>(6), w.p<float>(7), w.i(8),
                                 w.i(9), w.i(10), w.i(11), w.i(12), w.i(13), w.i(14), w.i(15),
                                 w.f(16), w.p<const float>(17), w.i(18), w.p<void>(19),
                                 static_cast<size_t>(w.v[20]), w.p<void>(21));
    case MEA_CALL_DECODE_WEIGHTS:
      return mea_decode_weights(w.p<const void>(0), w.p<const void>(1), w.p<const void>(2),
                                w.p<const int32_t>(3), w.p<const int32_t>(4), w.p<void>(5),
                                w.p<float>(6), w.p<float>(7), w.p<const float>(8),
                                static_cast<long long>(w.v[9]), w.i(10), w.i(11), w.i(12),
                                w.i(13), w.i(14), w.i(15), w.i(16), w.i(17), w.i(18), w.f(19),
                                w.p<const float>(20), w.i(21), w.p<void>(22),
                                static_cast<size_t>(w.v[23]), w.i(24), w.p<void>(25));
    case MEA_CALL_ATTENTION_WEIGHTS:
      return mea_attention_weights(w.p<const void>(0), w.p<const void>(1), w.p<const float>(2),
                                   w.p<const int32_t>(3), w.p<const int32_t>(4), w.p<float>(5),
                                   static_cast<long long>(w.v[6]), w.i(7), w.i(8), w.i(9),
                                   w.i(10), w.i(11), w.i(12), w.i(13), w.i(14), w.f(15), w.i(16),
                                   w.p<const float>(17), w.i(18), w.i(19), w.p<void>(20),
                                   static_cast<size_t>(w.v[21]), w.p<void>(22));
    case MEA_CALL_EVICT_PAGED:
      return mea_evict_paged(w.p<const void>(0), w.p<const void>(1), w.p<const int32_t>(2),
                             w.p<const int32_t>(3), w.p<const float>(4),
                             static_cast<long long>(w.v[5]), w.p<void>(6), w.p<void>(7),
                             w.p<const int32_t>(8), w.p<int32_t>(9), w.p<float>(10),
                             w.p<int32_t>(11), w.i(12), w.i(13), w.i(14), w.i(15), w.i(16),
                             w.i(17), w.i(18), w.i(19), w.i(20), w.i(21), w.i(22), w.i(23),
                             w.p<void>(24));
    case MEA_CALL_DECODE_TREE:
      return mea_decode_tree(w.p<const void>(0), w.p<const void>(1), w.p<const void>(2),
                             w.p<const int32_t>(3), w.p<const int32_t>(4), w.p<const int32_t>(5),
                             w.p<const int32_t>(6), w.p<void>(7), w.p<float>(8), w.i(9), w.i(10),
                             w.i(11), w.i(12), w.i(13), w.i(14), w.i(15), w.i(16), w.i(17),
                             w.i(18), w.i(19), w.f(20), w.p<const float>(21), w.i(22),
                             w.p<void>(23), static_cast<size_t>(w.v[24]), w.p<void>(25));
    default:
      return MEA_ERR_SHAPE;
  }
}

size_t mea_decode_tree_workspace_size(int n_heads_q, int n_heads_kv, int head_dim) {
  if (n_heads_q < 1 || n_heads_kv < 1 || n_heads_q % n_heads_kv || !dec_head_dim_ok(head_dim))
    return 0;
  DeviceInfo di;
  return tree_ws(head_dim, current_device_info(di) == MEA_OK ? di.sms : 148);
}

int mea_decode_tree(const void* q, const void* k_cache, const void* v_cache,
                    const int32_t* block_table, const int32_t* cu_seqlens_q,
                    const int32_t* cu_seqlens_k, const int32_t* tree_mask, void* out, float* lse,
                    int n_seqs, int total_q, int max_seqlen_q, int max_seqlen_k, int mask_words,
                    int num_blocks, int block_size, int max_blocks, int n_heads_q,
                    int n_heads_kv, int head_dim, float scale, const float* alibi_slopes,
                    int dtype, void* workspace, size_t workspace_bytes, void* stream) {
  if (!q || !k_cache || !v_cache || !block_table || !cu_seqlens_q || !cu_seqlens_k ||
      !tree_mask || !out)
    return MEA_ERR_NULL;
  if (n_seqs < 1 || total_q < 0 || max_seqlen_q < 0 || max_seqlen_q > total_q ||
      max_seqlen_k < 0 || mask_words < 1 ||
      static_cast<long long>(mask_words) * 32 < max_seqlen_q || num_blocks < 1 ||
      max_blocks < 1 || static_cast<long long>(max_blocks) * block_size < max_seqlen_k)
    return MEA_ERR_SHAPE;
  if (!(block_size == 16 || block_size == 32 || (block_size >= 64 && block_size % 64 == 0)))
    return MEA_ERR_SHAPE;
  if (n_heads_q < 1 || n_heads_kv < 1 || n_heads_q % n_heads_kv != 0) return MEA_ERR_HEADS;
  if (static_cast<long long>(total_q) * (n_heads_q / n_heads_kv) > 0x3fffffffll)
    return MEA_ERR_SHAPE;
  if (!dec_head_dim_ok(head_dim)) return MEA_ERR_HEAD_DIM;
  if (dtype != MEA_F16 && dtype != MEA_BF16) return MEA_ERR_DTYPE;
  if (!std::isfinite(scale)) return MEA_ERR_SCALE;
  if (!aligned(q, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(out, 16) ||
      (lse && !aligned(lse, 4)) || !aligned(cu_seqlens_q, 4) || !aligned(cu_seqlens_k, 4) ||
      !aligned(block_table, 4) || !aligned(tree_mask, 4) ||
      (alibi_slopes && !aligned(alibi_slopes, 4)))
    return MEA_ERR_ALIGN;
  if (!workspace || !aligned(workspace, 256)) return MEA_ERR_WORKSPACE;
  DeviceInfo di;
  if (int rc = current_device_info(di); rc != MEA_OK) return rc;
  if (workspace_bytes < tree_ws(head_dim, di.sms)) return MEA_ERR_WORKSPACE;
  if (total_q == 0 || max_seqlen_q == 0) return MEA_OK;

  mea::TreeParams p{};
  p.q = q;
  p.out = out;
  p.lse = lse;
  p.cu_q = cu_seqlens_q;
  p.cu_k = cu_seqlens_k;
  p.block_table = block_table;
  p.mask = reinterpret_cast<const uint32_t*>(tree_mask);
  p.slopes = alibi_slopes;
  p.ws_o = static_cast<float*>(workspace);
  p.ws_lse =
      reinterpret_cast<float*>(static_cast<char*>(workspace) + tree_ws_lse(head_dim, di.sms));
  p.n_seqs = n_seqs;
  p.total_q = total_q;
  p.hq = n_heads_q;
  p.hkv = n_heads_kv;
  p.dh = head_dim;
  p.R = n_heads_q / n_heads_kv;
  p.mask_words = mask_words;
  p.block_size = block_size;
  p.max_blocks = max_blocks;
  p.num_blocks = num_blocks;
  p.box_rows = block_size < 64 ? block_size : 64;
  p.c1 = scale * 1.4426950408889634f;
  p.timeout_ns = g_timeout_ns.load();
  CUtensorMap tk, tv;
  if (!encode_4d(&tk, k_cache, dtype, head_dim, n_heads_kv, block_size, num_blocks, 64, 1,
                 p.box_rows, 1) ||
      !encode_4d(&tv, v_cache, dtype, head_dim, n_heads_kv, block_size, num_blocks, 64, 1,
                 p.box_rows, 1))
    return MEA_ERR_CUDA;
  // No more CTAs than tiles. (Two tiles a CTA, side by side on its warpgroups, and half as many
  // partials to join, took 16.3 us where one takes 14.4 on 8 rows of 777 keys.)
  const long long most = static_cast<long long>(tree_rows(head_dim));
  const long long all = static_cast<long long>(max_seqlen_q) * p.R;  // rows of an item, at most `most`
  const int rows = static_cast<int>(all < most ? all : most);
  const long long parts = (all + most - 1) / most;
  const long long tiles = max_seqlen_k > 128 ? (static_cast<long long>(max_seqlen_k) + 127) / 128
                                             : 1;
  const double bound = static_cast<double>(n_seqs) * n_heads_kv * parts * tiles;
  const int grid = bound < di.sms ? static_cast<int>(bound) : di.sms;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool bf = dtype == MEA_BF16, al = alibi_slopes != nullptr;
#define MEA_TREE(DD)                                                                        \
  return bf ? (al ? launch_tree<DD, true, true>(tk, tv, p, grid, rows, s)                         \
                  : launch_tree<DD, true, false>(tk, tv, p, grid, rows, s))                       \
            : (al ? launch_tree<DD, false, true>(tk, tv, p, grid, rows, s)                        \
                  : launch_tree<DD, false, false>(tk, tv, p, grid, rows, s))
  if (head_dim > 128) MEA_TREE(256);
  if (head_dim > 64) MEA_TREE(128);
  MEA_TREE(64);
#undef MEA_TREE
}

size_t mea_attention_weights_workspace_size(int head_dim) {
  if (!dec_head_dim_ok(head_dim)) return 0;
  DeviceInfo di;
  return weights_ws(head_dim, current_device_info(di) == MEA_OK ? di.sms : 148);
}

int mea_attention_weights(const void* q, const void* k, const float* lse,
                          const int32_t* cu_seqlens_q, const int32_t* cu_seqlens_k,
                          float* weights, long long weights_stride, int n_seqs, int total_q,
                          int total_k, int max_seqlen_q, int max_seqlen_k, int n_heads_q,
                          int n_heads_kv, int head_dim, float scale, int mask_kind,
                          const float* alibi_slopes, int last_queries, int dtype,
                          void* workspace, size_t workspace_bytes, void* stream) {
  if (!cu_seqlens_q || !cu_seqlens_k || (total_q > 0 && (!q || !lse)) ||
      (max_seqlen_k > 0 && (!k || !weights)))
    return MEA_ERR_NULL;
  if (n_seqs < 1 || total_q < 0 || total_k < 0 || max_seqlen_q < 0 || max_seqlen_k < 0 ||
      max_seqlen_q > total_q || max_seqlen_k > total_k || weights_stride < max_seqlen_k ||
      last_queries < 0)
    return MEA_ERR_SHAPE;
  if (n_heads_q < 1 || n_heads_kv < 1 || n_heads_q % n_heads_kv != 0) return MEA_ERR_HEADS;
  if (!dec_head_dim_ok(head_dim)) return MEA_ERR_HEAD_DIM;
  if (dtype != MEA_F16 && dtype != MEA_BF16) return MEA_ERR_DTYPE;
  if (mask_kind != MEA_MASK_NONE && mask_kind != MEA_MASK_CAUSAL) return MEA_ERR_MASK;
  if (!std::isfinite(scale)) return MEA_ERR_SCALE;
  if (!aligned(q, 16) || !aligned(k, 16) || !aligned(lse, 4) || !aligned(cu_seqlens_q, 4) ||
      !aligned(cu_seqlens_k, 4) || !aligned(weights, 4) ||
      (alibi_slopes && !aligned(alibi_slopes, 4)))
    return MEA_ERR_ALIGN;
  if (!workspace || !aligned(workspace, 16)) return MEA_ERR_WORKSPACE;
  DeviceInfo di;
  if (int rc = current_device_info(di); rc != MEA_OK) return rc;
  if (workspace_bytes < weights_ws(head_dim, di.sms)) return MEA_ERR_WORKSPACE;
  if (max_seqlen_k == 0) return MEA_OK;
  const int R = n_heads_q / n_heads_kv;
  int log2_p = 0;
  while (log2_p < 7 && R % (2 << log2_p) == 0) ++log2_p;
  mea::WeightsParams p{};
  p.lse = lse;
  p.cu_q = cu_seqlens_q;
  p.cu_k = cu_seqlens_k;
  p.slopes = alibi_slopes;
  p.weights = weights;
  p.ws = static_cast<float*>(workspace);
  p.w_stride = weights_stride;
  p.n_seqs = n_seqs;
  p.total_q = total_q;
  p.hq = n_heads_q;
  p.hkv = n_heads_kv;
  p.R = R;
  p.last = last_queries;
  p.log2_p = log2_p;
  p.c1 = scale * 1.4426950408889634f;
  p.timeout_ns = g_timeout_ns.load();
  CUtensorMap tq, tk;
  // (without queries the q map is not used)
  if (!(total_q > 0 ? encode_3d(&tq, q, dtype, head_dim, n_heads_q, total_q, 64, 1u << log2_p,
                                128u >> log2_p)
                    : encode_3d(&tq, k, dtype, head_dim, n_heads_kv, total_k, 64, 1, 128)) ||
      !encode_3d(&tk, k, dtype, head_dim, n_heads_kv, total_k, 64, 1, 128))
    return MEA_ERR_CUDA;
  // No more CTAs than steps.
  const long long kt = weights_keys(head_dim), qt = 128 >> log2_p;
  const double items = static_cast<double>(n_seqs) * n_heads_kv *
                       ((static_cast<long long>(max_seqlen_k) + kt - 1) / kt);
  const double steps = items * (R >> log2_p) *
                       ((static_cast<long long>(max_seqlen_q) + qt - 1) / qt + 1);
  const int grid = steps < di.sms ? static_cast<int>(steps) : di.sms;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool causal = mask_kind == MEA_MASK_CAUSAL, bf = dtype == MEA_BF16;
  if (head_dim > 128)
    return bf ? launch_weights_d<256, true>(causal, tq, tk, p, grid, s)
              : launch_weights_d<256, false>(causal, tq, tk, p, grid, s);
  if (head_dim > 64)
    return bf ? launch_weights_d<128, true>(causal, tq, tk, p, grid, s)
              : launch_weights_d<128, false>(causal, tq, tk, p, grid, s);
  return bf ? launch_weights_d<64, true>(causal, tq, tk, p, grid, s)
            : launch_weights_d<64, false>(causal, tq, tk, p, grid, s);
}

}  // extern "C"
