// cache_sm100.cuh — operators on a paged K/V cache beside the attention that reads it, for
// sm_100a: the blocks' key ranges, the choice of the blocks a query attends to, and the removal of
// the keys with the least attention weight.
//
// Cache layout throughout: K and V are [num_blocks, block_size, Hkv, D] in 16 bits; key t of
// request b lives in block block_table[b, t / block_size], slot t % block_size. Ids outside
// [0, num_blocks) are skipped, never dereferenced.
#pragma once

#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <type_traits>

#include "ptx.cuh"

namespace mea {

template <bool BF16>
using Half2 = typename std::conditional<BF16, __nv_bfloat162, __half2>::type;
template <bool BF16>
using Half1 = typename std::conditional<BF16, __nv_bfloat16, __half>::type;

__device__ __forceinline__ float max_nan(float a, float b) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}
template <bool BF16>
__device__ __forceinline__ Half2<BF16> splat_half2(float x) {
  if constexpr (BF16)
    return __float2bfloat162_rn(x);
  else
    return __float2half2_rn(x);
}

// ------------------------------------------------------------------------------------------
// Key ranges: lo[blk, g, d] = min over the block's existing slots of K[slot, g, d], hi = max.
//
// Bound by reading K once (it writes 2 / block_size of what it reads). A thread owns 8 columns (16
// bytes) of one block's rows and walks its slots, so that a warp reads whole rows; eight slots are
// in flight per thread. Nothing is exchanged between threads.
// ------------------------------------------------------------------------------------------
struct BoundsParams {
  const void* k;
  void* bounds;  // [num_blocks, hkv, 2, D]
  const int32_t* block_table;
  const int32_t* cu_k;
  const int32_t* first_key;  // [n_seqs] or null: only blocks that hold keys >= first_key[b]
  int num_blocks, block_size, max_blocks, hkv, dh;
};

template <bool BF16>
__global__ void __launch_bounds__(256) mea_key_bounds_kernel(const BoundsParams p) {
  const int b = blockIdx.y;
  const int L = __ldg(p.cu_k + b + 1) - __ldg(p.cu_k + b);
  const int nblk = min((L + p.block_size - 1) / p.block_size, p.max_blocks);
  const int first = p.first_key ? max(__ldg(p.first_key + b), 0) / p.block_size : 0;
  const int row16 = p.hkv * p.dh / 8;  // 16-byte pieces of a slot's row over all heads
  const long long n = static_cast<long long>(nblk - first) * row16;
  const uint4* k = static_cast<const uint4*>(p.k);
  uint4* out = static_cast<uint4*>(p.bounds);
  for (long long u = static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x; u < n;
       u += static_cast<long long>(gridDim.x) * blockDim.x) {
    const int jj = static_cast<int>(u / row16);
    const int j = first + jj;
    const int ch = static_cast<int>(u - static_cast<long long>(jj) * row16);
    const int id = __ldg(p.block_table + static_cast<size_t>(b) * p.max_blocks + j);
    if (id < 0 || id >= p.num_blocks) continue;
    const int ns = min(p.block_size, L - j * p.block_size);
    const uint4* src = k + static_cast<size_t>(id) * p.block_size * row16 + ch;
    using H2 = Half2<BF16>;
    H2 lo[4], hi[4];
    uint4 v = __ldg(src);
#pragma unroll
    for (int i = 0; i < 4; ++i) lo[i] = hi[i] = reinterpret_cast<const H2*>(&v)[i];
    for (int t = 1; t < ns; t += 8) {
      uint4 w[8];
      // (slots past the last one repeat it)
#pragma unroll
      for (int q = 0; q < 8; ++q) w[q] = __ldg(src + static_cast<size_t>(min(t + q, ns - 1)) * row16);
#pragma unroll
      for (int q = 0; q < 8; ++q) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const H2 x = reinterpret_cast<const H2*>(&w[q])[i];
          lo[i] = __hmin2_nan(lo[i], x);
          hi[i] = __hmax2_nan(hi[i], x);
        }
      }
    }
    const int d8 = p.dh / 8;
    const int g = ch / d8, c = ch - g * d8;
    uint4* dst = out + (static_cast<size_t>(id) * p.hkv + g) * 2 * d8 + c;
    dst[0] = *reinterpret_cast<uint4*>(lo);
    dst[d8] = *reinterpret_cast<uint4*>(hi);
  }
}

// ------------------------------------------------------------------------------------------
// The k largest of n 32-bit keys by one CTA: radix selection of key - min, 8 bits a pass from the
// highest bit in which the keys differ at all. (Weights and scores share their leading bits: taken
// as they are, a pass counted all keys in a few bins, one after the other.)
// ------------------------------------------------------------------------------------------
// Order-preserving image of an fp32 value (as unsigned; -0 equals +0). NaN ranks above all.
__device__ __forceinline__ uint32_t rank_key(float x) {
  if (x != x) return 0xFFFFFFFEu;
  const uint32_t u = __float_as_uint(x + 0.f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
// The value back from its rank key.
__device__ __forceinline__ float rank_value(uint32_t k) {
  return __uint_as_float(k == 0xFFFFFFFEu ? 0x7FFFFFFFu : (k & 0x80000000u) ? k ^ 0x80000000u : ~k);
}
constexpr uint32_t kRankAlways = 0xFFFFFFFFu;  // ranks above every value

struct SelectScratch {
  int hist[2048];  // 4 x 256, one histogram a pass, or 2048 bins
  uint32_t least[32], most[32];
  int sum[2][32];
  int bin, above, in;
};

// Exclusive sum over the CTA's warps of `v` (one value per warp, left in sum[] by the caller).
template <int NT>
__device__ __forceinline__ int warps_before(const int* sum) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int v = lane < NT / 32 ? sum[lane] : 0;
  int incl = v;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, incl, off);
    if (lane >= off) incl += y;
  }
  return __shfl_sync(0xffffffffu, incl - v, warp);
}

// Returns the key T of the k-th largest (or one below it) and in `ties` how many of the keys equal to
// T belong to the k (the caller takes the lowest indices of them, beside all keys above T).
// 1 <= k <= n. Every pass costs one barrier: it has its own histogram, and every warp scans it.
template <int NT, class Get>
__device__ __forceinline__ uint32_t radix_select(Get get, int n, int k, SelectScratch& sc,
                                                 int& ties) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  for (int i = tid; i < 4 * 256; i += NT) sc.hist[i] = 0;
  uint32_t lo = 0xFFFFFFFFu, hi = 0u;
#pragma unroll 4
  for (int i = tid; i < n; i += NT) {
    const uint32_t x = get(i);
    if (x != kRankAlways) {  // (far above all others: they would take the first digits' range)
      lo = min(lo, x);
      hi = max(hi, x);
    }
  }
  lo = __reduce_min_sync(0xffffffffu, lo);
  hi = __reduce_max_sync(0xffffffffu, hi);
  if (lane == 0) {
    sc.least[warp] = lo;
    sc.most[warp] = hi;
  }
  __syncthreads();
  lo = __reduce_min_sync(0xffffffffu, lane < NT / 32 ? sc.least[lane] : 0xFFFFFFFFu);
  hi = __reduce_max_sync(0xffffffffu, lane < NT / 32 ? sc.most[lane] : 0u);
  ties = k;
  if (lo > hi) return kRankAlways;  // no other keys
  const uint32_t top = hi + 1u;     // stands for kRankAlways below
  uint32_t prefix = 0, high = 0;
  int need = k;
  int shift = max(24 - __clz(static_cast<int>(top - lo)), 0);
  for (int pass = 0;; ++pass) {
    int* h = sc.hist + 256 * pass;
#pragma unroll 4
    for (int i = tid; i < n; i += NT) {
      const uint32_t x = min(get(i), top) - lo;
      if ((x & high) == prefix) atomicAdd(&h[(x >> shift) & 255u], 1);
    }
    __syncthreads();
    int c[8], sum = 0;  // bins 255 - 8 lane, ... downwards
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      c[i] = h[255 - (lane * 8 + i)];
      sum += c[i];
    }
    int incl = sum;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, incl, off);
      if (lane >= off) incl += y;
    }
    const int src = __ffs(__ballot_sync(0xffffffffu, incl >= need)) - 1;
    int above = incl - sum, bin = 0, in = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (in == 0 && above + c[i] >= need) {
        bin = 255 - (lane * 8 + i);
        in = c[i];
      }
      if (in == 0) above += c[i];
    }
    bin = __shfl_sync(0xffffffffu, bin, src);
    in = __shfl_sync(0xffffffffu, in, src);
    need -= __shfl_sync(0xffffffffu, above, src);
    prefix |= static_cast<uint32_t>(bin) << shift;
    if (need == in) {  // the whole bin belongs: everything from its least value on
      ties = 0;
      return prefix + lo - 1u;  // (rank keys are above 0)
    }
    if (shift == 0) break;
    const int next = max(shift - 8, 0);
    high = 0xFFFFFFFFu << shift;
    shift = next;
  }
  ties = need;
  return prefix + lo == top ? kRankAlways : prefix + lo;
}

// The same for many keys, whose least and greatest (lo, hi; per thread, of its own keys) the caller has
// at hand from writing them: 11 bits a pass, the bins shared out over the threads. (With fixed digits
// from the top bit, weights filled four bins a binade and the passes were always three: 5003 weights to
// 1024 with their copy 11.3 us, so 10.6.)
template <int NT, class Get>
__device__ __forceinline__ uint32_t radix_select_wide(Get get, int n, int k, uint32_t lo,
                                                      uint32_t hi, SelectScratch& sc, int& ties) {
  constexpr int PER = 2048 / NT;  // bins per thread
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
#pragma unroll
  for (int i = 0; i < PER; ++i) sc.hist[tid * PER + i] = 0;
  lo = __reduce_min_sync(0xffffffffu, lo);
  hi = __reduce_max_sync(0xffffffffu, hi);
  if (lane == 0) {
    sc.least[warp] = lo;
    sc.most[warp] = hi;
  }
  __syncthreads();
  lo = __reduce_min_sync(0xffffffffu, lane < NT / 32 ? sc.least[lane] : 0xFFFFFFFFu);
  hi = __reduce_max_sync(0xffffffffu, lane < NT / 32 ? sc.most[lane] : 0u);
  uint32_t prefix = 0, high = 0;
  int need = k;
  int shift = max(21 - __clz(static_cast<int>(hi - lo)), 0);
#pragma unroll 1
  while (true) {
#pragma unroll 4
    for (int i = tid; i < n; i += NT) {
      const uint32_t x = get(i) - lo;
      if ((x & high) == prefix) atomicAdd(&sc.hist[(x >> shift) & 2047u], 1);
    }
    __syncthreads();
    // Thread tid takes the bins counted from the top, and clears them for the next pass.
    int c[PER], sum = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      int& h = sc.hist[2047 - (tid * PER + i)];
      c[i] = h;
      h = 0;
      sum += c[i];
    }
    int incl = sum;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, incl, off);
      if (lane >= off) incl += y;
    }
    if (lane == 31) sc.sum[0][warp] = incl;
    __syncthreads();
    int above = warps_before<NT>(sc.sum[0]) + incl - sum;
    if (above < need && need <= above + sum) {
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        if (above < need && need <= above + c[i]) {
          sc.bin = 2047 - (tid * PER + i);
          sc.above = above;
          sc.in = c[i];
        }
        above += c[i];
      }
    }
    __syncthreads();
    prefix |= static_cast<uint32_t>(sc.bin) << shift;
    need -= sc.above;
    if (need == sc.in) {  // the whole bin belongs: everything from its least value on
      ties = 0;
      return prefix + lo - 1u;  // (rank keys are above 0)
    }
    if (shift == 0) break;
    high = 0xFFFFFFFFu << shift;
    shift = max(shift - 11, 0);
  }
  ties = need;
  return prefix + lo;
}

// The request of rank `r` by length, longest first (equal ones by index), so that CTAs in rank order
// leave no long request to the end. n <= kRankedSeqs; len[n] and found[1] in shared memory.
// Every CTA counts for itself, n steps of n threads: worth it for few requests that can be long. With
// it and without, on 8 KV heads: eviction of 64 requests of up to 16384 keys 85 and 90 us, of 32 of
// 32768 56 and 60, but of 64 of 600 19.8 and 19.2, of 256 of 600 87 and 59, of 1024 of 600 1974 and
// 225; block choice for 64 requests of up to 1024 blocks 38.5 and 42, of 256 20.3 and 20.5, of 128
// 17.8 and 17.0, for 256 of 19 41 and 18.
constexpr int kRankedSeqs = 64;
__device__ __forceinline__ int nth_longest(const int32_t* cu, int n, int r, int* len, int* found) {
  const int t = threadIdx.x;
  int mine = 0;
  if (t < n) {
    mine = __ldg(cu + t + 1) - __ldg(cu + t);
    len[t] = mine;
  }
  __syncthreads();
  if (t < n) {
    int rank = 0;
    for (int u = 0; u < n; ++u) rank += len[u] > mine || (len[u] == mine && u < t);
    if (rank == r) found[0] = t;
  }
  __syncthreads();
  const int b = found[0];
  __syncthreads();
  return b;
}

// Hands the indices of the keys above T, and of the first `ties` keys equal to T, in ascending
// order to put(place, index, key). A warp takes a contiguous part: it counts, the counts are added up
// over the warps, then it places.
template <int NT, class Get, class Put>
__device__ __forceinline__ void compact_selected(Get get, Put put, int n, uint32_t T, int ties,
                                                 SelectScratch& sc) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const unsigned below = (1u << lane) - 1u;
  const int part = ((n + NT - 1) / NT) * 32;
  const int i0 = warp * part, i1 = min(n, i0 + part);
  int gt = 0, eq = 0;
  for (int b = i0; b < i1; b += 32) {
    const uint32_t x = b + lane < i1 ? get(b + lane) : 0u;
    gt += __popc(__ballot_sync(0xffffffffu, b + lane < i1 && x > T));
    eq += __popc(__ballot_sync(0xffffffffu, b + lane < i1 && x == T));
  }
  if (lane == 0) {
    sc.sum[0][warp] = gt;
    sc.sum[1][warp] = eq;
  }
  __syncthreads();
  gt = warps_before<NT>(sc.sum[0]);
  eq = warps_before<NT>(sc.sum[1]);
  for (int b = i0; b < i1; b += 32) {
    const bool in = b + lane < i1;
    const uint32_t x = in ? get(b + lane) : 0u;
    const bool is_gt = in && x > T, is_eq = in && x == T;
    const unsigned bg = __ballot_sync(0xffffffffu, is_gt);
    const unsigned be = __ballot_sync(0xffffffffu, is_eq);
    const int e = eq + __popc(be & below);
    if (is_gt || (is_eq && e < ties)) put(gt + __popc(bg & below) + min(e, ties), b + lane, x);
    gt += __popc(bg);
    eq += __popc(be);
  }
}

// ------------------------------------------------------------------------------------------
// Choice of blocks. For every key k of block j and the R query heads q_h of its KV head,
//     sum_h q_h . k <= sum_d up[d] hi[j, d] + down[d] lo[j, d],
//     up = sum_h max(q_h, 0),  down = sum_h min(q_h, 0)       (each term bounds its own product),
// which is the block's score: one dot product of length 2 D, whatever the group's size, because
// the bound of a sum of heads is linear in (up, down). The scores are summed in 64 bits and rounded
// to 32 once: then the order of summation does not show in the choice.
//
// Bound by reading the ranges (4 D bytes a block and head); in 64 bits throughout, the conversions and
// products took three times as long as that. So the scores are first computed on the tensor cores
// (mma.sync, 16 blocks a tile, w = (down, up) as three 16-bit pieces in three of the eight columns,
// fp32 sums), which is off by at most delta = CHUNKS 2^-17 sum|w| max|range| (2 CHUNKS instructions, each of
// which adds 17 terms aligned to the largest with an error of 2^-23 of it at most), and the blocks
// within 2 delta of the cut, a few as a rule, are scored again in 64 bits: a block further above (below)
// the cut than that is above (below) it in 64 bits too.
// A cluster of CTAs serves one (request, KV head): each CTA's warps score a share of its blocks and
// leave the rank keys in the first CTA's shared memory, which then selects.
// ------------------------------------------------------------------------------------------
struct SelectParams {
  const void* q;       // [n_seqs, hq, D]
  const void* bounds;  // [num_blocks, hkv, 2, D]
  const int32_t* block_table;
  const int32_t* cu_k;
  int32_t* selected;   // [n_seqs, hkv, n_select]
  int num_blocks, block_size, max_blocks, hq, hkv, dh, n_select, n_first, n_last;
  int n_seqs;
  int max_live;        // bound on a request's blocks: rank keys in shared memory
  int longest_first;
};

constexpr int kSelThreads = 256;

template <bool BF16>
__device__ __forceinline__ float half_f32(uint32_t w, int i) {
  const Half2<BF16> h = *reinterpret_cast<const Half2<BF16>*>(&w);
  return i ? __high2float(h) : __low2float(h);
}
template <bool BF16>
__device__ __forceinline__ uint32_t half_bits(float x) {
  const Half1<BF16> h = static_cast<Half1<BF16>>(x);
  return *reinterpret_cast<const unsigned short*>(&h);
}

// CHUNKS: 32-element pieces of a block's two rows (2 D elements), 4, 8 or 16.
template <bool BF16, int CHUNKS>
__global__ void __launch_bounds__(kSelThreads, CHUNKS == 16 ? 1 : 2)
    mea_select_blocks_kernel(const SelectParams p) {
  namespace cg = cooperative_groups;
  auto cluster = cg::this_cluster();
  const int cs = static_cast<int>(cluster.num_blocks());
  const int cr = static_cast<int>(cluster.block_rank());
  const int pair = blockIdx.x / cs;
  const int R = p.hq / p.hkv;
  extern __shared__ __align__(16) uint32_t s_keys[];
  __shared__ double s_w[2 * 256];  // [down][up]
  // w's 16-bit pieces as B fragments: [chunk][lane][4 words] (lanes 4 n + t4, n < 3, hold piece n)
  __shared__ __align__(16) uint32_t s_frag[CHUNKS * 32 * 4];
  __shared__ int s_again[32];
  __shared__ float s_most[8 * (kSelThreads / 32)];  // max |range| by warp of the cluster
  __shared__ SelectScratch s_sc;
  const int g = pair % p.hkv;
  int b = pair / p.hkv;
  pdl_trigger();
  if (p.longest_first)
    b = nth_longest(p.cu_k, p.n_seqs, b, reinterpret_cast<int*>(s_w), s_sc.sum[0]);
  const int L = __ldg(p.cu_k + b + 1) - __ldg(p.cu_k + b);
  const int nblk = min((L + p.block_size - 1) / p.block_size, min(p.max_blocks, p.max_live));
  int32_t* out = p.selected + (static_cast<size_t>(b) * p.hkv + g) * p.n_select;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (nblk <= p.n_select) {  // every block (the whole cluster takes this branch)
    if (cr == 0)
      for (int i = tid; i < p.n_select; i += kSelThreads) out[i] = i < nblk ? i : -1;
    return;
  }
  // The first CTA's shared memory must be live before the others write to it: each CTA says here
  // that it runs, and waits for the others' word only before its first such write.
  if (cs > 1) cluster.barrier_arrive();
  const int np = p.dh / 4;  // 16-byte pieces of a block's ranges
  const int32_t* row = p.block_table + static_cast<size_t>(b) * p.max_blocks;
  const uint4* bounds = static_cast<const uint4*>(p.bounds);
  const int g8 = lane >> 2, t4 = lane & 3;
  const int stride = cs * (kSelThreads / 32) * 16;
  const int jw = (cr * (kSelThreads / 32) + warp) * 16;
  // Rows g8 and g8 + 8 of a tile are blocks j + g8, j + g8 + 8; lane t4 reads pieces t4, t4 + 4, ... of
  // them (the sum does not mind which lane has which columns, as long as w goes by the same order).
  auto block_id = [&](int j) { return j < nblk ? __ldg(row + j) : -1; };
  auto source = [&](int id) {
    return (id >= 0 && id < p.num_blocks)
               ? bounds + (static_cast<size_t>(id) * p.hkv + g) * np + t4
               : nullptr;
  };
  uint4 v[CHUNKS][2];  // a whole tile; a chunk's registers take the next tile's as soon as it is used
  const uint4 *s0 = nullptr, *s1 = nullptr;
  auto load = [&](int c) {
    const bool in = c * 4 + t4 < np;
    v[c][0] = in && s0 ? __ldg(s0 + c * 4) : make_uint4(0u, 0u, 0u, 0u);
    v[c][1] = in && s1 ? __ldg(s1 + c * 4) : make_uint4(0u, 0u, 0u, 0u);
  };
  s0 = source(block_id(jw + g8));
  s1 = source(block_id(jw + g8 + 8));
#pragma unroll
  for (int c = 0; c < CHUNKS; ++c) load(c);
  int id0 = block_id(jw + stride + g8), id1 = block_id(jw + stride + g8 + 8);
  for (int i = tid; i < CHUNKS * 128; i += kSelThreads) s_frag[i] = 0u;
  __syncthreads();
  // up and down, while the first blocks are on their way
  const Half1<BF16>* q =
      static_cast<const Half1<BF16>*>(p.q) + (static_cast<size_t>(b) * p.hq + g * R) * p.dh;
  for (int d = tid; d < p.dh; d += kSelThreads) {
    double up = 0.0, down = 0.0;
#pragma unroll 8
    for (int h = 0; h < R; ++h) {
      const float x = static_cast<float>(q[static_cast<size_t>(h) * p.dh + d]);
      up += x > 0.f ? x : 0.f;
      down += x > 0.f ? 0.f : x;  // (a NaN goes here)
    }
    s_w[d] = down;
    s_w[p.dh + d] = up;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      double x = e ? up : down;
#pragma unroll
      for (int n = 0; n < 3; ++n) {
        const uint32_t bits = half_bits<BF16>(static_cast<float>(x));
        const int k = e * p.dh + d;  // column of (down, up): chunk k / 32, lane's piece (k / 8) % 4
        reinterpret_cast<unsigned short*>(
            s_frag)[(((k >> 5) * 32 + n * 4 + ((k >> 3) & 3)) * 4 + ((k >> 1) & 3)) * 2 + (k & 1)] =
            static_cast<unsigned short>(bits);
        x -= static_cast<double>(half_f32<BF16>(bits, 0));
      }
    }
  }
  __syncthreads();
  if (cs > 1) cluster.barrier_wait();
  uint32_t* keys = cs > 1 ? cluster.map_shared_rank(s_keys, 0) : s_keys;
  Half2<BF16> most = splat_half2<BF16>(0.f);
  for (int j = jw; j < nblk; j += stride) {
    float acc[4] = {0.f, 0.f, 0.f, 0.f};
    s0 = source(id0);
    s1 = source(id1);
    id0 = block_id(j + 2 * stride + g8);
    id1 = block_id(j + 2 * stride + g8 + 8);
#pragma unroll
    for (int c = 0; c < CHUNKS; ++c) {
      const uint32_t x[2][4] = {{v[c][0].x, v[c][0].y, v[c][0].z, v[c][0].w},
                                {v[c][1].x, v[c][1].y, v[c][1].z, v[c][1].w}};
      const uint32_t a0[4] = {x[0][0], x[1][0], x[0][1], x[1][1]};
      const uint32_t a1[4] = {x[0][2], x[1][2], x[0][3], x[1][3]};
      const uint4 w = *reinterpret_cast<const uint4*>(&s_frag[(c * 32 + lane) * 4]);
      mma16816<BF16>(acc, a0, w.x, w.y);
      mma16816<BF16>(acc, a1, w.z, w.w);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        most = __hmax2_nan(most, __habs2(*reinterpret_cast<const Half2<BF16>*>(&x[0][i])));
        most = __hmax2_nan(most, __habs2(*reinterpret_cast<const Half2<BF16>*>(&x[1][i])));
      }
      load(c);
    }
    // Columns 0 and 1 are lane t4 = 0's, column 2 lane t4 = 1's.
    const float third0 = __shfl_down_sync(0xffffffffu, acc[0], 1);
    const float third1 = __shfl_down_sync(0xffffffffu, acc[2], 1);
    if (t4 == 0) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int i = j + g8 + 8 * h;
        const float x = h ? (acc[2] + acc[3]) + third1 : (acc[0] + acc[1]) + third0;
        const bool always = i < p.n_first || i >= nblk - p.n_last;
        if (i < nblk) keys[i] = always ? kRankAlways : rank_key(x);
      }
    }
  }
  {
    float m = max_nan(__low2float(most), __high2float(most));
#pragma unroll
    for (int off = 16; off > 0; off >>= 1)
      m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, off));
    float* dst = cs > 1 ? cluster.map_shared_rank(s_most, 0) : s_most;
    if (lane == 0) dst[cr * (kSelThreads / 32) + warp] = m;
  }
  if (cs > 1)
    cluster.sync();
  else
    __syncthreads();
  if (cr != 0) return;
  auto get = [&](int i) { return s_keys[i]; };
  auto put = [&](int at, int i, uint32_t) {
    if (at < p.n_select) out[at] = i;
  };
  int ties = 0;
  uint32_t T = radix_select<kSelThreads>(get, nblk, p.n_select, s_sc, ties);
  if (T != kRankAlways) {
    // delta, in every warp
    float most_all = 0.f, sum_w = 0.f, most_w = 0.f;
    for (int i = lane; i < cs * (kSelThreads / 32); i += 32) most_all = max_nan(most_all, s_most[i]);
    for (int d = lane; d < 2 * p.dh; d += 32) {
      const float x = fabsf(static_cast<float>(s_w[d]));
      sum_w += x;
      most_w = max_nan(most_w, x);
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) {
      most_all = max_nan(most_all, __shfl_xor_sync(0xffffffffu, most_all, off));
      sum_w += __shfl_xor_sync(0xffffffffu, sum_w, off);
      most_w = max_nan(most_w, __shfl_xor_sync(0xffffffffu, most_w, off));
    }
    // (the last term: third pieces below a half's smallest step)
    const float delta = CHUNKS * 0x1p-17f * sum_w * most_all + 0x1p-15f * most_all;
    const float cut = rank_value(T);
    const float above = cut + 2.f * delta, below = cut - 2.f * delta;
    // Otherwise every block is scored again: a NaN or an infinity somewhere, sums that fp32 might not
    // hold, queries' sums that a half does not.
    const bool sane = delta < 0x1p100f && (BF16 || most_w < 65504.f);
    // Keys become "in", 1 (out) or 2 (to be scored again).
    int n_in = 0, n_again = 0;
    for (int i = tid; i < nblk; i += kSelThreads) {
      const uint32_t x = s_keys[i];
      uint32_t to = kRankAlways;
      if (x != kRankAlways) {
        const float f = rank_value(x);
        if (!(sane && f > above)) to = sane && f < below ? 1u : 2u;
      }
      s_keys[i] = to;
      n_in += to == kRankAlways;
      n_again += to == 2u;
    }
    n_in = __reduce_add_sync(0xffffffffu, n_in);
    n_again = __reduce_add_sync(0xffffffffu, n_again);
    __syncthreads();  // (the selection's sums have been read)
    if (lane == 0) {
      s_sc.sum[0][warp] = n_in;
      s_sc.sum[1][warp] = n_again;
    }
    __syncthreads();
    n_in = __reduce_add_sync(0xffffffffu, lane < kSelThreads / 32 ? s_sc.sum[0][lane] : 0);
    n_again = __reduce_add_sync(0xffffffffu, lane < kSelThreads / 32 ? s_sc.sum[1][lane] : 0);
    T = 1u;  // keys above: "in", and those marked 2 where all of them belong
    ties = 0;
    if (n_in + n_again != p.n_select) {
      auto exact = [&](int i) {  // warp-cooperative
        const int id = __ldg(row + i);
        const uint4* src = (id >= 0 && id < p.num_blocks)
                               ? bounds + (static_cast<size_t>(id) * p.hkv + g) * np
                               : nullptr;
        double x = 0.0;
        for (int c = lane; src && c < np; c += 32) {
          const uint4 r = __ldg(src + c);
          const uint32_t w4[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
          for (int e = 0; e < 8; ++e)
            x = fma(s_w[c * 8 + e], static_cast<double>(half_f32<BF16>(w4[e >> 1], e & 1)), x);
        }
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) x += __shfl_xor_sync(0xffffffffu, x, off);
        return rank_key(static_cast<float>(x));
      };
      if (n_again <= 32) {
        // A list of them in order, a warp each, and one warp that ranks them.
        if (warp == 0) {
          int n = 0;
          for (int i0 = 0; i0 < nblk; i0 += 32) {
            const bool mine = i0 + lane < nblk && s_keys[i0 + lane] == 2u;
            const unsigned m = __ballot_sync(0xffffffffu, mine);
            if (mine) s_again[n + __popc(m & ((1u << lane) - 1u))] = i0 + lane;
            n += __popc(m);
          }
        }
        __syncthreads();
        for (int a = warp; a < n_again; a += kSelThreads / 32) {
          const uint32_t x = exact(s_again[a]);
          if (lane == 0) s_sc.hist[a] = static_cast<int>(x);
        }
        __syncthreads();
        if (warp == 0 && lane < n_again) {
          const uint32_t x = static_cast<uint32_t>(s_sc.hist[lane]);
          int rank = 0;
          for (int a = 0; a < n_again; ++a) {
            const uint32_t y = static_cast<uint32_t>(s_sc.hist[a]);
            rank += y > x || (y == x && a < lane);
          }
          s_keys[s_again[lane]] = n_in + rank < p.n_select ? kRankAlways : 1u;
        }
      } else {
        for (int i0 = warp * 32; i0 < nblk; i0 += kSelThreads) {
          unsigned again = __ballot_sync(0xffffffffu, i0 + lane < nblk && s_keys[i0 + lane] == 2u);
          while (again) {
            const int i = i0 + __ffs(again) - 1;
            again &= again - 1;
            const uint32_t x = exact(i);
            if (lane == 0) s_keys[i] = x;
          }
        }
        __syncthreads();
        T = radix_select<kSelThreads>(get, nblk, p.n_select, s_sc, ties);
      }
    }
  }
  __syncthreads();
  compact_selected<kSelThreads>(get, put, nblk, T, ties, s_sc);
}

// ------------------------------------------------------------------------------------------
// Eviction, first kernel: the keys of (request b, KV head g) that stay: its last n_recent and, of
// the others, those with the largest weights, n_keep in all, in ascending order. One CTA per
// pair; the rank keys stay in shared memory when they fit. Bound by the passes over shared memory:
// at up to 32768 keys one CTA fits an SM, and with more pairs than SMs the longest requests go first
// (nth_longest).
// ------------------------------------------------------------------------------------------
struct EvictParams {
  const void* k;
  const void* v;
  void* k_out;
  void* v_out;
  const int32_t* block_table;
  const int32_t* out_table;  // [n_seqs, max_out_blocks]
  const int32_t* cu_k;
  const float* weights;      // [n_seqs, hkv, w_stride]
  float* out_weights;        // [n_seqs, hkv, n_keep]
  int32_t* kept;             // [n_seqs, hkv, n_keep]
  int32_t* out_cu;           // [n_seqs + 1]
  long long w_stride;
  int num_blocks, num_out_blocks, block_size, max_blocks, max_out_blocks, n_seqs, hkv, dh;
  int n_keep, n_recent;
  int smem_keys;             // rank keys that fit in shared memory
  int longest_first;         // more CTAs than SMs: long rows must not come last
};

constexpr int kEvictThreads = 1024;

// Keys of request b (never past the row of weights).
__device__ __forceinline__ int evict_keys(const EvictParams& p, int b) {
  const int L = max(__ldg(p.cu_k + b + 1) - __ldg(p.cu_k + b), 0);
  return p.w_stride < L ? static_cast<int>(p.w_stride) : L;
}

__global__ void __launch_bounds__(kEvictThreads) mea_evict_select_kernel(const EvictParams p) {
  extern __shared__ __align__(16) uint32_t s_keys[];
  __shared__ SelectScratch s_sc;
  const int g = blockIdx.x % p.hkv;
  int b = blockIdx.x / p.hkv;
  const int tid = threadIdx.x;
  pdl_trigger();
  if (p.longest_first) b = nth_longest(p.cu_k, p.n_seqs, b, s_sc.hist, s_sc.sum[0]);
  const int L = evict_keys(p, b);
  // The new prefix sums: one warp of the first CTA.
  if (blockIdx.x == 0 && tid < 32) {
    int base = 0;
    for (int i0 = 0; i0 < p.n_seqs; i0 += 32) {
      const int i = i0 + tid;
      int incl = i < p.n_seqs ? min(evict_keys(p, i), p.n_keep) : 0;
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, incl, off);
        if (tid >= off) incl += y;
      }
      if (i < p.n_seqs) p.out_cu[i + 1] = base + incl;
      base += __shfl_sync(0xffffffffu, incl, 31);
    }
    if (tid == 0) p.out_cu[0] = 0;
  }
  const size_t pair = static_cast<size_t>(b) * p.hkv + g;
  const float* w = p.weights + pair * p.w_stride;
  int32_t* kept = p.kept + pair * p.n_keep;
  float* ow = p.out_weights + pair * p.n_keep;
  if (L <= p.n_keep) {
    for (int i = tid; i < p.n_keep; i += kEvictThreads) {
      kept[i] = i < L ? i : -1;
      ow[i] = i < L ? w[i] : 0.f;
    }
    return;
  }
  const int m = L - p.n_recent;       // keys that compete, for
  const int k = p.n_keep - p.n_recent;  // this many places (k < m)
  if (k > 0) {
    auto put = [&](int at, int i, uint32_t x) {
      kept[at] = i;
      ow[at] = rank_value(x);
    };
    int ties = 0;
    uint32_t lo = 0xFFFFFFFFu, hi = 0u;
    if (m <= p.smem_keys) {
      for (int i0 = tid; i0 < m; i0 += kEvictThreads * 8) {
        float x[8];
#pragma unroll
        for (int u = 0; u < 8; ++u)
          x[u] = i0 + u * kEvictThreads < m ? __ldcs(w + i0 + u * kEvictThreads) : 0.f;
#pragma unroll
        for (int u = 0; u < 8; ++u) {
          if (i0 + u * kEvictThreads >= m) continue;
          const uint32_t y = rank_key(x[u]);
          s_keys[i0 + u * kEvictThreads] = y;
          lo = min(lo, y);
          hi = max(hi, y);
        }
      }
      auto get = [&](int i) { return s_keys[i]; };
      const uint32_t T = radix_select_wide<kEvictThreads>(get, m, k, lo, hi, s_sc, ties);
      compact_selected<kEvictThreads>(get, put, m, T, ties, s_sc);
    } else {
      auto get = [&](int i) { return rank_key(__ldg(w + i)); };
      for (int i = tid; i < m; i += kEvictThreads) {
        lo = min(lo, get(i));
        hi = max(hi, get(i));
      }
      const uint32_t T = radix_select_wide<kEvictThreads>(get, m, k, lo, hi, s_sc, ties);
      compact_selected<kEvictThreads>(get, put, m, T, ties, s_sc);
    }
  }
  for (int i = tid; i < p.n_recent; i += kEvictThreads) {
    kept[k + i] = m + i;
    ow[k + i] = w[m + i];
  }
}

// Second kernel: key kept[i]'s K and V rows of KV head g go to slot i of the request's new blocks.
// Bound by moving the rows once (read and write). A CTA takes 64 rows of one pair: it looks their
// places up once, then every thread moves 16-byte pieces, four loads in flight (eight take the registers
// of half the CTAs: 449 instead of 390 us for 64 x 8 x 4096 rows; two: 417 us).
constexpr int kEvictRows = 64;

__global__ void __launch_bounds__(256) mea_evict_copy_kernel(const EvictParams p) {
  __shared__ long long s_src[kEvictRows], s_dst[kEvictRows];  // 16-byte piece offsets, -1: none
  pdl_wait();
  const int tiles = (p.n_keep + kEvictRows - 1) / kEvictRows;
  const long long item = blockIdx.x;
  // Heads innermost: CTAs that run together write neighbouring pieces of the same slots.
  const int g = static_cast<int>(item % p.hkv);
  const int tile = static_cast<int>(item / p.hkv % tiles);
  const int b = static_cast<int>(item / p.hkv / tiles);
  const long long pair = static_cast<long long>(b) * p.hkv + g;
  const int L = evict_keys(p, b);
  const int n = min(min(L, p.n_keep) - tile * kEvictRows, kEvictRows);
  if (n <= 0) return;
  const int d8 = p.dh / 8;
  if (threadIdx.x < kEvictRows) {
    const int i = tile * kEvictRows + threadIdx.x;
    long long src = -1, dst = -1;
    if (threadIdx.x < n) {
      const int t = ld_after_wait(p.kept + static_cast<size_t>(pair) * p.n_keep + i);
      const int js = t / p.block_size, jd = i / p.block_size;
      if (js < p.max_blocks && jd < p.max_out_blocks) {
        const int is = __ldg(p.block_table + static_cast<size_t>(b) * p.max_blocks + js);
        const int id = __ldg(p.out_table + static_cast<size_t>(b) * p.max_out_blocks + jd);
        if (is >= 0 && is < p.num_blocks && id >= 0 && id < p.num_out_blocks) {
          src = ((static_cast<long long>(is) * p.block_size + t % p.block_size) * p.hkv + g) * d8;
          dst = ((static_cast<long long>(id) * p.block_size + i % p.block_size) * p.hkv + g) * d8;
        }
      }
    }
    s_src[threadIdx.x] = src;
    s_dst[threadIdx.x] = dst;
  }
  __syncthreads();
  const uint4* k = static_cast<const uint4*>(p.k);
  const uint4* v = static_cast<const uint4*>(p.v);
  uint4* ko = static_cast<uint4*>(p.k_out);
  uint4* vo = static_cast<uint4*>(p.v_out);
  const int total = n * 2 * d8;  // pieces: [row][K or V][d8]
  for (int i0 = threadIdx.x; i0 < total; i0 += 256 * 4) {
    uint4 x[4];
    long long to[4];
    bool is_v[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int i = i0 + u * 256;
      to[u] = -1;
      if (i < total) {
        const int half = i / d8, c = i - half * d8;
        const int row = half >> 1;
        is_v[u] = (half & 1) != 0;
        if (s_src[row] >= 0) {
          x[u] = __ldcs((is_v[u] ? v : k) + s_src[row] + c);
          to[u] = s_dst[row] + c;
        }
      }
    }
#pragma unroll
    for (int u = 0; u < 4; ++u)
      if (to[u] >= 0) (is_v[u] ? vo : ko)[to[u]] = x[u];
  }
}

}  // namespace mea
