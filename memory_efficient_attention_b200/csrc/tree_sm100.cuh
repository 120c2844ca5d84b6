// tree_sm100.cuh — attention of a tree of drafted tokens over a paged K/V cache, for sm_100a.
//
// Request b has n_b query tokens (drafted tokens, whose K and V are its cache's last n_b keys) and
// ctx = L_b - n_b keys before them. Token i attends to every key t < ctx and to drafted token j
// (key ctx + j) when bit j of its mask row is set: a row softmax like the forward's, with an
// arbitrary mask in the last keys only.
//
// Rows are (token, query head of one KV group) pairs: row rho of KV head g is token rho / R, head
// g R + rho % R, so a group's K/V tile is read once for up to ROWS rows (n_b R of them exist). An
// item is one (request, KV head, ROWS rows); it walks 128-key tiles.
//
// Schedule: all items' tiles form one line, cut into equal ranges, one per CTA (requests of
// any length mix then load every SM alike, and one long request is split over all of them). A range
// that covers a whole item writes its rows; a range that covers part of one writes a partial (O / l
// and log2-sum-exp, fp32) to the workspace, at most two per CTA, and the merge kernel joins them.
//
// Roles and tensor-memory use follow the forward kernel: two softmax warpgroups, one per 128-row
// sub-tile (thread = row = TMEM lane), an issuer warp that alternates the sub-tiles' Q K^T and P V
// (tcgen05, fp32 in TMEM), a producer warp, and a scheduler warp that hands the CTA's ranges, decoded,
// to the others through a small queue in shared memory. The softmax warps also put Q into shared memory
// (its rows are few and need not be a box of q). When an item's rows fit one sub-tile, both
// warpgroups take those rows and every second key tile each, so that one's softmax still runs
// beside the other's products; the first then joins the two O, which lie in the same TMEM lanes.
//
// P is rounded to the inputs' 16-bit type before P V, as in the forward: the product takes both its
// operands in one 16-bit type, and P in two 16-bit pieces would be half as many products again where
// the products are the bound. It moves an output by at most half a step of 16 bits of sum p |v|; the
// row sums and log-sum-exps come from the unrounded values, in fp32.
//
// Bound: with n_b R rows, a key costs 4 D bytes and 4 D n_b R flop; up to about 250 rows (bf16
// peak over HBM rate) that is HBM-bound, beyond it the tensor cores are.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <type_traits>

#include "fwd_sm100.cuh"
#include "ptx.cuh"

namespace mea {

struct TreeParams {
  const void* q;               // [total_q, hq, D]
  void* out;                   // [total_q, hq, D]
  float* lse;                  // [hq, total_q] or null
  const int32_t* cu_q;
  const int32_t* cu_k;
  const int32_t* block_table;  // [n_seqs, max_blocks]
  const uint32_t* mask;        // [total_q, mask_words]
  const float* slopes;
  float* ws_o;                 // [2 grid, ROWS, D] partial outputs
  float* ws_lse;               // [2 grid, ROWS] their log2-sum-exps
  int n_seqs, total_q, hq, hkv, dh, R, mask_words;
  int block_size, max_blocks, num_blocks;
  int box_rows;                // keys per TMA box: min(block_size, 64)
  float c1;                    // scale * log2(e)
  unsigned long long timeout_ns;
};

template <int D>
struct TreeCfg {
  static constexpr int SUBS = D == 256 ? 1 : 2;  // 128-row sub-tiles per item (TMEM: O is D wide)
  static constexpr int ROWS = 128 * SUBS;
  static constexpr int ATOMS = D / 64;
  static constexpr uint32_t ATOM_BYTES = 128 * 128;
  static constexpr uint32_t TILE_BYTES = 128 * D * 2;
  static constexpr int NS = D == 64 ? 8 : D == 128 ? 4 : 2;  // K and V tiles in the ring
  static constexpr uint32_t SMEM_Q = 0;
  static constexpr uint32_t SMEM_KV = SUBS * TILE_BYTES;
  static constexpr uint32_t SMEM_POS = SMEM_KV + NS * TILE_BYTES;  // 8 warps x 128 floats
  static constexpr uint32_t SMEM_ML = SMEM_POS + 8 * 512;  // the second warpgroup's (m, l) by row
  static constexpr uint32_t SMEM_MISC = SMEM_ML + 1024;
  static constexpr int QD = 4;                             // ranges in the queue, 64 bytes each
  static constexpr uint32_t MISC_QUEUE = 512;
  static constexpr uint32_t SMEM_TOTAL = SMEM_MISC + MISC_QUEUE + QD * 64 + 1024;
  static_assert(SMEM_TOTAL <= 232448, "shared memory per CTA");
  static constexpr int THREADS = 384;
  static constexpr int REGS_SOFTMAX = 216;
  static constexpr int REGS_OTHER = 72;
  static constexpr uint32_t TM_O = 256;
};

// A CTA's range of one item's tiles.
struct TreeFrag {
  int b, g, row0;        // request, KV head, first row of the item
  int q0, nq, ctx, L;    // first packed token, tokens, context keys, keys
  int t0, t1;            // tiles [t0, t1)
  bool dual;             // one sub-tile's rows: the warpgroups take key tiles in turn
  bool whole;            // the range is the whole item
  bool first;            // the CTA's first range
};

// A range in the queue: 32-bit words at these places; flags 0 ends the list.
enum : uint32_t { TQ_B = 0, TQ_G = 4, TQ_ROW0 = 8, TQ_Q0 = 12, TQ_NQ = 16, TQ_CTX = 20, TQ_L = 24,
                  TQ_T0 = 28, TQ_T1 = 32, TQ_FLAGS = 36 };
enum : int { TF_LIVE = 1, TF_DUAL = 2, TF_WHOLE = 4, TF_FIRST = 8 };

struct TreeSeq {
  int q0, nq, L, tiles, parts;
  long long work;  // tiles of all the request's items
};

template <int ROWS>
__device__ __forceinline__ TreeSeq tree_seq(const TreeParams& p, int b) {
  TreeSeq s;
  s.q0 = __ldg(p.cu_q + b);
  s.nq = max(__ldg(p.cu_q + b + 1) - s.q0, 0);
  s.L = max(__ldg(p.cu_k + b + 1) - __ldg(p.cu_k + b), 0);
  s.tiles = s.L > 128 ? (s.L + 127) / 128 : 1;  // (no keys: one tile that sees nothing)
  s.parts = (s.nq * p.R + ROWS - 1) / ROWS;
  s.work = static_cast<long long>(s.parts) * p.hkv * s.tiles;
  return s;
}

// Warp-cooperative: sum over all requests of their work.
template <int ROWS>
__device__ __forceinline__ long long tree_total(const TreeParams& p) {
  long long acc = 0;
  for (int b = threadIdx.x & 31; b < p.n_seqs; b += 32) acc += tree_seq<ROWS>(p, b).work;
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, off);
  return acc;
}

// Warp-cooperative: the request that tile `pos` of the line belongs to, and its first tile.
template <int ROWS>
__device__ __forceinline__ int tree_find(const TreeParams& p, long long pos, long long& base) {
  const int lane = threadIdx.x & 31;
  long long acc = 0;
  for (int b0 = 0; b0 < p.n_seqs; b0 += 32) {
    const long long w = b0 + lane < p.n_seqs ? tree_seq<ROWS>(p, b0 + lane).work : 0;
    long long incl = w;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, incl, off);
      if (lane >= off) incl += y;
    }
    const unsigned hit = __ballot_sync(0xffffffffu, pos < acc + incl);
    if (hit) {
      const int src = __ffs(hit) - 1;
      base = acc + __shfl_sync(0xffffffffu, incl - w, src);
      return b0 + src;
    }
    acc += __shfl_sync(0xffffffffu, incl, 31);
  }
  base = acc;
  return p.n_seqs;
}

// A CTA's walk over its range of the line.
template <int ROWS>
struct TreeWalk {
  long long pos, end, start, base;
  int b;
  TreeSeq s;
  __device__ __forceinline__ void init(const TreeParams& p) {
    const long long total = tree_total<ROWS>(p);
    const long long per = div_nn(total + gridDim.x - 1, gridDim.x);
    start = pos = per * blockIdx.x;
    end = min(total, pos + per);
    b = p.n_seqs;
    if (pos < end) {
      b = tree_find<ROWS>(p, pos, base);
      s = tree_seq<ROWS>(p, b);
    }
  }
  __device__ __forceinline__ bool next(const TreeParams& p, TreeFrag& f) {
    if (pos >= end) return false;
    while (pos >= base + s.work) {  // (ends: pos < end <= the line's length)
      base += s.work;
      s = tree_seq<ROWS>(p, ++b);
    }
    const long long off = pos - base;
    const int item = static_cast<int>(div_nn(off, s.tiles));
    f.t0 = static_cast<int>(off - static_cast<long long>(item) * s.tiles);
    f.t1 = static_cast<int>(min(static_cast<long long>(s.tiles), f.t0 + (end - pos)));
    f.g = item / s.parts;
    f.row0 = (item - f.g * s.parts) * ROWS;
    f.b = b;
    f.q0 = s.q0;
    f.nq = s.nq;
    f.L = s.L;
    f.ctx = s.L - s.nq;
    f.dual = ROWS == 256 && s.nq * p.R - f.row0 <= 128;
    f.whole = f.t0 == 0 && f.t1 == s.tiles;
    f.first = pos == start;
    pos += f.t1 - f.t0;
    return true;
  }
};

// 32 bits of a token's view of the keys [key, key + 32): context keys are seen, drafted ones by
// the mask row, keys past the end not.
__device__ __forceinline__ uint32_t tree_view(const uint32_t* row, int words, int key, int ctx,
                                              int L) {
  const int left = L - key;
  if (left <= 0) return 0u;
  const int j = key - ctx;  // draft index of bit 0
  uint32_t v;
  if (j <= -32) {
    v = 0xFFFFFFFFu;
  } else if (j < 0) {
    v = ((1u << (-j)) - 1u) | ((words > 0 ? __ldg(row) : 0u) << (-j));
  } else {
    const int i = j >> 5;
    const uint32_t lo = i < words ? __ldg(row + i) : 0u;
    const uint32_t hi = i + 1 < words ? __ldg(row + i + 1) : 0u;
    v = __funnelshift_r(lo, hi, j & 31);
  }
  return left >= 32 ? v : v & ((1u << left) - 1u);
}

// Ancestors of drafted token i: the set bits of its mask row other than its own.
__device__ __forceinline__ int tree_depth(const uint32_t* row, int words, int i, int nq) {
  int n = 0;
  for (int w = 0; w < words; ++w) {
    uint32_t x = __ldg(row + w);
    if ((i >> 5) == w) x &= ~(1u << (i & 31));
    const int left = nq - w * 32;  // (bits past the drafted tokens name none)
    if (left < 32) x &= left > 0 ? (1u << left) - 1u : 0u;
    n += __popc(x);
  }
  return n;
}

// Softmax of one tile that reaches into the drafted keys (or past the last key): the scores are
// masked one by one.
template <bool BF16, bool ALIBI>
__device__ __forceinline__ bool tree_masked_tile(float c1, uint32_t t_s, const uint32_t (&view)[4],
                                                 float pos, float slope2, const float* kpos,
                                                 float& m_ref, float& l, float& alpha) {
  uint32_t sr[128];
#pragma unroll
  for (int c4 = 0; c4 < 4; ++c4)
    tmem_ld32(t_s + c4 * 32, *reinterpret_cast<uint32_t(*)[32]>(&sr[c4 * 32]));
  tmem_wait_ld();
  float x[128];
#pragma unroll
  for (int c = 0; c < 128; ++c) {
    float v = __uint_as_float(sr[c]) * c1;
    if constexpr (ALIBI) v = fmaf(-slope2, fabsf(pos - kpos[c]), v);
    x[c] = (view[c >> 5] >> (c & 31)) & 1u ? v : -INFINITY;
  }
  const float m_new = fmaxf(m_ref, row_max128(x));
  alpha = 1.f;
  const bool resc = m_new > m_ref + 8.0f;
  if (resc) {
    alpha = ex2_approx(m_ref - m_new);
    l *= alpha;
    m_ref = m_new;
  }
  const float m_use = (m_ref == -INFINITY) ? 0.f : m_ref;
  l += exp_tile_to_tmem<BF16, false, false>(x, 1.f, 0.f, m_use, t_s);
  return resc;
}

template <int D, bool BF16, bool ALIBI>
__global__ void __launch_bounds__(384, 1)
    mea_tree_sm100_kernel(const __grid_constant__ CUtensorMap tm_k,
                          const __grid_constant__ CUtensorMap tm_v, const TreeParams p) {
  using C = TreeCfg<D>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  const uint32_t pad = (1024u - (smem_u32(smem_raw) & 1023u)) & 1023u;
  uint8_t* smem = smem_raw + pad;
  const uint32_t sbase = smem_u32(smem);
  const uint32_t q_s = sbase + C::SMEM_Q;
  const uint32_t kv_s0 = sbase + C::SMEM_KV;
  constexpr int B_QF = 0, B_QE = 1, B_KVF = 2, B_KVE = 2 + C::NS, B_SF = 2 + 2 * C::NS;
  constexpr int B_PF = B_SF + 2, B_OF = B_PF + 2, B_OE = B_OF + 2, B_ML = B_OE + 2;
  constexpr int B_IF = B_ML + 1, B_IE = B_IF + C::QD;
  constexpr int B_DR = B_IE + C::QD, N_BARS = B_DR + 1;
  static_assert(8 * N_BARS + 8 <= C::MISC_QUEUE, "barrier region");
  const uint32_t bar0 = sbase + C::SMEM_MISC;
#define BAR(i) (bar0 + 8u * static_cast<uint32_t>(i))
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::SMEM_MISC + 8 * N_BARS);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const uint64_t tmo = p.timeout_ns;
  const unsigned ecode = KID_TREE << 8;

  if (threadIdx.x == 0) {
    mbar_init(BAR(B_QF), 4 * C::SUBS);  // one elected arrival per softmax warp
    mbar_init(BAR(B_QE), 1);
    for (int s = 0; s < C::NS; ++s) {
      mbar_init(BAR(B_KVF + s), 1);
      mbar_init(BAR(B_KVE + s), 1);
    }
    for (int h = 0; h < 2; ++h) {
      mbar_init(BAR(B_SF + h), 1);
      mbar_init(BAR(B_PF + h), 4);
      mbar_init(BAR(B_OF + h), 1);
      mbar_init(BAR(B_OE + h), 128);
    }
    mbar_init(BAR(B_ML), 4);
    for (int s = 0; s < C::QD; ++s) {
      mbar_init(BAR(B_IF + s), 1);
      mbar_init(BAR(B_IE + s), 2 + 4 * C::SUBS);  // producer, issuer, softmax warps
    }
    mbar_init(BAR(B_DR), 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 9 && lane == 0) {
    tma_prefetch_desc(&tm_k);
    tma_prefetch_desc(&tm_v);
  }
  if (warp == 8) {
    tmem_alloc(smem_u32(tmem_slot), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const uint32_t queue = sbase + C::SMEM_MISC + C::MISC_QUEUE;
  pdl_trigger();

  static_assert(256 * C::REGS_SOFTMAX + 128 * C::REGS_OTHER <= 384 * 168, "register split");
  if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::REGS_OTHER));
    if (warp == 9) {
      // -------------------------------------------------------------- TMA producer
      uint32_t cnt = 0, n_frag = 0;
      bool ok = true;
      // One box of box_rows keys x 64 columns per lane (at most 8 x 4 boxes a tile).
      const int nbox = 128 / p.box_rows * C::ATOMS;
      const int piece = lane / C::ATOMS, atom = lane % C::ATOMS;
      const bool issuer = lane < nbox;
      while (true) {
        const uint32_t e = queue + 64u * (n_frag % C::QD);
        ok = mbar_wait(BAR(B_IF + n_frag % C::QD), (n_frag / C::QD) & 1u, abort_flag, tmo,
                       ecode | 13);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok || lds_s32(e + TQ_FLAGS) == 0) break;
        const int fg = lds_s32(e + TQ_G), ft1 = lds_s32(e + TQ_T1);
        const int L = lds_s32(e + TQ_L);
        const int32_t* row =
            p.block_table + static_cast<size_t>(lds_s32(e + TQ_B)) * p.max_blocks;
        const int nblk = min((L + p.block_size - 1) / p.block_size, p.max_blocks);
        const int n = ft1 - lds_s32(e + TQ_T0);
        __syncwarp();
        if (lane == 0) mbar_arrive(BAR(B_IE + n_frag % C::QD));
        ++n_frag;
        // Tiles go from the last one down. A block past the request's last one takes id num_blocks,
        // which the TMA fills with zeros; ids are read three tiles ahead of their use.
        auto block_id = [&](int jj) {
          const int blk = ((ft1 - 1 - jj) * 128 + piece * p.box_rows) / p.block_size;
          return (issuer && jj < n && blk < nblk) ? __ldg(row + blk) : p.num_blocks;
        };
        int id_q[3];
#pragma unroll
        for (int u = 0; u < 3; ++u) id_q[u] = block_id(u);
        for (int jj = 0; jj < n && ok; ++jj) {
          const int id = id_q[0];
          id_q[0] = id_q[1];
          id_q[1] = id_q[2];
          id_q[2] = block_id(jj + 3);
          const int r0 = ((ft1 - 1 - jj) * 128 + piece * p.box_rows) % p.block_size;
#pragma unroll 1
          for (int kv = 0; kv < 2; ++kv) {
            const uint32_t s = cnt % C::NS;
            if (lane == 0) {
              ok = mbar_wait(BAR(B_KVE + s), ((cnt / C::NS) & 1u) ^ 1u, abort_flag, tmo, ecode | 1);
              if (ok) mbar_arrive_expect_tx(BAR(B_KVF + s), C::TILE_BYTES);
            }
            ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
            if (!ok) break;
            if (issuer)
              tma_load_4d(kv_s0 + s * C::TILE_BYTES + atom * C::ATOM_BYTES +
                              static_cast<uint32_t>(piece * p.box_rows * 128),
                          kv ? &tm_v : &tm_k, BAR(B_KVF + s), atom * 64, fg, r0, id);
            ++cnt;
          }
        }
        if (!ok) break;
      }
      if (!ok && lane == 0) {
        // Let the loads already issued land before the CTA's shared memory goes away.
        for (uint32_t s = 0; s < C::NS && s < cnt; ++s) {
          const uint32_t last = cnt - 1 - ((cnt - 1 - s) % C::NS);
          volatile int never = 0;
          mbar_wait(BAR(B_KVF + s), (last / C::NS) & 1u, &never, tmo, ecode | 15);
        }
      }
      __syncwarp();
    } else if (warp == 8) {
      // -------------------------------------------------------------- tcgen05 issuer
      if (lane == 0) {
        constexpr uint32_t IDESC_QK = umma_idesc_f16(BF16, 128, 128, false, false);
        constexpr uint32_t IDESC_PV = umma_idesc_f16(BF16, 128, D, false, true);
        uint32_t kv_cnt = 0, n_frag = 0;
        uint32_t pv_cnt[2] = {0, 0}, oe_cnt[2] = {0, 0};
        bool ok = true;
        while (ok) {
          const uint32_t e = queue + 64u * (n_frag % C::QD);
          ok = mbar_wait(BAR(B_IF + n_frag % C::QD), (n_frag / C::QD) & 1u, abort_flag, tmo,
                         ecode | 16);
          if (!ok) break;
          const int flags = lds_s32(e + TQ_FLAGS);
          if (flags == 0) break;
          const int n = lds_s32(e + TQ_T1) - lds_s32(e + TQ_T0);
          const bool dual = (flags & TF_DUAL) != 0;
          mbar_arrive(BAR(B_IE + n_frag % C::QD));
          ok = mbar_wait(BAR(B_QF), n_frag & 1u, abort_flag, tmo, ecode | 6);
          if (!ok) break;
          tc_fence_after();
          const uint32_t base = kv_cnt;
          // Each sub-tile in turn: O_h += P_h V of its last tile, then S_h = Q K^T of its next one (S_h
          // is free then: P lies over it). Both sub-tiles take every tile, or (dual) every second.
          const int step = dual ? 2 : 1;
          for (int t0 = 0; t0 < n + step && ok; t0 += step) {
#pragma unroll
            for (int h = 0; h < C::SUBS; ++h) {
              const int t = t0 + (dual ? h : 0), tp = t - step;
              const bool frees = dual || h == C::SUBS - 1;  // no other sub-tile needs the K or V
              if (tp >= 0 && tp < n) {
                const uint32_t vi = base + 2 * tp + 1, vs = vi % C::NS;
                ok = mbar_wait(BAR(B_KVF + vs), (vi / C::NS) & 1u, abort_flag, tmo, ecode | 5);
                if (!ok) break;
                ok = mbar_wait_spin(BAR(B_PF + h), pv_cnt[h] & 1u, abort_flag, tmo, ecode | 3);
                if (!ok) break;
                if (tp < step) {  // the sub-tile's first tile: O_h has been read
                  ok = mbar_wait(BAR(B_OE + h), (oe_cnt[h] & 1u) ^ 1u, abort_flag, tmo, ecode | 4);
                  if (!ok) break;
                  ++oe_cnt[h];
                }
                tc_fence_after();
                const uint32_t vbase = kv_s0 + vs * C::TILE_BYTES;
#pragma unroll
                for (int kk = 0; kk < 8; ++kk) {
                  const uint64_t bd = umma_desc_sw128(vbase + kk * 16 * 128, C::ATOM_BYTES, 1024);
                  mma_ts(tmem + C::TM_O + h * D, tmem + h * 128 + kk * 8, bd, IDESC_PV,
                         (tp < step && kk == 0) ? 0u : 1u);
                }
                ++pv_cnt[h];
                if (tp + step >= n) mma_commit(BAR(B_OF + h));
                if (frees) mma_commit(BAR(B_KVE + vs));
              }
              if (t < n) {
                const uint32_t ki = base + 2 * t, ks = ki % C::NS;
                ok = mbar_wait(BAR(B_KVF + ks), (ki / C::NS) & 1u, abort_flag, tmo, ecode | 7);
                if (!ok) break;
                tc_fence_after();
                const uint32_t kbase = kv_s0 + ks * C::TILE_BYTES;
                const uint32_t qbase = q_s + (dual ? 0 : h) * C::TILE_BYTES;
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk) {
                  const uint32_t off = (kk >> 2) * C::ATOM_BYTES + (kk & 3) * 32;
                  mma_ss(tmem + h * 128, umma_desc_sw128(qbase + off, 16, 1024),
                         umma_desc_sw128(kbase + off, 16, 1024), IDESC_QK, kk > 0 ? 1u : 0u);
                }
                mma_commit(BAR(B_SF + h));
                if (frees) mma_commit(BAR(B_KVE + ks));
                if (frees && t == n - 1) mma_commit(BAR(B_QE));
              }
            }
          }
          if (!ok) break;
          kv_cnt = base + 2 * n;
          ++n_frag;
        }
        // Every MMA issued so far must finish before TMEM is released.
        mma_commit(BAR(B_DR));
        volatile int never = 0;
        mbar_wait(BAR(B_DR), 0, &never, tmo, ecode | 14);
      }
      __syncwarp();
    } else if (warp == 10) {
      // -------------------------------------------------------------- scheduler
      TreeWalk<C::ROWS> w;
      w.init(p);
      if (lane == 0) {
        TreeFrag f;
        for (uint32_t k = 0;; ++k) {
          const uint32_t e = queue + 64u * (k % C::QD);
          if (!mbar_wait(BAR(B_IE + k % C::QD), ((k / C::QD) & 1u) ^ 1u, abort_flag, tmo,
                         ecode | 17))
            break;
          const bool more = w.next(p, f);
          int flags = 0;
          if (more) {
            sts_s32(e + TQ_B, f.b);
            sts_s32(e + TQ_G, f.g);
            sts_s32(e + TQ_ROW0, f.row0);
            sts_s32(e + TQ_Q0, f.q0);
            sts_s32(e + TQ_NQ, f.nq);
            sts_s32(e + TQ_CTX, f.ctx);
            sts_s32(e + TQ_L, f.L);
            sts_s32(e + TQ_T0, f.t0);
            sts_s32(e + TQ_T1, f.t1);
            flags = TF_LIVE | (f.dual ? TF_DUAL : 0) | (f.whole ? TF_WHOLE : 0) |
                    (f.first ? TF_FIRST : 0);
          }
          sts_s32(e + TQ_FLAGS, flags);
          mbar_arrive(BAR(B_IF + k % C::QD));
          if (!more) break;
        }
      }
      __syncwarp();
    }
    fwd_teardown(warp == 8, tmem, 512);
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::REGS_SOFTMAX));
    // ---------------------------------------------------------------- softmax warpgroups
    const int h = warp >> 2;
    const int wq = warp & 3;
    const int r = threadIdx.x & 127;
    if (h < C::SUBS) {
      const uint32_t t_lane = tmem + (static_cast<uint32_t>(wq * 32) << 16);
      const uint32_t t_s = t_lane + h * 128;
      const uint32_t t_o = t_lane + C::TM_O + h * D;
      float* kpos = reinterpret_cast<float*>(smem + C::SMEM_POS) + warp * 128;
      constexpr float LOG2E = 1.4426950408889634f;
      constexpr float LN2 = 0.6931471805599453f;
      using OutT = typename std::conditional<BF16, __nv_bfloat16, __half>::type;
      const bool al32 = (reinterpret_cast<uintptr_t>(p.out) & 31u) == 0 && (p.dh & 15) == 0;
      FwdParams fp{};
      fp.c1 = p.c1;
      float* ml = reinterpret_cast<float*>(smem + C::SMEM_ML) + 2 * r;
      uint32_t n_frag = 0, tile = 0, ocnt = 0, ocnt1 = 0, mcnt = 0, kv_cnt = 0;
      bool ok = true;
      // This thread's row of the range at queue entry e: token, head, whether there is one.
      auto my_row = [&](uint32_t e, int sub, int& tok, int& head) {
        const int rho = lds_s32(e + TQ_ROW0) + sub * 128 + r;
        const bool live = rho < lds_s32(e + TQ_NQ) * p.R;
        tok = live ? rho / p.R : 0;
        head = lds_s32(e + TQ_G) * p.R + (live ? rho - tok * p.R : 0);
        return live;
      };
      while (ok) {
        const uint32_t e = queue + 64u * (n_frag % C::QD);
        const uint32_t bar_ie = BAR(B_IE + n_frag % C::QD);
        ok = mbar_wait(BAR(B_IF + n_frag % C::QD), (n_frag / C::QD) & 1u, abort_flag, tmo,
                       ecode | 18);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        const int flags = lds_s32(e + TQ_FLAGS);
        if (flags == 0) break;
        const int t1 = lds_s32(e + TQ_T1);
        const int n = t1 - lds_s32(e + TQ_T0);
        const int ctx = lds_s32(e + TQ_CTX);
        const bool dual = (flags & TF_DUAL) != 0;
        const int hq = dual ? 0 : h;  // sub-tile of this warpgroup's rows
        // ---- Q row -> shared memory (128-byte swizzle), once the previous item's Q K^T are done
        ok = mbar_wait(BAR(B_QE), (n_frag & 1u) ^ 1u, abort_flag, tmo, ecode | 2);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        int qtok;  // this row's packed token (what else is needed rarely stays in the queue entry)
        float slope2 = 0.f;
        int pos = 0;
        {
          int tok, head;
          const bool live = my_row(e, hq, tok, head);
          const int q0 = lds_s32(e + TQ_Q0);
          qtok = q0 + tok;
          if constexpr (ALIBI) {
            slope2 = __ldg(p.slopes + head) * LOG2E;
            pos = ctx + tree_depth(p.mask + static_cast<size_t>(qtok) * p.mask_words, p.mask_words,
                                   tok, lds_s32(e + TQ_NQ));
          }
          if (h == hq) {
            const uint4* src = reinterpret_cast<const uint4*>(
                reinterpret_cast<const OutT*>(p.q) +
                (static_cast<size_t>(qtok) * p.hq + head) * p.dh);
            const uint32_t dst = q_s + h * C::TILE_BYTES + static_cast<uint32_t>(r) * 128u;
            const int n16 = p.dh >> 3;
#pragma unroll
            for (int i = 0; i < D / 8; ++i) {
              const uint4 v = (live && i < n16) ? __ldg(src + i) : make_uint4(0u, 0u, 0u, 0u);
              st_shared_v4(dst + (i >> 3) * C::ATOM_BYTES +
                               (static_cast<uint32_t>((i & 7) ^ (r & 7)) << 4),
                           v.x, v.y, v.z, v.w);
            }
            fence_proxy_async_smem();
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(BAR(B_QF));
        ++n_frag;
        const int step = dual ? 2 : 1, jj0 = dual ? h : 0;  // this warpgroup's tiles
        if (jj0 >= n) {  // (the second warpgroup of a single tile)
          kv_cnt += 2 * n;
          if (lane == 0) mbar_arrive(bar_ie);
          continue;
        }
        // Slots past the sequence end may hold anything (0 * NaN is NaN in P V): the first
        // warpgroup zeroes their V rows. V cannot be replaced meanwhile, since its P V waits for this P.
        auto zero_tail = [&](int kv0, uint32_t vi) {
          const uint32_t vst = kv_s0 + (vi % C::NS) * C::TILE_BYTES;
          const int L = lds_s32(e + TQ_L);
          bool good = mbar_wait(BAR(B_KVF + vi % C::NS), (vi / C::NS) & 1u, abort_flag, tmo,
                                ecode | 9);
          good = __all_sync(0xffffffffu, good);
          const int v0 = max(L - kv0, 0);
          for (int i = r; good && i < (128 - v0) * (D / 8); i += 128) {
            const int rr = v0 + i / (D / 8), ch = i % (D / 8);
            st_shared_v4(vst + (ch >> 3) * C::ATOM_BYTES + rr * 128 + ((ch & 7) << 4), 0, 0, 0, 0);
          }
          fence_proxy_async_smem();
          return good;
        };
        // A warp without rows only keeps the pace: no one reads its lanes of P and O. (Its own loop:
        // a branch around the softmax below cost the warps with rows 40 %, in spilled registers.)
        if (lds_s32(e + TQ_ROW0) + hq * 128 + wq * 32 >= lds_s32(e + TQ_NQ) * p.R) {
          for (int jj = jj0; jj < n && ok; jj += step, ++tile) {
            const int kv0 = (t1 - 1 - jj) * 128;
            ok = mbar_wait(BAR(B_SF + h), tile & 1u, abort_flag, tmo, ecode | 8);
            ok = __all_sync(0xffffffffu, ok);
            if (ok && h == 0 && kv0 + 128 > lds_s32(e + TQ_L))
              ok = zero_tail(kv0, kv_cnt + 2 * jj + 1);
            __syncwarp();
            if (ok && lane == 0) mbar_arrive(BAR(B_PF + h));
          }
          kv_cnt += 2 * n;
          const bool second = dual && n > 1;
          if (second && h == 1 && lane == 0 && ok) mbar_arrive(BAR(B_ML));
          if (!(dual && h == 1)) {
            // (O must not be overwritten while the other warps still read it: this warp's word counts
            // as theirs do, and comes after the product that the word is about)
            if (ok) ok = mbar_wait(BAR(B_OF + h), ocnt & 1u, abort_flag, tmo, ecode | 10);
            if (ok && second)
              ok = mbar_wait(BAR(B_OF + 1), ocnt1 & 1u, abort_flag, tmo, ecode | 11) &&
                   mbar_wait(BAR(B_ML), mcnt & 1u, abort_flag, tmo, ecode | 12);
            ok = __all_sync(0xffffffffu, ok);
            if (ok) mbar_arrive(BAR(B_OE + h));
            if (ok && second) {
              mbar_arrive(BAR(B_OE + 1));
              ++mcnt;
            }
            if (second || !dual) ++ocnt1;
          }
          ++ocnt;
          __syncwarp();
          if (lane == 0) mbar_arrive(bar_ie);
          continue;
        }
        float m_ref = -INFINITY, l = 0.f;
        for (int jj = jj0; jj < n; jj += step) {
          const int kv0 = (t1 - 1 - jj) * 128;
          ok = mbar_wait(BAR(B_SF + h), tile & 1u, abort_flag, tmo, ecode | 8);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          tc_fence_after();
          float alpha = 1.f;
          bool resc;
          if (kv0 + 128 <= ctx) {
            resc = fwd_softmax_tile<BF16, ALIBI, ALIBI, false>(
                fp, t_s, kv0, 0x3fffffff, pos, 0x3fffffff, slope2, m_ref, l, alpha);
          } else {
            const int L = lds_s32(e + TQ_L);
            const uint32_t* mrow = p.mask + static_cast<size_t>(qtok) * p.mask_words;
            if constexpr (ALIBI) {
              // Positions of the tile's keys: four per lane, for the whole warp.
              __syncwarp();
#pragma unroll
              for (int u = 0; u < 4; ++u) {
                const int t = kv0 + lane * 4 + u;
                const int j = t - ctx;
                int kp = t;
                if (j >= 0 && t < L)
                  kp = ctx + tree_depth(
                                 p.mask + static_cast<size_t>(lds_s32(e + TQ_Q0) + j) *
                                              p.mask_words,
                                 p.mask_words, j, L - ctx);
                kpos[lane * 4 + u] = static_cast<float>(kp);
              }
              __syncwarp();
            }
            uint32_t view[4];
#pragma unroll
            for (int u = 0; u < 4; ++u)
              view[u] = tree_view(mrow, p.mask_words, kv0 + u * 32, ctx, L);
            resc = tree_masked_tile<BF16, ALIBI>(p.c1, t_s, view, static_cast<float>(pos), slope2,
                                                 kpos, m_ref, l, alpha);
            if (h == 0 && kv0 + 128 > L) {
              ok = zero_tail(kv0, kv_cnt + 2 * jj + 1);
              if (!ok) break;
            }
          }
          // O_h holds the tiles visited before this one, and its last P V has completed (it was
          // issued before this Q K^T).
          if (jj > jj0 && __any_sync(0xffffffffu, resc)) {
#pragma unroll 1
            for (int c4 = 0; c4 < D / 32; ++c4) {
              uint32_t o[32];
              tmem_ld32(t_o + c4 * 32, o);
              tmem_wait_ld();
#pragma unroll
              for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha);
              tmem_st32(t_o + c4 * 32, o);
            }
          }
          tmem_wait_st();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(BAR(B_PF + h));
          ++tile;
        }
        if (!ok) break;
        kv_cnt += 2 * n;
        // ---- epilogue: O / l and the log-sum-exp, to the outputs or to the partials
        if (dual && h == 1) {  // the first warpgroup has the rest
          ml[0] = m_ref;
          ml[1] = l;
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(BAR(B_ML));
            mbar_arrive(bar_ie);
          }
          ++ocnt;  // (the first warpgroup waits for this O)
          continue;
        }
        ok = mbar_wait(BAR(B_OF + h), ocnt & 1u, abort_flag, tmo, ecode | 10);
        const bool joined = dual && n > 1;
        if (joined) {
          if (ok) ok = mbar_wait(BAR(B_OF + 1), ocnt1 & 1u, abort_flag, tmo, ecode | 11);
          if (ok) ok = mbar_wait(BAR(B_ML), mcnt & 1u, abort_flag, tmo, ecode | 12);
        }
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        ++ocnt;
        if (joined || !dual) ++ocnt1;  // phases of the second O's barrier
        tc_fence_after();
        // Weights of this warpgroup's O and, where joined, of the second's.
        float s0 = 1.f, s1 = 0.f;
        if (joined) {
          ++mcnt;
          const float m1 = ml[0], l1 = ml[1];
          const float m = fmaxf(m_ref, m1);
          s0 = m == -INFINITY ? 0.f : ex2_approx(m_ref - m);
          s1 = m == -INFINITY ? 0.f : ex2_approx(m1 - m);
          l = l * s0 + l1 * s1;
          m_ref = m;
        }
        const float inv_l = l > 0.f ? 1.f / l : 0.f;
        const float lse2 = l > 0.f ? m_ref + __log2f(l) : -INFINITY;
        s0 *= inv_l;
        s1 *= inv_l;
        int tok, head;
        const bool live = my_row(e, hq, tok, head);
        const bool whole = (flags & TF_WHOLE) != 0;
        const int q0 = lds_s32(e + TQ_Q0);
        const size_t orow = (static_cast<size_t>(q0 + tok) * p.hq + head) * p.dh;
        __syncwarp();
        if (lane == 0) mbar_arrive(bar_ie);  // the entry has been read
        const size_t slot = (2 * static_cast<size_t>(blockIdx.x) + (flags & TF_FIRST ? 0 : 1)) *
                                C::ROWS + hq * 128 + r;
        if (live) {
          if (!whole)
            p.ws_lse[slot] = lse2;
          else if (p.lse)
            p.lse[static_cast<size_t>(head) * p.total_q + q0 + tok] = lse2 * LN2;
        }
#pragma unroll
        for (int c4 = 0; c4 < D / 32; ++c4) {
          uint32_t o[32];
          uint32_t o1[32];
          tmem_ld32(t_o + c4 * 32, o);
          if (joined) tmem_ld32(t_o + D + c4 * 32, o1);
          tmem_wait_ld();
          if (c4 == D / 32 - 1) {
            // O has been read: it is free for the next item's P V.
            tc_fence_before();
            mbar_arrive(BAR(B_OE + h));
            if (joined) mbar_arrive(BAR(B_OE + 1));
          }
          if (!live) continue;
          if (joined) {
#pragma unroll
            for (int i = 0; i < 32; ++i)
              o[i] = __float_as_uint(__uint_as_float(o[i]) * s0 + __uint_as_float(o1[i]) * s1);
          } else {
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * s0);
          }
          if (whole) {
#pragma unroll
            for (int i = 0; i < 16; ++i)
              o[i] = pack2<BF16>(__uint_as_float(o[2 * i]), __uint_as_float(o[2 * i + 1]));
            OutT* dst = reinterpret_cast<OutT*>(p.out) + orow + c4 * 32;
            const int left = p.dh - c4 * 32;  // columns of this piece that exist
            if (al32) {
              if (left >= 16) st_global_v8(dst, &o[0]);
              if (left >= 32) st_global_v8(dst + 16, &o[8]);
            } else {
#pragma unroll
              for (int i = 0; i < 4; ++i)
                if (left >= 8 * (i + 1))
                  reinterpret_cast<uint4*>(dst)[i] =
                      make_uint4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
            }
          } else {
            float* dst = p.ws_o + slot * D + c4 * 32;
#pragma unroll
            for (int i = 0; i < 4; ++i) st_global_v8(dst + 8 * i, &o[8 * i]);
          }
        }
      }
    }
    __syncwarp();
    fwd_teardown(false, tmem, 512);
  }
#undef BAR
}

// Joins the partials of the items that several CTAs shared. CTA (c, y) looks at the boundary
// between the ranges of CTAs c and c + 1: when an item crosses it and no earlier one, warp w joins
// rows y * 8 + w, ...: out = sum_f 2^(lse_f - M) O_f / sum_f 2^(lse_f - M).
template <int D, bool BF16>
__global__ void __launch_bounds__(256) mea_tree_merge_kernel(const TreeParams p, int grid) {
  using C = TreeCfg<D>;
  constexpr int ROWS = C::ROWS;
  const long long total = tree_total<ROWS>(p);
  const long long per = div_nn(total + grid - 1, grid);
  const long long pos = per * (blockIdx.x + 1);
  long long base = 0, i0 = 0, i1 = 0;  // the item's tiles [i0, i1)
  TreeSeq s{};
  int item = 0;
  bool mine = pos < total;
  if (mine) {
    s = tree_seq<ROWS>(p, tree_find<ROWS>(p, pos, base));
    item = static_cast<int>(div_nn(pos - base, s.tiles));
    i0 = base + static_cast<long long>(item) * s.tiles;
    i1 = i0 + s.tiles;
    mine = i0 < pos && i0 >= pos - per;  // crossed here, and not earlier
  }
  // Up to here nothing that the first kernel writes was read. (Every CTA waits, also those that then
  // have nothing to do: this grid must not end before the first one.)
  pdl_wait();
  if (!mine) return;
  const int c0 = blockIdx.x;
  const int c1 = static_cast<int>(div_nn(i1 - 1, per));  // last CTA with a part
  const int g = item / s.parts;
  const int row0 = (item - g * s.parts) * ROWS;
  const int rows = min(ROWS, s.nq * p.R - row0);
  // CTA c0's part is its first range only when the item starts there; later CTAs' always is.
  const int skip = i0 == pos - per ? 0 : 1;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  using OutT = typename std::conditional<BF16, __nv_bfloat16, __half>::type;
  for (int row = blockIdx.y * 8 + warp; row < rows; row += gridDim.y * 8) {
    auto slot = [&](int c) {
      return (2 * static_cast<size_t>(c) + (c == c0 ? skip : 0)) * ROWS + row;
    };
    float M = -INFINITY;
    for (int c = c0 + lane; c <= c1; c += 32) M = fmaxf(M, p.ws_lse[slot(c)]);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, off));
    float z = 0.f;
    float acc[D / 32];
#pragma unroll
    for (int i = 0; i < D / 32; ++i) acc[i] = 0.f;
    if (M != -INFINITY) {
#pragma unroll 4
      for (int c = c0; c <= c1; ++c) {
        const float wt = ex2_approx(p.ws_lse[slot(c)] - M);
        z += wt;
        const float* o = p.ws_o + slot(c) * D + lane;
#pragma unroll
        for (int i = 0; i < D / 32; ++i) acc[i] = fmaf(wt, o[i * 32], acc[i]);
      }
    }
    const float inv = z > 0.f ? 1.f / z : 0.f;
    const int rho = row0 + row;
    const int tok = rho / p.R, head = g * p.R + rho % p.R;
    OutT* dst = reinterpret_cast<OutT*>(p.out) +
                (static_cast<size_t>(s.q0 + tok) * p.hq + head) * p.dh;
#pragma unroll
    for (int i = 0; i < D / 32; ++i)
      if (i * 32 + lane < p.dh) dst[i * 32 + lane] = static_cast<OutT>(acc[i] * inv);
    if (lane == 0 && p.lse)
      p.lse[static_cast<size_t>(head) * p.total_q + s.q0 + tok] =
          z > 0.f ? (M + __log2f(z)) * 0.6931471805599453f : -INFINITY;
  }
}

}  // namespace mea
