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
// (tcgen05, fp32 in TMEM), a producer warp. The softmax warps also put Q into shared memory
// (its rows are few and need not be a box of q).
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
  static constexpr uint32_t SMEM_MISC = SMEM_POS + 8 * 512;
  static constexpr uint32_t SMEM_TOTAL = SMEM_MISC + 512 + 1024;
  static_assert(SMEM_TOTAL <= 232448, "shared memory per CTA");
  static constexpr int THREADS = 384;
  static constexpr int REGS_SOFTMAX = 208;
  static constexpr int REGS_OTHER = 80;
  static constexpr uint32_t TM_O = 256;
};

// A CTA's range of one item's tiles.
struct TreeFrag {
  int b, g, row0;        // request, KV head, first row of the item
  int q0, nq, ctx, L;    // first packed token, tokens, context keys, keys
  int t0, t1;            // tiles [t0, t1)
  bool whole;            // the range is the whole item
  bool first;            // the CTA's first range
};

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
    const long long per = (total + gridDim.x - 1) / gridDim.x;
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
    const int item = static_cast<int>(off / s.tiles);
    f.t0 = static_cast<int>(off - static_cast<long long>(item) * s.tiles);
    f.t1 = static_cast<int>(min(static_cast<long long>(s.tiles), f.t0 + (end - pos)));
    f.g = item / s.parts;
    f.row0 = (item - f.g * s.parts) * ROWS;
    f.b = b;
    f.q0 = s.q0;
    f.nq = s.nq;
    f.L = s.L;
    f.ctx = s.L - s.nq;
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
  constexpr int B_PF = B_SF + 2, B_OF = B_PF + 2, B_OE = B_OF + 2, B_DR = B_OE + 2;
  constexpr int N_BARS = B_DR + 1;
  static_assert(8 * N_BARS + 8 <= 512, "barrier region");
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
  pdl_trigger();

  static_assert(256 * C::REGS_SOFTMAX + 128 * C::REGS_OTHER <= 384 * 168, "register split");
  if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::REGS_OTHER));
    if (warp == 9) {
      // -------------------------------------------------------------- TMA producer
      TreeWalk<C::ROWS> w;
      w.init(p);
      TreeFrag f;
      uint32_t cnt = 0;
      bool ok = true;
      // One box of box_rows keys x 64 columns per lane (at most 8 x 4 boxes a tile).
      const int nbox = 128 / p.box_rows * C::ATOMS;
      const int piece = lane / C::ATOMS, atom = lane % C::ATOMS;
      const bool issuer = lane < nbox;
      while (ok && w.next(p, f)) {
        const int32_t* row = p.block_table + static_cast<size_t>(f.b) * p.max_blocks;
        const int nblk = min((f.L + p.block_size - 1) / p.block_size, p.max_blocks);
        const int n = f.t1 - f.t0;
        // Tiles go from the last one down. A block past the request's last one takes id num_blocks,
        // which the TMA fills with zeros; ids are read three tiles ahead of their use.
        auto block_id = [&](int jj) {
          const int blk = ((f.t1 - 1 - jj) * 128 + piece * p.box_rows) / p.block_size;
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
          const int r0 = ((f.t1 - 1 - jj) * 128 + piece * p.box_rows) % p.block_size;
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
                          kv ? &tm_v : &tm_k, BAR(B_KVF + s), atom * 64, f.g, r0, id);
            ++cnt;
          }
        }
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
      TreeWalk<C::ROWS> w;
      w.init(p);
      if (lane == 0) {
        constexpr uint32_t IDESC_QK = umma_idesc_f16(BF16, 128, 128, false, false);
        constexpr uint32_t IDESC_PV = umma_idesc_f16(BF16, 128, D, false, true);
        TreeFrag f;
        uint32_t kv_cnt = 0, n_frag = 0;
        uint32_t pv_cnt[2] = {0, 0}, oe_cnt[2] = {0, 0};
        bool ok = true;
        while (ok && w.next(p, f)) {
          const int n = f.t1 - f.t0;
          const int subs = (C::SUBS == 2 && f.nq * p.R - f.row0 > 128) ? 2 : 1;
          ok = mbar_wait(BAR(B_QF), n_frag & 1u, abort_flag, tmo, ecode | 6);
          if (!ok) break;
          tc_fence_after();
          const uint32_t base = kv_cnt;
          for (int j = 0; j <= n && ok; ++j) {
            const uint32_t ks = (base + 2 * j) % C::NS;
            const uint32_t vs = (base + 2 * j - 1) % C::NS;  // slot of V_{j-1} (j >= 1)
            bool v_ready = false, k_ready = false;
#pragma unroll
            for (int h = 0; h < C::SUBS; ++h) {
              if (h >= subs) break;
              if (j >= 1) {
                // ---- O_h += P_h(j-1) V_{j-1}
                if (!v_ready) {
                  ok = mbar_wait(BAR(B_KVF + vs), ((base + 2 * j - 1) / C::NS) & 1u, abort_flag,
                                 tmo, ecode | 5);
                  if (!ok) break;
                  v_ready = true;
                }
                ok = mbar_wait_spin(BAR(B_PF + h), pv_cnt[h] & 1u, abort_flag, tmo, ecode | 3);
                if (!ok) break;
                if (j == 1) {
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
                         (j == 1 && kk == 0) ? 0u : 1u);
                }
                ++pv_cnt[h];
                if (j == n) mma_commit(BAR(B_OF + h));
              }
              if (j < n) {
                // ---- S_h = Q_h K_j^T
                if (!k_ready) {
                  ok = mbar_wait(BAR(B_KVF + ks), ((base + 2 * j) / C::NS) & 1u, abort_flag, tmo,
                                 ecode | 7);
                  if (!ok) break;
                  tc_fence_after();
                  k_ready = true;
                }
                const uint32_t kbase = kv_s0 + ks * C::TILE_BYTES;
                const uint32_t qbase = q_s + h * C::TILE_BYTES;
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk) {
                  const uint32_t off = (kk >> 2) * C::ATOM_BYTES + (kk & 3) * 32;
                  mma_ss(tmem + h * 128, umma_desc_sw128(qbase + off, 16, 1024),
                         umma_desc_sw128(kbase + off, 16, 1024), IDESC_QK, kk > 0 ? 1u : 0u);
                }
                mma_commit(BAR(B_SF + h));
              }
            }
            if (!ok) break;
            if (j >= 1) mma_commit(BAR(B_KVE + vs));
            if (j < n) mma_commit(BAR(B_KVE + ks));
            if (j == n - 1) mma_commit(BAR(B_QE));
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
      TreeWalk<C::ROWS> w;
      w.init(p);
      TreeFrag f;
      uint32_t n_frag = 0, tile = 0, ocnt = 0, kv_cnt = 0;
      bool ok = true;
      while (ok && w.next(p, f)) {
        const int n = f.t1 - f.t0;
        const int rho = f.row0 + h * 128 + r;
        const bool live = rho < f.nq * p.R;
        const int tok = live ? rho / p.R : 0;
        const int head = f.g * p.R + (live ? rho - tok * p.R : 0);
        const size_t orow = (static_cast<size_t>(f.q0 + tok) * p.hq + head) * p.dh;
        // ---- Q row -> shared memory (128-byte swizzle), once the previous item's Q K^T are done
        ok = mbar_wait(BAR(B_QE), (n_frag & 1u) ^ 1u, abort_flag, tmo, ecode | 2);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        {
          const uint4* src = reinterpret_cast<const uint4*>(
              reinterpret_cast<const OutT*>(p.q) + orow);
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
          __syncwarp();
          if (lane == 0) mbar_arrive(BAR(B_QF));
        }
        ++n_frag;
        const bool active = h == 0 || f.nq * p.R - f.row0 > 128;
        if (!active) {
          kv_cnt += 2 * n;
          continue;
        }
        const uint32_t* mrow = p.mask + static_cast<size_t>(f.q0 + tok) * p.mask_words;
        float slope2 = 0.f;
        int pos = 0;
        if constexpr (ALIBI) {
          slope2 = __ldg(p.slopes + head) * LOG2E;
          pos = f.ctx + tree_depth(mrow, p.mask_words, tok, f.nq);
        }
        float m_ref = -INFINITY, l = 0.f;
        for (int jj = 0; jj < n; ++jj) {
          const int kv0 = (f.t1 - 1 - jj) * 128;
          ok = mbar_wait(BAR(B_SF + h), tile & 1u, abort_flag, tmo, ecode | 8);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          tc_fence_after();
          float alpha = 1.f;
          bool resc;
          if (kv0 + 128 <= f.ctx) {
            resc = fwd_softmax_tile<BF16, ALIBI, ALIBI, false>(
                fp, t_s, kv0, 0x3fffffff, pos, 0x3fffffff, slope2, m_ref, l, alpha);
          } else {
            if constexpr (ALIBI) {
              // Positions of the tile's keys: four per lane, for the whole warp.
              __syncwarp();
#pragma unroll
              for (int u = 0; u < 4; ++u) {
                const int t = kv0 + lane * 4 + u;
                const int j = t - f.ctx;
                int kp = t;
                if (j >= 0 && j < f.nq)
                  kp = f.ctx + tree_depth(p.mask + static_cast<size_t>(f.q0 + j) * p.mask_words,
                                          p.mask_words, j, f.nq);
                kpos[lane * 4 + u] = static_cast<float>(kp);
              }
              __syncwarp();
            }
            uint32_t view[4];
#pragma unroll
            for (int u = 0; u < 4; ++u)
              view[u] = tree_view(mrow, p.mask_words, kv0 + u * 32, f.ctx, f.L);
            resc = tree_masked_tile<BF16, ALIBI>(p.c1, t_s, view, static_cast<float>(pos), slope2,
                                                 kpos, m_ref, l, alpha);
            if (h == 0 && kv0 + 128 > f.L) {
              // Slots past the sequence end may hold anything (0 * NaN is NaN in P V): zero their V
              // rows. V cannot be replaced meanwhile, since its P V waits for this P.
              const uint32_t vi = kv_cnt + 2 * jj + 1;
              const uint32_t vst = kv_s0 + (vi % C::NS) * C::TILE_BYTES;
              ok = mbar_wait(BAR(B_KVF + vi % C::NS), (vi / C::NS) & 1u, abort_flag, tmo,
                             ecode | 9);
              ok = __all_sync(0xffffffffu, ok);
              if (!ok) break;
              const int v0 = max(f.L - kv0, 0);
              for (int i = r; i < (128 - v0) * (D / 8); i += 128) {
                const int rr = v0 + i / (D / 8), ch = i % (D / 8);
                st_shared_v4(vst + (ch >> 3) * C::ATOM_BYTES + rr * 128 + ((ch & 7) << 4), 0, 0, 0,
                             0);
              }
              fence_proxy_async_smem();
            }
          }
          // O_h holds the tiles visited before this one, and its last P V has completed (it was
          // issued before this Q K^T).
          if (jj > 0 && __any_sync(0xffffffffu, resc)) {
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
        ok = mbar_wait(BAR(B_OF + h), ocnt & 1u, abort_flag, tmo, ecode | 10);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        ++ocnt;
        tc_fence_after();
        const float inv_l = l > 0.f ? 1.f / l : 0.f;
        const float lse2 = l > 0.f ? m_ref + __log2f(l) : -INFINITY;
        const size_t slot = (2 * static_cast<size_t>(blockIdx.x) + (f.first ? 0 : 1)) * C::ROWS +
                            h * 128 + r;
        if (live) {
          if (!f.whole)
            p.ws_lse[slot] = lse2;
          else if (p.lse)
            p.lse[static_cast<size_t>(head) * p.total_q + f.q0 + tok] = lse2 * LN2;
        }
#pragma unroll
        for (int c4 = 0; c4 < D / 32; ++c4) {
          uint32_t o[32];
          tmem_ld32(t_o + c4 * 32, o);
          tmem_wait_ld();
          if (c4 == D / 32 - 1) {
            // O_h has been read: it is free for the next item's P V.
            tc_fence_before();
            mbar_arrive(BAR(B_OE + h));
          }
          if (!live) continue;
          if (f.whole) {
#pragma unroll
            for (int i = 0; i < 16; ++i)
              o[i] = pack2<BF16>(__uint_as_float(o[2 * i]) * inv_l,
                                 __uint_as_float(o[2 * i + 1]) * inv_l);
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
#pragma unroll
            for (int i = 0; i < 32; ++i)
              o[i] = __float_as_uint(__uint_as_float(o[i]) * inv_l);
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
  pdl_wait();
  const long long total = tree_total<ROWS>(p);
  const long long per = (total + grid - 1) / grid;
  const long long pos = per * (blockIdx.x + 1);
  if (pos >= total) return;
  long long base = 0;
  const int b = tree_find<ROWS>(p, pos, base);
  const TreeSeq s = tree_seq<ROWS>(p, b);
  const int item = static_cast<int>((pos - base) / s.tiles);
  const long long i0 = base + static_cast<long long>(item) * s.tiles;  // the item's tiles
  const long long i1 = i0 + s.tiles;
  if (i0 == pos || i0 < pos - per) return;  // not crossed here, or first crossed earlier
  const int c0 = blockIdx.x;
  const int c1 = static_cast<int>((i1 - 1) / per);  // last CTA with a part
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
