// weights_sm100.cuh — the attention weight that a prompt's queries put on its keys, for sm_100a.
//
//     w[s, g, j] = sum over heads h of KV group g, sum over queries i of
//                  exp(scale q_hi . k_gj + bias - lse_hi)
//
// with the forward's masks, ALiBi and log-sum-exps; only a prompt's last `last` queries count where
// that is given. The score matrix is recomputed tile by tile and never stored.
//
// The scores are computed transposed, S^T = K Q^T (tcgen05, M = 128 keys, N = 128 columns), so that a
// key is a TMEM lane and a thread's sum over the columns needs no other thread. A column is a (query,
// head) pair: a Q tile holds 128 / P queries of P heads of one KV group (P the largest power of two
// that divides the group), so that a short window of queries fills the tile with heads, and a causal
// diagonal wastes 128 / P columns, not 128.
//
// An item is (segment, KV head, KT keys): its K tiles stay in shared memory (the next item's arrive
// meanwhile) and its Q tiles stream past, one a step; SUBS key tiles share each Q tile, since one
// would need half again the L2's bandwidth to keep up. All items' steps form one line, cut into equal
// ranges, one per persistent CTA (a causal prompt's early keys have the most steps, and a short
// window has few items; both load every SM alike). A range that covers part of an item leaves its
// sums in the workspace and a second kernel adds them in order: every sum has one order, so the
// result is deterministic.
//
// Roles: warp 16 the tcgen05 issuer, warp 17 the TMA producer, warp 18 the columns' terms (log-sum-exp
// and ALiBi), warp 19 the schedule (it hands the CTA's ranges, decoded, to the others through a small
// queue in shared memory: walked by every warp, the line cost a short range's warps more than its
// exponentials), warpgroups 0-3 the sums: warpgroup w takes key tile w % SUBS of every NBUF-th step (a
// step costs a warp about 100 instructions beside its columns', so half tiles of every step are
// slower).
//
// Bound by the exponentials: a score costs 2 D flop on the tensor cores and one exp2, and an SM does
// 16 exp2 a clock: 1024 clocks for a 128 x 128 tile. Its product is not far behind: eight 128 x 128 x
// 16 instructions at D = 128, 108 clocks each with both operands in shared memory (64 at the pipe's
// peak), are 864. (A quarter to three eighths of the exponentials by a polynomial on the FMA pipes took
// fewer clocks and as much time or more: the card is at its power limit here, and the longer
// instruction stream lowers the clock.)
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "ptx.cuh"

namespace mea {

struct WeightsParams {
  const float* lse;  // [hq, total_q]
  const int32_t* cu_q;
  const int32_t* cu_k;
  const float* slopes;
  float* weights;    // [n_seqs, hkv, w_stride]
  float* ws;         // [2 grid, KT] sums of the ranges that cover part of an item
  long long w_stride;
  int n_seqs, total_q, hq, hkv, R, last;
  int log2_p;        // P = 1 << log2_p heads in a Q tile
  float c1;          // scale * log2(e)
  unsigned long long timeout_ns;
};

template <int D>
struct WeightsCfg {
  static constexpr int SUBS = D == 256 ? 1 : 2;  // 128-key tiles per item
  static constexpr int KT = 128 * SUBS;
  static constexpr int NBUF = 4 / SUBS;          // S buffers (512 TMEM columns), one per step
  static constexpr int ATOMS = D / 64;
  static constexpr uint32_t ATOM_BYTES = 128 * 128;
  static constexpr uint32_t TILE_BYTES = 128 * D * 2;
  static constexpr int NK = D == 256 ? 1 : 2;    // items whose K is in shared memory
  static constexpr int NQ = D == 64 ? 4 : 2;     // Q tiles in the ring
  static constexpr uint32_t SMEM_K = 0;
  static constexpr uint32_t SMEM_Q = NK * SUBS * TILE_BYTES;
  // Column terms, 2 NBUF slots: nl[128], and with ALiBi slopes[128] and (not causal) positions[128];
  // under a causal mask one such nl, slopes for every 32 keys.
  static constexpr int GROUPS = KT / 32;
  static constexpr int SLOT = GROUPS * 256;  // floats
  static constexpr uint32_t SMEM_T = SMEM_Q + NQ * TILE_BYTES;
  static constexpr uint32_t SMEM_SUM = SMEM_T + 2 * NBUF * SLOT * 4;  // 3 warpgroups x 128 floats
  static constexpr uint32_t SMEM_MISC = SMEM_SUM + 3 * 512;
  static constexpr int QD = 4;                   // ranges in the queue, 64 bytes each
  static constexpr uint32_t MISC_QUEUE = 256;
  static constexpr uint32_t SMEM_TOTAL = SMEM_MISC + MISC_QUEUE + QD * 64 + 1024;
  static_assert(SMEM_TOTAL <= 232448, "shared memory per CTA");
  static constexpr int THREADS = 640;
  // Launched at 96 registers a thread (640 x 96 = 61440): the warps beside the sums give theirs down
  // to REGS_OTHER, and 512 * REGS_SUM + 128 * REGS_OTHER must not exceed 61440.
  static constexpr int REGS_SUM = 104;
  static constexpr int REGS_OTHER = 64;
  static_assert(512 * REGS_SUM + 128 * REGS_OTHER <= 640 * 96, "register split");
};

// A CTA's range of one item's steps.
struct WeightsFrag {
  int seg, g, q0, lq, k0, lk, j0;  // segment, KV head, its rows, first key
  int qbeg, nt;                    // first query, Q tiles per head block
  int s0, s1;                      // steps [s0, s1); step s is head block s / nt, Q tile s % nt
  bool whole, first;
};

// A range in the queue, as 32-bit words (flags 0 ends the list).
struct WeightsEntry {
  int seg, g, q0, lq, k0, lk, j0, qbeg, nt, s0, s1, flags;
};
enum : int { WF_LIVE = 1, WF_WHOLE = 2, WF_FIRST = 4 };

// A segment's items: items before n0 have queries [qw, lq) and nt0 Q tiles; under a causal mask those
// from n0 on start at their first key's own query, and have a - kt * (KT / QT) Q tiles (KT is a
// multiple of a Q tile's QT queries, so the tile counts fall in equal steps).
struct WeightsSeq {
  int q0, lq, k0, lk, items, n0, nt0, a, qw;
  long long work;  // steps of the segment's items of one KV head
};

// Steps per head block before item kt.
template <int KT>
__device__ __forceinline__ long long weights_before(const WeightsParams& p, const WeightsSeq& s,
                                                    int kt) {
  if (kt <= s.n0) return static_cast<long long>(kt) * s.nt0;
  const int drop = KT >> (7 - p.log2_p);  // KT / QT
  const long long m = kt - s.n0;
  return static_cast<long long>(s.n0) * s.nt0 + m * s.a - drop * ((s.n0 + kt - 1) * m / 2);
}

template <int KT, bool CAUSAL>
__device__ __forceinline__ WeightsSeq weights_seq(const WeightsParams& p, int seg) {
  WeightsSeq s;
  s.q0 = __ldg(p.cu_q + seg);
  s.lq = max(__ldg(p.cu_q + seg + 1) - s.q0, 0);
  s.k0 = __ldg(p.cu_k + seg);
  s.lk = max(__ldg(p.cu_k + seg + 1) - s.k0, 0);
  s.items = (s.lk + KT - 1) / KT;
  const int lqt = 7 - p.log2_p, qt1 = (1 << lqt) - 1;
  s.qw = p.last > 0 ? max(s.lq - p.last, 0) : 0;
  // (an item that no query sees still has a step, which finds nothing, so that zeros are written)
  s.nt0 = max((s.lq - s.qw + qt1) >> lqt, 1);
  s.a = (s.lk + qt1) >> lqt;
  s.n0 = s.items;
  if (CAUSAL) {
    const int first = s.qw + s.lk - s.lq;  // key position of the first query that counts
    s.n0 = first < 0 ? 0 : min(first / KT + 1, s.items);
  }
  s.work = weights_before<KT>(p, s, s.items) * (p.R >> p.log2_p);
  return s;
}

// Warp-cooperative: steps of all segments (all KV heads).
template <int KT, bool CAUSAL>
__device__ __forceinline__ long long weights_total(const WeightsParams& p) {
  long long acc = 0;
  for (int s = threadIdx.x & 31; s < p.n_seqs; s += 32)
    acc += weights_seq<KT, CAUSAL>(p, s).work * p.hkv;
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, off);
  return acc;
}

// Warp-cooperative: the segment that step `pos` of the line belongs to, and its first step.
template <int KT, bool CAUSAL>
__device__ __forceinline__ int weights_find(const WeightsParams& p, long long pos,
                                            long long& base) {
  const int lane = threadIdx.x & 31;
  long long acc = 0;
  for (int b0 = 0; b0 < p.n_seqs; b0 += 32) {
    const long long w =
        b0 + lane < p.n_seqs ? weights_seq<KT, CAUSAL>(p, b0 + lane).work * p.hkv : 0;
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

// A CTA's walk over its range of the line (segments, then KV heads, then items).
template <int KT, bool CAUSAL>
struct WeightsWalk {
  long long pos, end, start, base;  // base: first step of item (seg, g, kt)
  int seg, g, kt, qbeg, nt, len;    // len: steps of the item
  WeightsSeq s;
  __device__ __forceinline__ void load_item(const WeightsParams& p) {
    nt = kt < s.n0 ? s.nt0 : s.a - kt * (KT >> (7 - p.log2_p));
    qbeg = kt < s.n0 ? s.qw : kt * KT - (s.lk - s.lq);
    len = nt * (p.R >> p.log2_p);
  }
  // Moves to the item that holds step `pos` (at or after the current one).
  __device__ __forceinline__ void advance(const WeightsParams& p) {
    while (pos >= base + len) {
      base += len;
      if (++kt == s.items) {
        kt = 0;
        if (++g == p.hkv) {
          g = 0;
          do s = weights_seq<KT, CAUSAL>(p, ++seg);
          while (s.items == 0);  // (ends: pos lies before the line's end)
        }
      }
      load_item(p);
    }
  }
  __device__ __forceinline__ void init(const WeightsParams& p, int grid, int cta) {
    const long long total = weights_total<KT, CAUSAL>(p);
    const long long per = div_nn(total + grid - 1, grid);
    start = pos = per * cta;
    end = min(total, pos + per);
    if (pos >= end) return;
    seek(p, pos);
  }
  __device__ __forceinline__ void seek(const WeightsParams& p, long long at) {
    pos = at;
    seg = weights_find<KT, CAUSAL>(p, at, base);
    s = weights_seq<KT, CAUSAL>(p, seg);
    g = static_cast<int>(div_nn(at - base, s.work));
    base += s.work * g;
    // The last item that starts at or before `at`.
    const int hbn = p.R >> p.log2_p;
    int lo = 0, hi = s.items - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (weights_before<KT>(p, s, mid) * hbn <= at - base)
        lo = mid;
      else
        hi = mid - 1;
    }
    kt = lo;
    base += weights_before<KT>(p, s, kt) * hbn;
    load_item(p);
  }
  __device__ __forceinline__ bool next(const WeightsParams& p, WeightsFrag& f) {
    if (pos >= end) return false;
    advance(p);
    f.seg = seg;
    f.g = g;
    f.q0 = s.q0;
    f.lq = s.lq;
    f.k0 = s.k0;
    f.lk = s.lk;
    f.j0 = kt * KT;
    f.qbeg = qbeg;
    f.nt = nt;
    f.s0 = static_cast<int>(pos - base);
    f.s1 = static_cast<int>(min(static_cast<long long>(len), f.s0 + (end - pos)));
    f.whole = f.s0 == 0 && f.s1 == len;
    f.first = pos == start;
    pos += f.s1 - f.s0;
    return true;
  }
};

// Adds 2^score over 32 columns of one key to acc. x: the raw products; terms: shared memory, this
// chunk's column terms (nl, and with ALiBi the slopes and, non-causal, the queries' positions); key:
// the key's index in the item (causal: from the middle of its warp's 32). EDGE: only the columns whose bit of `live` is set count.
template <bool CAUSAL, bool ALIBI, bool EDGE>
__device__ __forceinline__ void weights_chunk(const uint32_t (&x)[32], const float* terms,
                                              uint64_t c1x2, float key, uint32_t live,
                                              uint64_t (&acc)[4]) {
  const uint64_t keyx2 = f2_pack(key, key);
#pragma unroll
  for (int i = 0; i < 32; i += 4) {
    const ulonglong2 nl2 = *reinterpret_cast<const ulonglong2*>(terms + i);
    const uint64_t nl[2] = {nl2.x, nl2.y};
    uint64_t sl[2] = {0ull, 0ull}, ps[2] = {0ull, 0ull};
    if constexpr (ALIBI) {
      const ulonglong2 v = *reinterpret_cast<const ulonglong2*>(terms + 128 + i);
      sl[0] = v.x;
      sl[1] = v.y;
    }
    if constexpr (ALIBI && !CAUSAL) {
      const ulonglong2 v = *reinterpret_cast<const ulonglong2*>(terms + 256 + i);
      ps[0] = v.x;
      ps[1] = v.y;
    }
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int c = i + 2 * u;
      uint64_t e = f2_fma(f2_pack(__uint_as_float(x[c]), __uint_as_float(x[c + 1])), c1x2, nl[u]);
      if constexpr (ALIBI && CAUSAL) e = f2_fma(sl[u], keyx2, e);
      if constexpr (ALIBI && !CAUSAL) {
        float p0, p1;
        f2_unpack(ps[u], p0, p1);
        e = f2_fma(sl[u], f2_pack(-fabsf(p0 - key), -fabsf(p1 - key)), e);
      }
      float w0, w1;
      f2_unpack(e, w0, w1);
      w0 = ex2_approx(w0);
      w1 = ex2_approx(w1);
      if constexpr (EDGE) {  // (a column that does not count may hold anything)
        w0 = (live >> c) & 1u ? w0 : 0.f;
        w1 = (live >> (c + 1)) & 1u ? w1 : 0.f;
      }
      acc[(i >> 1 & 2) + u] = f2_add(acc[(i >> 1 & 2) + u], f2_pack(w0, w1));
    }
  }
}

// Bits [lo, hi) of a chunk of 32 (either end may lie outside it).
__device__ __forceinline__ uint32_t weights_live(int lo, int hi) {
  const uint32_t below = hi >= 32 ? 0xFFFFFFFFu : hi <= 0 ? 0u : (1u << hi) - 1u;
  return lo >= 32 ? 0u : lo <= 0 ? below : below & (0xFFFFFFFFu << lo);
}

template <int D, bool BF16, bool CAUSAL, bool ALIBI>
__global__ void __launch_bounds__(640, 1)
    mea_weights_sm100_kernel(const __grid_constant__ CUtensorMap tm_q,
                             const __grid_constant__ CUtensorMap tm_k, const WeightsParams p) {
  using C = WeightsCfg<D>;
  constexpr float LOG2E = 1.4426950408889634f;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  const uint32_t pad = (1024u - (smem_u32(smem_raw) & 1023u)) & 1023u;
  uint8_t* smem = smem_raw + pad;
  const uint32_t sbase = smem_u32(smem);
  constexpr int B_KF = 0, B_KE = B_KF + C::NK, B_QF = B_KE + C::NK, B_QE = B_QF + C::NQ;
  constexpr int B_SF = B_QE + C::NQ, B_SE = B_SF + 4, B_CF = B_SE + 4;  // S: per (buffer, tile)
  constexpr int B_CE = B_CF + 1, B_IF = B_CE + 1, B_IE = B_IF + C::QD, B_DR = B_IE + C::QD;
  constexpr int N_BARS = B_DR + 1;
  static_assert(8 * N_BARS + 8 <= C::MISC_QUEUE, "barrier region");
  const uint32_t bar0 = sbase + C::SMEM_MISC;
#define BAR(i) (bar0 + 8u * static_cast<uint32_t>(i))
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::SMEM_MISC + 8 * N_BARS);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const uint64_t tmo = p.timeout_ns;
  const unsigned ecode = KID_WEIGHTS << 8;
  if (threadIdx.x == 0) {
    for (int s = 0; s < C::NK; ++s) {
      mbar_init(BAR(B_KF + s), 1);
      mbar_init(BAR(B_KE + s), 1);
    }
    for (int s = 0; s < C::NQ; ++s) {
      mbar_init(BAR(B_QF + s), 1);
      mbar_init(BAR(B_QE + s), 1);
    }
    for (int s = 0; s < 4; ++s) {
      mbar_init(BAR(B_SF + s), 2);  // the step's products, and its column terms
      mbar_init(BAR(B_SE + s), 4);  // one elected arrival per warp that reads the buffer
    }
    mbar_init(BAR(B_CF), 4 * (4 - C::SUBS));  // warps of the buffers after the first
    mbar_init(BAR(B_CE), 4 * C::SUBS);        // warps of the first buffer
    for (int s = 0; s < C::QD; ++s) {
      mbar_init(BAR(B_IF + s), 1);
      mbar_init(BAR(B_IE + s), 19);  // one elected lane of every other warp
    }
    mbar_init(BAR(B_DR), 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 16) {
    tmem_alloc(smem_u32(tmem_slot), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  bool ok = true;
  pdl_trigger();
  volatile WeightsEntry* queue = reinterpret_cast<volatile WeightsEntry*>(
      smem + C::SMEM_MISC + C::MISC_QUEUE);
  static_assert(sizeof(WeightsEntry) <= 64, "queue entry");
  // Range `i` of the CTA, once it is there (null: the end of the list, or a wait that gave up); for
  // one lane, or with `warp_wide` for a whole warp alike.
  auto range = [&](uint32_t i, bool warp_wide) {
    ok = mbar_wait(BAR(B_IF + i % C::QD), (i / C::QD) & 1u, abort_flag, tmo, ecode | 11);
    if (warp_wide) ok = __all_sync(0xffffffffu, ok);
    volatile WeightsEntry* e = reinterpret_cast<volatile WeightsEntry*>(
        reinterpret_cast<volatile uint8_t*>(queue) + 64u * (i % C::QD));
    return ok && e->flags != 0 ? e : nullptr;
  };

  if (warp >= 16)
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::REGS_OTHER));
  else
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::REGS_SUM));
  if (warp == 17) {
    // ---------------------------------------------------------------- TMA producer
    if (lane == 0) {
      uint32_t n_frag = 0, k = 0;
      while (volatile WeightsEntry* e = range(n_frag, false)) {
        const int g = e->g, q_row = e->q0 + e->qbeg, k_row = e->k0 + e->j0, nt = e->nt;
        const int s0 = e->s0, s1 = e->s1;
        const bool none = e->qbeg >= e->lq;  // no query: the step's columns may hold anything
        mbar_arrive(BAR(B_IE + n_frag % C::QD));
        const uint32_t kb = n_frag % C::NK;
        ok = mbar_wait(BAR(B_KE + kb), ((n_frag / C::NK) & 1u) ^ 1u, abort_flag, tmo, ecode | 1);
        if (!ok) break;
        mbar_arrive_expect_tx(BAR(B_KF + kb), C::SUBS * C::TILE_BYTES);
#pragma unroll
        for (int h = 0; h < C::SUBS; ++h)
#pragma unroll
          for (int a = 0; a < C::ATOMS; ++a)
            tma_load_3d(sbase + C::SMEM_K + (kb * C::SUBS + h) * C::TILE_BYTES + a * C::ATOM_BYTES,
                        &tm_k, BAR(B_KF + kb), a * 64, g, k_row + h * 128);
        ++n_frag;
        int hb = s0 / nt, t = s0 - hb * nt;
        for (int st = s0; st < s1; ++st, ++k) {
          const uint32_t s = k % C::NQ;
          ok = mbar_wait(BAR(B_QE + s), ((k / C::NQ) & 1u) ^ 1u, abort_flag, tmo, ecode | 2);
          if (!ok) break;
          if (none) {
            mbar_arrive(BAR(B_QF + s));
            continue;
          }
          mbar_arrive_expect_tx(BAR(B_QF + s), C::TILE_BYTES);
#pragma unroll
          for (int a = 0; a < C::ATOMS; ++a)
            tma_load_3d(sbase + C::SMEM_Q + s * C::TILE_BYTES + a * C::ATOM_BYTES, &tm_q,
                        BAR(B_QF + s), a * 64, g * p.R + (hb << p.log2_p),
                        q_row + t * (128 >> p.log2_p));
          if (++t == nt) {
            t = 0;
            ++hb;
          }
        }
        if (!ok) break;
      }
      if (!ok) {
        // Let the loads already issued land before the CTA's shared memory goes away.
        volatile int never = 0;
        for (uint32_t s = 0; s < C::NQ && s < k; ++s) {
          const uint32_t last = k - 1 - ((k - 1 - s) % C::NQ);
          mbar_wait(BAR(B_QF + s), (last / C::NQ) & 1u, &never, tmo, ecode | 15);
        }
        for (uint32_t s = 0; s < C::NK && s < n_frag; ++s) {
          const uint32_t last = n_frag - 1 - ((n_frag - 1 - s) % C::NK);
          mbar_wait(BAR(B_KF + s), (last / C::NK) & 1u, &never, tmo, ecode | 15);
        }
      }
    }
    __syncwarp();
  } else if (warp == 16) {
    // ---------------------------------------------------------------- tcgen05 issuer
    if (lane == 0) {
      constexpr uint32_t IDESC = umma_idesc_f16(BF16, 128, 128, false, false);
      uint32_t n_frag = 0, k = 0;
      while (volatile WeightsEntry* e = range(n_frag, false)) {
        const int s0 = e->s0, s1 = e->s1;
        mbar_arrive(BAR(B_IE + n_frag % C::QD));
        const uint32_t kb = n_frag % C::NK;
        ok = mbar_wait(BAR(B_KF + kb), (n_frag / C::NK) & 1u, abort_flag, tmo, ecode | 3);
        if (!ok) break;
        ++n_frag;
        for (int st = s0; st < s1; ++st, ++k) {
          const uint32_t s = k % C::NQ, b = k % C::NBUF;
          ok = mbar_wait(BAR(B_QF + s), (k / C::NQ) & 1u, abort_flag, tmo, ecode | 4);
          if (!ok) break;
          const uint32_t qb = sbase + C::SMEM_Q + s * C::TILE_BYTES;
#pragma unroll
          for (int h = 0; h < C::SUBS; ++h) {
            ok = mbar_wait_spin(BAR(B_SE + b * C::SUBS + h), ((k / C::NBUF) & 1u) ^ 1u, abort_flag,
                                tmo, ecode | 5);
            if (!ok) break;
            tc_fence_after();
            const uint32_t kbase = sbase + C::SMEM_K + (kb * C::SUBS + h) * C::TILE_BYTES;
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
              const uint32_t o = (kk >> 2) * C::ATOM_BYTES + (kk & 3) * 32;
              mma_ss(tmem + (b * C::SUBS + h) * 128, umma_desc_sw128(kbase + o, 16, 1024),
                     umma_desc_sw128(qb + o, 16, 1024), IDESC, kk > 0 ? 1u : 0u);
            }
            mma_commit(BAR(B_SF + b * C::SUBS + h));
          }
          if (!ok) break;
          mma_commit(BAR(B_QE + s));
          if (st == s1 - 1) mma_commit(BAR(B_KE + kb));
        }
        if (!ok) break;
      }
      // Every MMA issued so far must finish before TMEM is released.
      mma_commit(BAR(B_DR));
      volatile int never = 0;
      mbar_wait(BAR(B_DR), 0, &never, tmo, ecode | 14);
    }
    __syncwarp();
  } else if (warp == 18) {
    // ---------------------------------------------------------------- column terms
    //   nl[c] = -lse2, sl[c] = slope2, ps[c] = p_c - j0. Under a causal mask the distance term is
    //   split, slope2 (key - m) - slope2 (p_c - m), and its second half added here, so that a thread
    //   loads two terms a column and not three (the loads take as long as the exponentials then: 32.4
    //   us instead of 27.9 for the last 32 queries of 16 prompts). m is the middle of the 32 keys of
    //   the key's warp: where a weight counts, both halves are within slope2 * 16 of the whole, and
    //   so is their rounding. (With m the item's first key, up to 255 slope2 away, weights were off
    //   by 2e-4 under slopes of 16.)
    uint32_t n_frag = 0, k = 0;
    while (volatile WeightsEntry* e = range(n_frag, true)) {
      const int g = e->g, q0 = e->q0, lq = e->lq, qbeg = e->qbeg, nt = e->nt;
      const int s0 = e->s0, s1 = e->s1, pos0 = e->lk - lq - e->j0;
      __syncwarp();
      if (lane == 0) mbar_arrive(BAR(B_IE + n_frag % C::QD));
      ++n_frag;
      int hb = s0 / nt, t = s0 - hb * nt;
      for (int st = s0; st < s1; ++st, ++k) {
        const uint32_t b = k % C::NBUF;
        float nl[4], sl[4], ps[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          // (where a table goes to every 32 keys, a lane has four columns next to each other)
          const int c = ALIBI && CAUSAL ? 4 * lane + u : u * 32 + lane;
          const int i = qbeg + t * (128 >> p.log2_p) + (c >> p.log2_p);
          const int head = g * p.R + (hb << p.log2_p) + (c & ((1 << p.log2_p) - 1));
          nl[u] = -INFINITY;
          sl[u] = ps[u] = 0.f;
          if (i < lq) {
            nl[u] = -LOG2E * __ldg(p.lse + static_cast<size_t>(head) * p.total_q + q0 + i);
            if (nl[u] == INFINITY) nl[u] = -INFINITY;  // (a row that attends to nothing)
            if constexpr (ALIBI) {
              sl[u] = __ldg(p.slopes + head) * LOG2E;
              ps[u] = static_cast<float>(i + pos0);
            }
          }
        }
        if (lane < C::SUBS)
          ok = mbar_wait(BAR(B_SE + b * C::SUBS + lane), ((k / C::NBUF) & 1u) ^ 1u, abort_flag, tmo,
                         ecode | 6);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        float* dst = reinterpret_cast<float*>(smem + C::SMEM_T) + (k % (2 * C::NBUF)) * C::SLOT;
        if constexpr (ALIBI && CAUSAL) {
          float4* dst4 = reinterpret_cast<float4*>(dst) + lane;
#pragma unroll
          for (int m = 0; m < C::GROUPS; ++m) {
            const float mid = m * 32 + 16;
            dst4[m * 64] = make_float4(fmaf(-sl[0], ps[0] - mid, nl[0]),
                                      fmaf(-sl[1], ps[1] - mid, nl[1]),
                                      fmaf(-sl[2], ps[2] - mid, nl[2]),
                                      fmaf(-sl[3], ps[3] - mid, nl[3]));
            dst4[m * 64 + 32] = make_float4(sl[0], sl[1], sl[2], sl[3]);
          }
        } else {
          dst += lane;
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            dst[u * 32] = nl[u];
            if constexpr (ALIBI) {
              dst[128 + u * 32] = sl[u];
              dst[256 + u * 32] = ps[u];
            }
          }
        }
        __syncwarp();
        if (lane < C::SUBS) mbar_arrive(BAR(B_SF + b * C::SUBS + lane));
        if (++t == nt) {
          t = 0;
          ++hb;
        }
      }
      if (!ok) break;
    }
  } else if (warp == 19) {
    // ---------------------------------------------------------------- schedule
    WeightsWalk<C::KT, CAUSAL> w;
    w.init(p, gridDim.x, blockIdx.x);
    if (lane == 0) {
      WeightsFrag f;
      for (uint32_t i = 0;; ++i) {
        if (!mbar_wait(BAR(B_IE + i % C::QD), ((i / C::QD) & 1u) ^ 1u, abort_flag, tmo, ecode | 12))
          break;
        volatile WeightsEntry* e = reinterpret_cast<volatile WeightsEntry*>(
            reinterpret_cast<volatile uint8_t*>(queue) + 64u * (i % C::QD));
        const bool more = w.next(p, f);
        if (more) {
          e->seg = f.seg;
          e->g = f.g;
          e->q0 = f.q0;
          e->lq = f.lq;
          e->k0 = f.k0;
          e->lk = f.lk;
          e->j0 = f.j0;
          e->qbeg = f.qbeg;
          e->nt = f.nt;
          e->s0 = f.s0;
          e->s1 = f.s1;
        }
        e->flags = more ? WF_LIVE | (f.whole ? WF_WHOLE : 0) | (f.first ? WF_FIRST : 0) : 0;
        mbar_arrive(BAR(B_IF + i % C::QD));
        if (!more) break;
      }
    }
    __syncwarp();
  } else if (warp < 16) {
    // ---------------------------------------------------------------- sums (thread = key)
    const int wg = warp >> 2;
    const int h = wg % C::SUBS, buf = wg / C::SUBS;
    const int r = threadIdx.x & 127;
    const uint32_t t_s = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16) +
                         (buf * C::SUBS + h) * 128;
    // This warp's column terms: two slots per buffer, in turn.
    const float* terms0 = reinterpret_cast<const float*>(smem + C::SMEM_T) + buf * C::SLOT +
                          (ALIBI && CAUSAL ? (h * 4 + (warp & 3)) * 256 : 0);
    int slot = 0;
    const uint32_t bar_f = BAR(B_SF + wg), bar_e = BAR(B_SE + wg);  // (wg = buf * SUBS + h)
    const uint64_t c1x2 = f2_pack(p.c1, p.c1);
    const float key = static_cast<float>(CAUSAL ? lane - 16 : h * 128 + r);
    float* sums = reinterpret_cast<float*>(smem + C::SMEM_SUM);
    uint32_t n_frag = 0, n_join = 0, phase = 0;
    int ahead = buf;  // steps until this warpgroup's next one
    while (volatile WeightsEntry* e = range(n_frag, true)) {
      const uint32_t bar_ie = BAR(B_IE + n_frag % C::QD);
      ++n_frag;
      float sum = 0.f, comp = 0.f;  // running sum and what it lost
      const int s0 = e->s0, s1 = e->s1, nt = e->nt, qbeg = e->qbeg;
      const int j = e->j0 + h * 128 - (e->lk - e->lq) - qbeg;  // first key, counted in queries
      const int left = e->lq - qbeg;
      int t = (s0 + ahead) % nt;
      int n = s1 - s0 - ahead;
      const bool mine = n > 0;
      for (; n > 0; n -= C::NBUF) {
        const int qi = t << (7 - p.log2_p);  // first query of the tile
        t += C::NBUF;
        while (t >= nt) t -= nt;
        // Columns [lo, hi) count for this key; every key of the tile sees all 128 off the edges.
        const int hi = min(left - qi, 128) << p.log2_p;
        const bool edge = hi < 128 || (CAUSAL && qi < j + 127);
        ok = mbar_wait(bar_f, phase, abort_flag, tmo, ecode | 8);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        phase ^= 1u;
        const float* terms = terms0 + slot;
        slot = C::NBUF * C::SLOT - slot;
        tc_fence_after();
        uint64_t acc[4] = {0ull, 0ull, 0ull, 0ull};
        // 32 columns at a time; once the last ones are in registers the buffer is free, and the next
        // product runs under their exponentials.
        auto load = [&](int c, uint32_t (&x)[32]) {
          tmem_ld32(t_s + c, x);
          tmem_wait_ld();
          if (c == 96) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar_e);
          }
        };
        if (!edge) {
#pragma unroll 1
          for (int c = 0; c < 128; c += 32) {
            uint32_t x[32];
            load(c, x);
            weights_chunk<CAUSAL, ALIBI, false>(x, terms + c, c1x2, key, 0u, acc);
          }
        } else {
          const int lo = CAUSAL ? max(j + r - qi, 0) << p.log2_p : 0;
#pragma unroll 1
          for (int c = 0; c < 128; c += 32) {
            uint32_t x[32];
            load(c, x);
            const uint32_t live = weights_live(lo - c, hi - c);
            // (columns that no key of the warp counts are left out)
            if (__any_sync(0xffffffffu, live != 0u))
              weights_chunk<CAUSAL, ALIBI, true>(x, terms + c, c1x2, key, live, acc);
          }
        }
        float a0, a1;
        f2_unpack(f2_add(f2_add(acc[0], acc[1]), f2_add(acc[2], acc[3])), a0, a1);
        // Long prompts add thousands of tile sums: carry the rounding along.
        const float y = (a0 + a1) - comp;
        const float s2 = sum + y;
        comp = (s2 - sum) - y;
        sum = s2;
      }
      ahead = -n;
      if (!ok) break;
      // ---- the warpgroups' sums join, and the item's (or the range's) are written. A range of one
      // step is its warpgroups' alone: the others have gone on.
      const bool solo = s1 - s0 == 1;
      if (solo && !mine) {
        __syncwarp();
        if (lane == 0) mbar_arrive(bar_ie);
        continue;
      }
      if (!solo) {
        if (buf > 0) {
          ok = mbar_wait(BAR(B_CE), (n_join & 1u) ^ 1u, abort_flag, tmo, ecode | 9);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          sums[(wg - C::SUBS) * 128 + r] = sum;
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(BAR(B_CF));
            mbar_arrive(bar_ie);
          }
          ++n_join;
          continue;
        }
        ok = mbar_wait(BAR(B_CF), n_join & 1u, abort_flag, tmo, ecode | 10);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
#pragma unroll
        for (int q = 1; q < C::NBUF; ++q) sum += sums[(q * C::SUBS + h - C::SUBS) * 128 + r];
        __syncwarp();
        if (lane == 0) mbar_arrive(BAR(B_CE));
        ++n_join;
      }
      const int row = h * 128 + r;
      const int flags = e->flags, key0 = e->j0 + row, lk = e->lk;
      const size_t out = (static_cast<size_t>(e->seg) * p.hkv + e->g) * p.w_stride + key0;
      __syncwarp();
      if (lane == 0) mbar_arrive(bar_ie);
      if (!(flags & WF_WHOLE))
        p.ws[(2 * static_cast<size_t>(blockIdx.x) + (flags & WF_FIRST ? 0 : 1)) * C::KT + row] = sum;
      else if (key0 < lk && key0 < p.w_stride)
        p.weights[out] = sum;
    }
  }
#undef BAR
  tc_fence_before();
  __syncthreads();
  if (warp == 16) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// Adds up the sums of the items that several CTAs shared: CTA c looks at the boundary between the
// ranges of CTAs c and c + 1; when an item crosses it and no earlier one, thread = key.
template <int D, bool CAUSAL>
__global__ void __launch_bounds__(WeightsCfg<D>::KT)
    mea_weights_merge_kernel(const WeightsParams p, int grid) {
  constexpr int KT = WeightsCfg<D>::KT;
  pdl_wait();
  const long long total = weights_total<KT, CAUSAL>(p);
  const long long per = div_nn(total + grid - 1, grid);
  const long long pos = per * (blockIdx.x + 1);
  if (pos >= total) return;
  WeightsWalk<KT, CAUSAL> w;
  w.seek(p, pos);
  if (w.base == pos || w.base < pos - per) return;  // not crossed here, or first crossed earlier
  const int c0 = blockIdx.x;
  const int c1 = static_cast<int>(div_nn(w.base + w.len - 1, per));  // last CTA with a part
  // CTA c0's part is its first range only when the item starts there; later CTAs' always is.
  const int skip = w.base == pos - per ? 0 : 1;
  const int row = threadIdx.x;
  float sum = 0.f;
  for (int c = c0; c <= c1; ++c)
    sum += p.ws[(2 * static_cast<size_t>(c) + (c == c0 ? skip : 0)) * KT + row];
  const int j = w.kt * KT + row;
  if (j < w.s.lk && j < p.w_stride)
    p.weights[(static_cast<size_t>(w.seg) * p.hkv + w.g) * p.w_stride + j] = sum;
}

}  // namespace mea
