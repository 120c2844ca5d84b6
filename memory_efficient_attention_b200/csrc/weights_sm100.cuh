// weights_sm100.cuh — the attention weight that a prompt's queries put on its keys, for sm_100a.
//
//     w[s, g, j] = sum over heads h of KV group g, sum over queries i of
//                  exp(scale q_hi . k_gj + bias - lse_hi)
//
// with the forward's masks, ALiBi and log-sum-exps; only a prompt's last `last` queries count where
// that is given. The score matrix is recomputed tile by tile and never stored.
//
// One CTA per (key tile of 128, KV head, segment): the scores are computed transposed, S^T = K Q^T
// (tcgen05, M = 128 keys, N = 128 queries), so that a key is a TMEM lane and a thread's sum over
// the queries needs no other thread. K stays in shared memory, Q tiles of the group's heads stream
// past it. Two warpgroups take the steps in turn, one S buffer each; every sum has one order, so
// the result is deterministic.
//
// Bound by the exponentials: a score costs 2 D flop on the tensor cores and one exp2, and an SM
// does 16 exp2 a clock (1024 clocks for a 128 x 128 tile, whose product takes a quarter of that at
// D = 128).
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
  long long w_stride;
  int n_seqs, total_q, hq, hkv, R, last;
  float c1;          // scale * log2(e)
  unsigned long long timeout_ns;
};

template <int D>
struct WeightsCfg {
  static constexpr int ATOMS = D / 64;
  static constexpr uint32_t ATOM_BYTES = 128 * 128;
  static constexpr uint32_t TILE_BYTES = 128 * D * 2;
  static constexpr int NQ = 2;  // Q tiles in the ring
  static constexpr uint32_t SMEM_K = 0;
  static constexpr uint32_t SMEM_Q = TILE_BYTES;
  static constexpr uint32_t SMEM_NL = SMEM_Q + NQ * TILE_BYTES;  // 8 warps x 128 row terms
  static constexpr uint32_t SMEM_SUM = SMEM_NL + 8 * 512;        // 128 floats
  static constexpr uint32_t SMEM_MISC = SMEM_SUM + 512;
  static constexpr uint32_t SMEM_TOTAL = SMEM_MISC + 256 + 1024;
  static_assert(SMEM_TOTAL <= 232448, "shared memory per CTA");
  static constexpr int CTAS = D == 256 ? 1 : 2;  // per SM
  static constexpr int THREADS = 320;
};

template <int D, bool BF16, bool CAUSAL, bool ALIBI>
__global__ void __launch_bounds__(320, WeightsCfg<D>::CTAS)
    mea_weights_sm100_kernel(const __grid_constant__ CUtensorMap tm_q,
                             const __grid_constant__ CUtensorMap tm_k, const WeightsParams p) {
  using C = WeightsCfg<D>;
  constexpr float LOG2E = 1.4426950408889634f;
  const int seg = blockIdx.x / p.hkv, g = blockIdx.x - seg * p.hkv;
  const int q0 = __ldg(p.cu_q + seg), lq = max(__ldg(p.cu_q + seg + 1) - q0, 0);
  const int k0 = __ldg(p.cu_k + seg), lk = max(__ldg(p.cu_k + seg + 1) - k0, 0);
  const int j0 = blockIdx.y * 128;
  if (j0 >= lk) return;
  const int off = lk - lq;  // key position of query 0
  int qbeg = p.last > 0 ? max(lq - p.last, 0) : 0;
  if (CAUSAL) qbeg = max(qbeg, j0 - off);  // the first query that sees key j0
  const int nt = qbeg < lq ? (lq - qbeg + 127) / 128 : 0;
  const int steps = nt * p.R;

  extern __shared__ __align__(1024) uint8_t smem_raw[];
  const uint32_t pad = (1024u - (smem_u32(smem_raw) & 1023u)) & 1023u;
  uint8_t* smem = smem_raw + pad;
  const uint32_t sbase = smem_u32(smem);
  constexpr int B_KF = 0, B_QF = 1, B_QE = B_QF + C::NQ, B_SF = B_QE + C::NQ, B_SE = B_SF + 2;
  constexpr int B_CM = B_SE + 2, B_DR = B_CM + 1, N_BARS = B_DR + 1;
  static_assert(8 * N_BARS + 8 <= 256, "barrier region");
  const uint32_t bar0 = sbase + C::SMEM_MISC;
#define BAR(i) (bar0 + 8u * static_cast<uint32_t>(i))
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::SMEM_MISC + 8 * N_BARS);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const uint64_t tmo = p.timeout_ns;
  const unsigned ecode = KID_WEIGHTS << 8;
  if (threadIdx.x == 0) {
    mbar_init(BAR(B_KF), 1);
    for (int s = 0; s < C::NQ; ++s) {
      mbar_init(BAR(B_QF + s), 1);
      mbar_init(BAR(B_QE + s), 1);
    }
    for (int h = 0; h < 2; ++h) {
      mbar_init(BAR(B_SF + h), 1);
      mbar_init(BAR(B_SE + h), 4);  // one elected arrival per warp
    }
    mbar_init(BAR(B_CM), 4);
    mbar_init(BAR(B_DR), 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 8) {
    tmem_alloc(smem_u32(tmem_slot), 256);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  if (warp == 9) {
    // ---------------------------------------------------------------- TMA producer
    if (lane == 0 && steps > 0) {
      mbar_arrive_expect_tx(BAR(B_KF), C::TILE_BYTES);
#pragma unroll
      for (int a = 0; a < C::ATOMS; ++a)
        tma_load_3d(sbase + C::SMEM_K + a * C::ATOM_BYTES, &tm_k, BAR(B_KF), a * 64, g, k0 + j0);
      bool ok = true;
      int t = 0, head = g * p.R, k = 0;
      for (; k < steps; ++k) {
        const uint32_t s = k % C::NQ;
        ok = mbar_wait(BAR(B_QE + s), ((k / C::NQ) & 1u) ^ 1u, abort_flag, tmo, ecode | 1);
        if (!ok) break;
        mbar_arrive_expect_tx(BAR(B_QF + s), C::TILE_BYTES);
#pragma unroll
        for (int a = 0; a < C::ATOMS; ++a)
          tma_load_3d(sbase + C::SMEM_Q + s * C::TILE_BYTES + a * C::ATOM_BYTES, &tm_q,
                      BAR(B_QF + s), a * 64, head, q0 + qbeg + t * 128);
        if (++t == nt) {
          t = 0;
          ++head;
        }
      }
      if (!ok) {
        // Let the loads already issued land before the CTA's shared memory goes away.
        volatile int never = 0;
        for (int s = 0; s < C::NQ && s < k; ++s) {
          const int last = k - 1 - ((k - 1 - s) % C::NQ);
          mbar_wait(BAR(B_QF + s), (last / C::NQ) & 1u, &never, tmo, ecode | 15);
        }
        mbar_wait(BAR(B_KF), 0, &never, tmo, ecode | 15);
      }
    }
    __syncwarp();
  } else if (warp == 8) {
    // ---------------------------------------------------------------- tcgen05 issuer
    if (lane == 0 && steps > 0) {
      constexpr uint32_t IDESC = umma_idesc_f16(BF16, 128, 128, false, false);
      bool ok = mbar_wait(BAR(B_KF), 0, abort_flag, tmo, ecode | 2);
      for (int k = 0; k < steps && ok; ++k) {
        const uint32_t s = k % C::NQ, h = k & 1;
        ok = mbar_wait(BAR(B_QF + s), (k / C::NQ) & 1u, abort_flag, tmo, ecode | 3);
        if (!ok) break;
        ok = mbar_wait_spin(BAR(B_SE + h), ((k >> 1) & 1u) ^ 1u, abort_flag, tmo, ecode | 4);
        if (!ok) break;
        tc_fence_after();
        const uint32_t qb = sbase + C::SMEM_Q + s * C::TILE_BYTES;
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t o = (kk >> 2) * C::ATOM_BYTES + (kk & 3) * 32;
          mma_ss(tmem + h * 128, umma_desc_sw128(sbase + C::SMEM_K + o, 16, 1024),
                 umma_desc_sw128(qb + o, 16, 1024), IDESC, kk > 0 ? 1u : 0u);
        }
        mma_commit(BAR(B_SF + h));
        mma_commit(BAR(B_QE + s));
      }
      // Every MMA issued so far must finish before TMEM is released.
      mma_commit(BAR(B_DR));
      volatile int never = 0;
      mbar_wait(BAR(B_DR), 0, &never, tmo, ecode | 14);
    }
    __syncwarp();
  } else {
    // ---------------------------------------------------------------- sums (thread = key)
    const int h = warp >> 2;
    const int r = threadIdx.x & 127;
    const uint32_t t_s = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16) + h * 128;
    float* nl = reinterpret_cast<float*>(smem + C::SMEM_NL) + warp * 128;
    const uint32_t nl_s = sbase + C::SMEM_NL + static_cast<uint32_t>(warp) * 512u;
    const uint64_t c1x2 = f2_pack(p.c1, p.c1);
    float sum = 0.f, comp = 0.f;  // running sum and what it lost
    bool ok = true;
    int t = h, head = g * p.R;    // this warpgroup's first step is number h
    while (nt > 0 && t >= nt) {
      t -= nt;
      ++head;
    }
    for (int k = h; k < steps; k += 2) {
      const int qt = qbeg + t * 128;
      const int cols = min(lq - qt, 128);  // queries of the tile that exist
      float slope2 = 0.f;
      if constexpr (ALIBI) slope2 = __ldg(p.slopes + head) * LOG2E;
      // Row terms: column c adds nl[c] = -lse2 (causal ALiBi: - slope2 (p_i - j0) as well, so that
      // the key's own term is small too).
      __syncwarp();
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int c = u * 32 + lane;
        float v = -INFINITY;
        if (c < cols) {
          v = -LOG2E * __ldg(p.lse + static_cast<size_t>(head) * p.total_q + q0 + qt + c);
          if (v == INFINITY) v = -INFINITY;  // (a row that attends to nothing)
          if constexpr (ALIBI && CAUSAL) v -= slope2 * static_cast<float>(qt + c + off - j0);
        }
        nl[c] = v;
      }
      __syncwarp();
      ok = mbar_wait(BAR(B_SF + h), (k >> 1) & 1u, abort_flag, tmo, ecode | 5);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      tc_fence_after();
      const bool edge = cols < 128 || (CAUSAL && qt + off < j0 + 127);
      const int clo = CAUSAL ? j0 + r - off - qt : 0;  // first column that sees this key
      const float aj = ALIBI && CAUSAL ? slope2 * static_cast<float>(r) : 0.f;
      const uint64_t ajx2 = f2_pack(aj, aj);
      uint64_t acc[4] = {0ull, 0ull, 0ull, 0ull};
#pragma unroll
      for (int c4 = 0; c4 < 4; ++c4) {
        if (c4 * 32 >= cols) break;
        uint32_t x[32];
        tmem_ld32(t_s + c4 * 32, x);
        tmem_wait_ld();
#pragma unroll
        for (int i = 0; i < 32; i += 4) {
          uint64_t n0, n1;
          asm volatile("ld.shared.v2.b64 {%0, %1}, [%2];"
                       : "=l"(n0), "=l"(n1)
                       : "r"(nl_s + (c4 * 32 + i) * 4));
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            const int c = c4 * 32 + i + 2 * u;
            uint64_t e = f2_fma(f2_pack(__uint_as_float(x[i + 2 * u]),
                                        __uint_as_float(x[i + 2 * u + 1])),
                                c1x2, u ? n1 : n0);
            if constexpr (ALIBI && CAUSAL) e = f2_add(e, ajx2);
            float e0, e1;
            f2_unpack(e, e0, e1);
            if constexpr (ALIBI && !CAUSAL) {
              const float d0 = static_cast<float>(qt + off - j0 - r);
              e0 = fmaf(-slope2, fabsf(d0 + static_cast<float>(c)), e0);
              e1 = fmaf(-slope2, fabsf(d0 + static_cast<float>(c + 1)), e1);
            }
            if (edge) {
              if (c < clo || c >= cols) e0 = -INFINITY;
              if (c + 1 < clo || c + 1 >= cols) e1 = -INFINITY;
            }
            acc[(i >> 1 & 2) + u] =
                f2_add(acc[(i >> 1 & 2) + u], f2_pack(ex2_approx(e0), ex2_approx(e1)));
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(BAR(B_SE + h));
      float a0, a1;
      f2_unpack(f2_add(f2_add(acc[0], acc[1]), f2_add(acc[2], acc[3])), a0, a1);
      // Long prompts add thousands of tile sums: carry the rounding along.
      const float y = (a0 + a1) - comp;
      const float s2 = sum + y;
      comp = (s2 - sum) - y;
      sum = s2;
      t += 2;
      while (t >= nt) {
        t -= nt;
        ++head;
      }
    }
    // ---- the second warpgroup's sums join the first's
    float* part = reinterpret_cast<float*>(smem + C::SMEM_SUM);
    if (h == 1) {
      part[r] = sum;
      __syncwarp();
      if (lane == 0) mbar_arrive(BAR(B_CM));
    } else {
      if (ok) ok = mbar_wait(BAR(B_CM), 0, abort_flag, tmo, ecode | 6);
      ok = __all_sync(0xffffffffu, ok);
      if (ok && j0 + r < lk && j0 + r < p.w_stride)
        p.weights[(static_cast<size_t>(seg) * p.hkv + g) * p.w_stride + j0 + r] = sum + part[r];
    }
  }
#undef BAR
  tc_fence_before();
  __syncthreads();
  if (warp == 8) {
    tc_fence_after();
    tmem_dealloc(tmem, 256);
  }
}

}  // namespace mea
