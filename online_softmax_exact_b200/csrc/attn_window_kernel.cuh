// attn_window_kernel.cuh - exact attention with a sliding window and a few first tokens
// that stay visible (sinks), forward, for prompts.
//
// Query row i at position p_i sees the keys at positions <= p_i that are also > p_i - W
// or < S. The method and the B200 mapping are those of attn_fwd_kernel.cuh (one CTA per
// SM, work units of two 128-row query tiles, TMA producer, tcgen05 products
// with S, P and O in tensor memory, one softmax thread per row, one division at the end);
// what differs is which key tiles are visited:
//   * a unit's list is the 128-key tiles that hold sinks and the tiles of its rows'
//     windows, each once, however long the sequence is;
//   * where query heads share key/value heads in even groups, a unit's two query tiles are
//     the same 128 rows of two heads, so that both see the same key tiles: 9 window tiles
//     at W = 1024, in 9 steps;
//   * elsewhere they are 256 rows of one head, and each skips the tiles of the list that none
//     of its own rows sees (the list's last window tile for the first, its first for the
//     second): 9 of 10 tiles each, in 10 steps;
//   * tiles cut by a row's limits (about two of nine) mask element by element, from one
//     bit mask per row and 32 keys; the scores are then reduced by the same code as in
//     whole tiles, a masked score being -inf.
// P enters P.V as one bf16 number, rounded, as in attn_fwd_kernel (32k rows, bf16 output:
// error against 64 bits 0.0023, of which the output's own rounding is 0.0016). A second part,
// as in window_token_kernel.cuh, would double the P.V product.
// Bound: as in attn_fwd_kernel the tensor core and the exponentials of the visited tiles.
// Measured: 32 768 rows, 32 heads on 8, window 1024, 64 sinks: 657 us in a short run (1.05
// PFLOP/s of visited tiles), 753 us under the power cap; pairs of row tiles of one head took
// 707. 2 x 16 heads of 4001 rows: 91 and 98 us.
//
// The K/V tensor maps end with the chunk, so rows past it read as zero. A key row inside
// the chunk that some row of a visited tile does not see still enters that row's product
// with weight 0, so K and V rows of the chunk must be finite.
#pragma once

#include "attn_fwd_kernel.cuh"
#include "serve_ptx.cuh"
#include "serve_params.h"

namespace osx {

template <int D>
struct WindowCfg : FwdCfg<D> {
  // the epilogue's buffers, at both head sizes
  static constexpr uint32_t kSmemBytes = FwdCfg<D>::kStageOff + 8 * 4096 + 1024;
  static_assert(kSmemBytes <= 232448, "shared memory per block");
};

// The key tiles of one query tile of a unit: sink tiles [0, s), window tiles [first, last]
struct WindowTile {
  int s, first, last;
  __device__ bool sees(int kt) const { return kt < s || (kt >= first && kt <= last); }
  __device__ bool any() const { return s > 0 || last >= first; }
};

struct WindowUnit {
  int head[2], row0[2];  // of the two query tiles: B Hq head and first row
  int n, n_s, w0;  // the unit's list: tiles 0 .. n_s - 1, then w0 ..
  WindowTile t[2];
  __device__ int tile(int j) const { return j < n_s ? j : w0 + j - n_s; }
  // last step of the list that query tile i sees (-1: none)
  __device__ int last_step(int i) const {
    return t[i].last >= t[i].first ? n_s + t[i].last - w0 : t[i].s - 1;
  }
};

__device__ __forceinline__ WindowTile window_tile(const WindowParams& p, int row_a) {
  WindowTile w{0, 1, 0};
  if (row_a >= p.Nq) return w;
  const int row_b = row_a + 127 < p.Nq - 1 ? row_a + 127 : p.Nq - 1;
  long long hi = p.rel + row_b;  // last key row that the tile's last row sees
  if (hi > p.Nkv - 1) hi = p.Nkv - 1;
  if (hi < 0) return w;
  long long lo = p.rel + row_a - p.window + 1;  // first key row of its first row's window
  if (lo < 0) lo = 0;
  if (lo <= hi) {
    w.first = (int)(lo / 128);
    w.last = (int)(hi / 128);
  }
  const int cnt = p.sinks < hi + 1 ? p.sinks : (int)(hi + 1);
  w.s = (cnt + 127) / 128;
  return w;
}

// Unit u's head and row block. First the row blocks whose windows lie whole inside the
// sequence (all of one cost), head by head, so that the CTAs running at one time share a
// few heads' keys in L2; then those that the sequence's start cuts, longest first, so that
// the grid's last units are its shortest. (Measured: 2 x 16 heads of 4001 rows, window
// 1024, 103 us with row blocks in order, 93 us like this.)
__device__ __forceinline__ void window_place(const WindowParams& p, int u, int* bh, int* qp) {
  const int n_full = p.row_blocks - p.cut_blocks;
  const int full = p.heads * n_full;
  if (u < full) {
    *bh = u / n_full;
    *qp = p.row_blocks - 1 - (u - *bh * n_full);
  } else {
    const int r = (u - full) / p.heads;
    *qp = p.cut_blocks - 1 - r;
    *bh = u - full - r * p.heads;
  }
}

// Head and first row of the query tiles of unit u (see WindowParams::pair).
__device__ __forceinline__ void window_tiles(const WindowParams& p, int u, int (&head)[2],
                                             int (&row0)[2]) {
  int bh, qp;
  window_place(p, u, &bh, &qp);
  if (p.pair) {
    head[0] = 2 * bh;
    head[1] = 2 * bh + 1;
    row0[0] = row0[1] = qp * 128;
  } else {
    head[0] = head[1] = bh;
    row0[0] = qp * 256;
    row0[1] = qp * 256 + 128;
  }
}

__device__ __forceinline__ WindowUnit window_unit(const WindowParams& p, int u) {
  WindowUnit un;
  window_tiles(p, u, un.head, un.row0);
  un.t[0] = window_tile(p, un.row0[0]);
  un.t[1] = window_tile(p, un.row0[1]);
  const WindowTile &a = un.t[0], &b = un.t[1];
  const bool wa = a.last >= a.first, wb = b.last >= b.first;
  un.n_s = a.s > b.s ? a.s : b.s;
  un.w0 = 0;
  int n_w = 0;
  if (wa || wb) {
    un.w0 = !wb || (wa && a.first < b.first) ? a.first : b.first;
    const int w1 = !wb || (wa && a.last > b.last) ? a.last : b.last;
    n_w = w1 - un.w0 + 1;
    if (un.n_s > un.w0) un.n_s = un.w0;
  }
  un.n = un.n_s + n_w;
  return un;
}

// bits [0, n) of a word, n clamped to 0..32
__device__ __forceinline__ uint32_t low_bits(int n) {
  return n <= 0 ? 0u : (n >= 32 ? 0xffffffffu : (1u << n) - 1u);
}

template <int D>
__global__ void __launch_bounds__(FwdCfg<D>::kThreads, 1)
attn_window_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                   const __grid_constant__ CUtensorMap tmV, const __grid_constant__ WindowParams p) {
  using C = WindowCfg<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const uint32_t sbase = smem_u32(smem);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::kBarOff);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::kMiscOff);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::kMiscOff + 4);

  auto bar = [&](int i) { return smem_u32(&bars[i]); };
  constexpr int B_QF = 0, B_QE = 1;
  constexpr int B_KF = 2, B_KE = B_KF + C::kKStages, B_VF = B_KE + C::kKStages,
                B_VE = B_VF + C::kVStages;
  constexpr int B_SF = B_VE + C::kVStages, B_PF = B_SF + 2, B_OD = B_SF + 4, B_DRAIN = B_SF + 6;
  static_assert(B_DRAIN + 1 == C::kNumBars, "barriers");

  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  if (threadIdx.x == 0) {
    *abort_flag = 0;
    for (int i = 0; i < C::kNumBars; ++i)
      mbar_init(bar(i), i == B_PF || i == B_PF + 1 ? C::kPFullCount : 1);
    fence_mbar_init();
  }
  if (warp == C::kWarpMma) {
    tmem_alloc(smem_u32(tmem_slot), 512);
    tmem_relinquish();
  }
  if (warp == C::kWarpProducer && lane == 0) {
    tma_prefetch_desc(&tmQ);
    tma_prefetch_desc(&tmK);
    tma_prefetch_desc(&tmV);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  grid_dependents_launch();
  grid_dependency_wait();
  const uint32_t tmem = *tmem_slot;
  const int G = gridDim.x;

  if (warp >= C::kSoftmaxWarps) {
    regs_decrease<C::kRegsOther>();
    if (warp == C::kWarpProducer) {
      // ---------------------------------------------------------------- TMA producer
      if (lane == 0) {
        int ks = 0, kph = 0, vs = 0, vph = 0, qcount = 0;
        int k_arms = 0, v_arms = 0;
        bool ok = true;
        for (int r = 0; ok; ++r) {
          const int u = unit_for_round(r, blockIdx.x, G);
          if (u >= p.units) break;
          const WindowUnit un = window_unit(p, u);
          if (un.n == 0) continue;
          const int kvh = un.head[0] / p.group;  // B Hkv head: groups lie side by side
          {
            // the next unit's Q into L2 (its buffer is free only after this unit's last
            // Q.K^T)
            const int u2 = unit_for_round(r + 1, blockIdx.x, G);
            if (u2 < p.units) {
              int head2[2], row2[2];
              window_tiles(p, u2, head2, row2);
              for (int t = 0; t < 2; ++t)
                for (int h = 0; h < D / 64; ++h)
                  tma_prefetch_l2_3d(&tmQ, h * 64, row2[t], head2[t]);
            }
          }
          if (!(ok = mbar_wait(bar(B_QE), (qcount & 1) ^ 1, abort_flag, p.status))) break;
          ++qcount;
          mbar_arrive_expect_tx(bar(B_QF), 2 * C::kTileBytes);
          for (int t = 0; t < 2; ++t)
            for (int h = 0; h < D / 64; ++h)
              tma_load_3d(sbase + C::kQOff + t * C::kTileBytes + h * 16384, &tmQ, bar(B_QF),
                          h * 64, un.row0[t], un.head[t]);
          for (int j = 0; j < un.n; ++j) {
            const int row = un.tile(j) * 128;
            if (!(ok = mbar_wait(bar(B_KE + ks), kph ^ 1, abort_flag, p.status))) break;
            mbar_arrive_expect_tx(bar(B_KF + ks), C::kTileBytes);
            for (int h = 0; h < D / 64; ++h)
              tma_load_3d(sbase + C::kKOff + ks * C::kTileBytes + h * 16384, &tmK, bar(B_KF + ks),
                          h * 64, row, kvh);
            ++k_arms;
            if (++ks == C::kKStages) { ks = 0; kph ^= 1; }
            if (!(ok = mbar_wait(bar(B_VE + vs), vph ^ 1, abort_flag, p.status))) break;
            mbar_arrive_expect_tx(bar(B_VF + vs), C::kTileBytes);
            for (int h = 0; h < D / 64; ++h)
              tma_load_3d(sbase + C::kVOff + vs * C::kTileBytes + h * 16384, &tmV, bar(B_VF + vs),
                          h * 64, row, kvh);
            ++v_arms;
            if (++vs == C::kVStages) { vs = 0; vph ^= 1; }
          }
        }
        // every copy issued lands before the CTA exits (bounded; see attn_fwd_kernel)
        bool drained = true;
        if (qcount > 0) drained &= mbar_wait_drain(bar(B_QF), (qcount - 1) & 1, kDrainLimitNs);
        for (int st = 0; st < C::kKStages; ++st) {
          const int kn = k_arms / C::kKStages + (st < k_arms % C::kKStages ? 1 : 0);
          if (kn > 0) drained &= mbar_wait_drain(bar(B_KF + st), (kn - 1) & 1, kDrainLimitNs);
        }
        for (int st = 0; st < C::kVStages; ++st) {
          const int vn = v_arms / C::kVStages + (st < v_arms % C::kVStages ? 1 : 0);
          if (vn > 0) drained &= mbar_wait_drain(bar(B_VF + st), (vn - 1) & 1, kDrainLimitNs);
        }
        if (!drained) {
          const unsigned long long t0 = globaltimer_ns();
          while (globaltimer_ns() - t0 < 200000ull) {
          }
        }
      }
    } else if (warp == C::kWarpMma) {
      // ---------------------------------------------------------------- MMA issuer
      if (C::kWarpIssue || lane == 0) {
        constexpr uint32_t idesc_qk = idesc_bf16_f32(128, 128, 0, 0);
        constexpr uint32_t idesc_pv = idesc_bf16_f32(128, D, 0, 1);
        int ks = 0, kph = 0, vs = 0, vph = 0, qcount = 0;
        int steps[2] = {0, 0};  // P.V products issued for each query tile (p_full's parity)
        bool ok = true;
        auto wait_u = [&](uint32_t b, int parity) -> bool {
          const bool r = mbar_wait(b, parity, abort_flag, p.status);
          if constexpr (C::kWarpIssue) return __all_sync(0xffffffffu, r);
          return r;
        };
        auto commit = [&](uint32_t b) {
          if constexpr (C::kWarpIssue) mma_commit_warp(b); else mma_commit(b);
        };
        const uint64_t dq0 = sdesc_sw128(sbase + C::kQOff, 16, 1024);
        const uint64_t dk0 = sdesc_sw128(sbase + C::kKOff, 16, 1024);
        const uint64_t dv0 = sdesc_sw128(sbase + C::kVOff, 16384, 1024);
        constexpr uint64_t kTileStep = C::kTileBytes >> 4;
        auto issue_pv = [&](int t, int vstage, bool acc) {
          uint64_t dv = dv0 + (uint64_t)vstage * kTileStep;
          const uint32_t tO = tmem + (t ? C::kColO1 : C::kColO0);
          const uint32_t tP = tmem + (t ? C::kColS1 : C::kColS0);
          opaque(dv);
#pragma unroll
          for (int kk = 0; kk < 8; ++kk) {
            const uint64_t b = dv + (uint64_t)(kk * 128);
            const uint32_t en = (acc || kk > 0) ? 1u : 0u;
            if constexpr (C::kWarpIssue)
              mma_ts_warp(tO, tP + kk * 8, b, idesc_pv, en);
            else
              mma_ts(tO, tP + kk * 8, b, idesc_pv, en);
          }
        };
        auto issue_qk = [&](int t, int kstage) {
          uint64_t dq = dq0 + (uint64_t)t * kTileStep;
          uint64_t dk = dk0 + (uint64_t)kstage * kTileStep;
          const uint32_t tS = tmem + (t ? C::kColS1 : C::kColS0);
          opaque(dq);
          opaque(dk);
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            const uint64_t off = (uint64_t)((kk / 4) * 1024 + (kk % 4) * 2);
            if constexpr (C::kWarpIssue)
              mma_ss_warp(tS, dq + off, dk + off, idesc_qk, kk > 0 ? 1u : 0u);
            else
              mma_ss(tS, dq + off, dk + off, idesc_qk, kk > 0 ? 1u : 0u);
          }
        };

        for (int r = 0; ok; ++r) {
          const int u = unit_for_round(r, blockIdx.x, G);
          if (u >= p.units) break;
          const WindowUnit un = window_unit(p, u);
          if (un.n == 0) continue;
          if (!(ok = wait_u(bar(B_QF), qcount & 1))) break;
          ++qcount;
          tc_fence_after();
          bool started[2] = {false, false};  // O_t holds this unit's products
          // step j: P.V of tile j - 1, then Q.K^T of tile j, for each query tile that sees it
          for (int j = 0; j <= un.n && ok; ++j) {
            if (j < un.n) {
              if (!(ok = wait_u(bar(B_KF + ks), kph))) break;
            }
            if (j > 0) {
              if (!(ok = wait_u(bar(B_VF + vs), vph))) break;
            }
            tc_fence_after();
#pragma unroll
            for (int t = 0; t < 2; ++t) {
              if (j > 0 && un.t[t].sees(un.tile(j - 1))) {
                if (!(ok = wait_u(bar(B_PF + t), steps[t] & 1))) break;
                ++steps[t];
                tc_fence_after();
                issue_pv(t, vs, started[t]);
                started[t] = true;
                if (j - 1 == un.last_step(t)) commit(bar(B_OD + t));
              }
              if (j < un.n && un.t[t].sees(un.tile(j))) {
                issue_qk(t, ks);
                commit(bar(B_SF + t));
              }
            }
            if (!ok) break;
            if (j < un.n) {
              commit(bar(B_KE + ks));
              if (++ks == C::kKStages) { ks = 0; kph ^= 1; }
              if (j == un.n - 1) commit(bar(B_QE));
            }
            if (j > 0) {
              commit(bar(B_VE + vs));
              if (++vs == C::kVStages) { vs = 0; vph ^= 1; }
            }
          }
        }
      }
    }
  } else {
    regs_increase<C::kRegsSoftmax>();
    // ------------------------------------------------------------------ softmax
    const int t = warp / 4, wq = warp % 4, r = wq * 32 + lane;
    const uint32_t lane_base = static_cast<uint32_t>(wq * 32) << 16;
    const uint32_t tS = tmem + lane_base + (t ? C::kColS1 : C::kColS0);
    const uint32_t tO = tmem + lane_base + (t ? C::kColO1 : C::kColO0);
    const float c = p.scale_log2;
    int scount = 0, ocount = 0;
    bool ok = true;

    for (int rr = 0; ok; ++rr) {
      const int u = unit_for_round(rr, blockIdx.x, G);
      if (u >= p.units) break;
      const WindowUnit un = window_unit(p, u);
      const WindowTile wt = t ? un.t[1] : un.t[0];
      const int row0 = t ? un.row0[1] : un.row0[0];  // first row of this tile
      const int head = t ? un.head[1] : un.head[0];
      const long long row = (long long)row0 + r;
      float m = -INFINITY, l = 0.f;

      if (wt.any()) {
        // limits of this row and of the tile's outer rows, as key rows of the chunk
        const long long rel = p.rel + row, rel0 = p.rel + row0;
        const long long last = p.Nkv - 1;
        const int hi_row = (int)(rel < last ? (rel < -1 ? -1 : rel) : last);
        const int hi_all = (int)(rel0 < last ? (rel0 < -1 ? -1 : rel0) : last);
        auto clip = [&](long long x) { return (int)(x < 0 ? 0 : (x < p.Nkv ? x : p.Nkv)); };
        const int lo_row = clip(rel - p.window + 1);
        const int lo_all = clip(rel0 + 127 - p.window + 1);
        bool first = true;

        for (int j = 0; j < un.n; ++j) {
          const int k0 = un.tile(j) * 128;
          if (!wt.sees(un.tile(j))) continue;
          ok = mbar_wait(bar(B_SF + t), scount & 1, abort_flag, p.status);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          ++scount;
          tc_fence_after();

          uint32_t s[4][32];
#pragma unroll
          for (int q = 0; q < 4; ++q) tmem_ld32(tS + 32 * q, s[q]);
          tmem_ld_wait(s[0]);
          reg_fence(s[1]);
          reg_fence(s[2]);
          reg_fence(s[3]);

          // the same for every row of the tile
          if (k0 + 127 > hi_all || (k0 < lo_all && k0 + 127 >= p.sinks)) {
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              const int kq = k0 + 32 * q;
              const uint32_t see = low_bits(hi_row + 1 - kq) &
                                   (~low_bits(lo_row - kq) | low_bits(p.sinks - kq));
#pragma unroll
              for (int i = 0; i < 32; ++i)
                if (!(see & (1u << i))) s[q][i] = 0xff800000u;  // -inf
            }
          }
          float mxa[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
          for (int q = 0; q < 4; ++q)
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              float& acc = mxa[(q & 1) * 2 + (i & 1)];
              acc = fmax3(acc, __uint_as_float(s[q][2 * i]), __uint_as_float(s[q][2 * i + 1]));
            }
          const float mx = fmaxf(fmaxf(mxa[0], mxa[1]), fmaxf(mxa[2], mxa[3]));
          const float m_tile = (mx == -INFINITY) ? -INFINITY : mx * c;
          const float m_new = (m_tile > m + 8.0f) ? m_tile : m;
          const float alpha = (m_new == m) ? 1.f : ex2_approx(m - m_new);
          const float m_use = (m_new == -INFINITY) ? 0.f : m_new;

          // c > 0, so a masked score's exponent is -inf and its P exactly 0
          float sum = softmax_row32<false, 0u>(s[0], tS, c, m_use, 127);
          sum += softmax_row32<false, 0u>(s[1], tS + 16, c, m_use, 127);
          sum += softmax_row32<false, 0u>(s[2], tS + 32, c, m_use, 127);
          sum += softmax_row32<false, 0u>(s[3], tS + 48, c, m_use, 127);
          l = l * alpha + sum;

          // rescale this row of O when its base moved (the P.V of this tile's previous
          // step has completed: the Q.K^T commit that released S follows it)
          const bool moved = (m_new != m) && !first;
          if (__any_sync(0xffffffffu, moved)) {
            const float a = moved ? alpha : 1.f;
#pragma unroll 1
            for (int q4 = 0; q4 < D / 32; ++q4) {
              uint32_t ov[32];
              tmem_ld32(tO + q4 * 32, ov);
              tmem_ld_wait(ov);
#pragma unroll
              for (int i = 0; i < 32; ++i) ov[i] = __float_as_uint(__uint_as_float(ov[i]) * a);
              tmem_st32(tO + q4 * 32, ov);
            }
          }
          first = false;
          m = m_new;
          tmem_st_wait();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(B_PF + t));
        }
        if (!ok) break;
        ok = mbar_wait(bar(B_OD + t), ocount & 1, abort_flag, p.status);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        ++ocount;
        tc_fence_after();
      }
      if (row0 >= p.Nq) continue;

      // ---------------------------------------------------------------- epilogue
      // O leaves through a per-warp buffer of 32 rows x 128 bytes (16-byte pieces swizzled
      // by row), four rows' 128-byte segments per store; rows without a key give 0
      const bool seen = l > 0.f;
      const float b = seen ? 1.f / l : 0.f;
      uint4* stage = reinterpret_cast<uint4*>(smem + C::kStageOff + warp * 4096);
      const int ch = lane & 7;
      const int wrow0 = row0 + wq * 32;
      const int per = p.o_bf16 ? 64 : 32;  // values of a row's 128 bytes
      const int es = p.o_bf16 ? 2 : 4;
      char* base = static_cast<char*>(p.o) + ((long long)head * p.Nq + wrow0) * D * es;
#pragma unroll 1
      for (int q4 = 0; q4 < D / per; ++q4) {
        if (wt.any()) {
#pragma unroll 1
          for (int half = 0; half < per / 32; ++half) {
            uint32_t ov[32];
            tmem_ld32(tO + q4 * per + half * 32, ov);
            tmem_ld_wait(ov);
#pragma unroll
            for (int i = 0; i < 32; ++i)
              ov[i] = seen ? __float_as_uint(__uint_as_float(ov[i]) * b) : 0u;
            if (p.o_bf16) {
#pragma unroll
              for (int x = 0; x < 4; ++x) {
                const int piece = half * 4 + x;
                stage[lane * 8 + (piece ^ (lane & 7))] = make_uint4(
                    pack_bf16x2(__uint_as_float(ov[8 * x]), __uint_as_float(ov[8 * x + 1])),
                    pack_bf16x2(__uint_as_float(ov[8 * x + 2]), __uint_as_float(ov[8 * x + 3])),
                    pack_bf16x2(__uint_as_float(ov[8 * x + 4]), __uint_as_float(ov[8 * x + 5])),
                    pack_bf16x2(__uint_as_float(ov[8 * x + 6]), __uint_as_float(ov[8 * x + 7])));
              }
            } else {
#pragma unroll
              for (int x = 0; x < 8; ++x)
                stage[lane * 8 + (x ^ (lane & 7))] =
                    make_uint4(ov[4 * x], ov[4 * x + 1], ov[4 * x + 2], ov[4 * x + 3]);
            }
          }
        } else {
#pragma unroll
          for (int x = 0; x < 8; ++x) stage[lane * 8 + x] = make_uint4(0, 0, 0, 0);
        }
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int rl = i * 4 + (lane >> 3);
          const uint4 v = stage[rl * 8 + (ch ^ (rl & 7))];
          if (wrow0 + rl < p.Nq)
            *reinterpret_cast<uint4*>(base + ((long long)rl * D + q4 * per) * es + ch * 16) = v;
        }
        __syncwarp();  // the buffer is rewritten by the next chunk
      }
      if (row < p.Nq)
        p.lse[(long long)head * p.Nq + row] =
            seen ? (m + lg2_approx(l)) * 0.69314718055994530942f : -INFINITY;
      tc_fence_before();
    }
  }

  // ---------------------------------------------------------------------- teardown
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (*abort_flag) {
    // in-flight tensor-core work completes before TMEM is freed
    if (warp == C::kWarpMma && (C::kWarpIssue || lane == 0)) {
      if constexpr (C::kWarpIssue)
        mma_commit_warp(bar(B_DRAIN));
      else
        mma_commit(bar(B_DRAIN));
      mbar_wait_drain(bar(B_DRAIN), 0, kDrainLimitNs);
    }
    __syncthreads();
  }
  if (warp == C::kWarpMma) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

}  // namespace osx
