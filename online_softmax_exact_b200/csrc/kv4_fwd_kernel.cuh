// kv4_fwd_kernel.cuh - attention of the newest tokens over the paged 4-bit cache.
//
// For request b, the query rows of one key/value head (group heads x Nq tokens) against
// the keys j < lens[b] with j <= p_i (p_i: the row's position), and with a window W > 0
// only j > p_i - W or j < sinks. Online softmax, one division at the end; returns O and
// LSE like the other attention calls.
//
// Bound: memory, 1.25 d bytes a token and head (keys, values and their parameters), and
// close behind it instruction issue: the codes have to become matrix operands. So
//   * a unit of work is one request and key/value head with 8 NT query rows; its keys
//     are shared by all of them (a group of 8 heads reads the cache once);
//   * a warp runs its own stages of kSB blocks of 16 tokens: one lane per block fetches
//     it with one bulk copy (a block is contiguous), through a ring of kStages slots, and
//     no warp waits for another before the final join;
//   * products run as S^T = K Q^T and O^T = V^T P^T on mma.m16n8k16 with the keys (the
//     values' channels) as the 16 rows and 8 query rows as columns, so a few query rows
//     waste nothing. (tcgen05 would need 128 rows of unpacked bf16 keys in shared
//     memory: four times the traffic that the cache itself costs there.) The cache's
//     word order is the operand order, so unpacking is a shift, a mask and a bias;
//   * codes enter the products as small integers: 0x4300 | c is the bf16 number 128 + c.
//     A group's scale and zero point are applied to the fp32 sums:
//       s_j = sum over groups of scale (sum_i (128 + c_i) q_i) + (zero - 128 scale) sum_i q_i
//     and for the values the scale goes to P, and the codes are centred (c - 8, exact), so
//     that the rounding of P * scale to bf16 stays relative to a value's own size:
//       O = sum_j bf16(P_j scale_j) (c_j - 8) + sum_j P_j (zero_j + 8 scale_j),
//     the second sum in fp32;
//   * a cluster of up to 16 blocks shares a unit where units are few, joined through
//     distributed shared memory (decode_merge.cuh).
// Statistics, sums and the output are fp32; P * scale (the matrix operand) is bf16.
//
// Pages are looked up in the table and checked against n_pages: keys on a page outside
// the cache are invisible. Rows of a page past a request's length may hold anything.
#pragma once

#include <cuda_bf16.h>

#include <cstdint>

#include "serve_params.h"

#include "decode_merge.cuh"
#include "kv4_layout.cuh"

namespace osx {

template <int D, int NT>
struct Kv4FwdCfg {
  static constexpr int kWarps = 8;
  static constexpr int kSB = D == 128 ? 2 : 4;      // blocks of 16 tokens per stage
  static constexpr int kStages = 2;
  static constexpr uint32_t kStageBytes = kSB * Kv4<D>::kBytes;
  static constexpr uint32_t kWarpBytes = kStages * kStageBytes;
  using Merge = DecodeMerge<D, NT, kWarps>;
  static_assert(kWarpBytes >= 8 * NT * D * 4, "a warp's rows reuse its ring");
  static constexpr uint32_t kMergeOff = kWarps * kWarpBytes;
  static constexpr uint32_t kBarOff = kMergeOff + Merge::kBytes;
  static constexpr uint32_t kSmemBytes = kBarOff + kWarps * kStages * 8 + 16;
  static_assert(kBarOff % 8 == 0, "mbarrier alignment");
};

__device__ __forceinline__ uint32_t codes_plus_128(uint32_t x) {
  return (x & 0x000f000fu) | 0x43004300u;
}
// (128 + c) - 136 = c - 8, exact in bf16
__device__ __forceinline__ uint32_t codes_centred(uint32_t x) {
  uint32_t y;
  asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(y) : "r"(codes_plus_128(x)), "r"(0x43084308u));
  return y;
}

template <int D, int NT>
__global__ void __launch_bounds__(Kv4FwdCfg<D, NT>::kWarps * 32, NT == 1 ? 2 : 1)
kv4_fwd_kernel(const __grid_constant__ Kv4FwdParams p) {
  using C = Kv4FwdCfg<D, NT>;
  using L = Kv4<D>;
  constexpr int kG = L::kGroups;
  extern __shared__ __align__(128) uint8_t smem[];
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, g = lane >> 2, t = lane & 3;
  uint8_t* ring = smem + warp * C::kWarpBytes;
  const uint32_t ring_u = smem_u32(ring);
  const uint32_t bar0 = smem_u32(smem + C::kBarOff) + warp * C::kStages * 8;
  volatile int* abort_flag =
      reinterpret_cast<volatile int*>(smem + C::kBarOff + C::kWarps * C::kStages * 8);
  if (lane == 0) {
    for (int s = 0; s < C::kStages; ++s) mbar_init(bar0 + 8 * s, 1);
    fence_mbar_init();
  }
  if (threadIdx.x == 0) *abort_flag = 0;

  const int rank = p.splits > 1 ? (int)cluster_rank() : 0;
  int item = blockIdx.x / p.splits;
  const int rt = item % p.row_tiles;
  item /= p.row_tiles;
  const int hkv = item % p.Hkv, b = item / p.Hkv;

  // ---- the keys of this unit: blocks [0, n_s) of the sinks, then the window's
  const long long room = (long long)p.width * p.blocks_per_page * 16;
  int len = p.lens[b];
  if (len < 0) len = 0;
  if (len > room) len = (int)room;
  const long long p0 = p.q_pos ? (long long)p.q_pos[b] : (long long)len - p.Nq;
  const long long hi_l = p0 + p.Nq < len ? p0 + p.Nq : len;        // keys below may be seen
  const int hi = hi_l > 0 ? (int)hi_l : 0;
  const long long lo_l = p.window ? p0 - p.window + 1 : 0;
  const int lo = lo_l <= 0 ? 0 : (lo_l < hi ? (int)lo_l : hi);
  const int sink_end = p.window ? (p.sinks < hi ? p.sinks : hi) : 0;
  const int w0 = lo / 16;
  const int n_w = hi > lo ? (hi - 1) / 16 - w0 + 1 : 0;
  int n_s = (sink_end + 15) / 16;
  if (n_w > 0 && n_s > w0) n_s = w0;
  const int n_blocks = n_s + n_w;
  const int n_stages = (n_blocks + C::kSB - 1) / C::kSB;
  const int* row_table = p.table + (long long)b * p.width;

  // ---- this lane's page of stage s (lanes below kSB), -1: none
  auto page_of = [&](int s) {
    const int bi = s * C::kSB + lane;
    if (lane >= C::kSB || bi >= n_blocks) return -1;
    const int lb = bi < n_s ? bi : w0 + bi - n_s;
    return __ldg(row_table + lb / p.blocks_per_page);
  };
  uint32_t masks = 0;  // blocks present, 4 bits per slot
  auto issue = [&](int s, int slot, int page) {
    const bool ok = page >= 0 && page < p.n_pages;
    const uint32_t m = __ballot_sync(0xffffffffu, ok);
    masks = (masks & ~(0xfu << (4 * slot))) | (m << (4 * slot));
    if (lane == 0) mbar_arrive_expect_tx(bar0 + 8 * slot, __popc(m) * L::kBytes);
    __syncwarp();
    if (ok) {
      const int bi = s * C::kSB + lane;
      const int lb = bi < n_s ? bi : w0 + bi - n_s;
      const uint32_t* src =
          p.cache + (((long long)page * p.Hkv + hkv) * p.blocks_per_page + lb % p.blocks_per_page) *
                        L::kWords;
      bulk_load(ring_u + slot * C::kStageBytes + lane * L::kBytes, src, L::kBytes, bar0 + 8 * slot);
    }
  };
  const int step = p.splits * C::kWarps;
  const int s_first = rank * C::kWarps + warp;
  int s_next = s_first;        // next stage to fetch
  int page_next = s_next < n_stages ? page_of(s_next) : -1;
  __syncwarp();  // the barriers are initialised
  int n_issued = 0;
#pragma unroll
  for (int k = 0; k < C::kStages; ++k) {
    if (s_next < n_stages) {
      issue(s_next, k, page_next);
      s_next += step;
      ++n_issued;
      page_next = s_next < n_stages ? page_of(s_next) : -1;
    }
  }

  // ---- queries: B operands. Lane (g, t) holds, for row g of each 8-row tile and each
  // group i, values 32 i + 8 t + (0..7) paired as the codes come out of a word: (e, e + 4)
  const int row0 = rt * 8 * NT;
  const int rows = p.rows - row0 < 8 * NT ? p.rows - row0 : 8 * NT;
  const long long q_row0 = ((long long)b * p.Hkv + hkv) * p.rows + row0;  // = (b Hq + h) Nq + i
  uint32_t qf[NT][kG][4];
  float qs[NT][kG][2];  // sums of q over a group, for the columns 2t, 2t + 1
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const int r = nt * 8 + g;
#pragma unroll
    for (int i = 0; i < kG; ++i) {
      uint4 u = make_uint4(0, 0, 0, 0);
      if (r < rows)
        u = *reinterpret_cast<const uint4*>(p.q + (q_row0 + r) * D + 32 * i + 8 * t);
      // u: pairs (0,1) (2,3) (4,5) (6,7)
      qf[nt][i][0] = __byte_perm(u.x, u.z, 0x5410);
      qf[nt][i][1] = __byte_perm(u.x, u.z, 0x7632);
      qf[nt][i][2] = __byte_perm(u.y, u.w, 0x5410);
      qf[nt][i][3] = __byte_perm(u.y, u.w, 0x7632);
      float s = 0.f;
#pragma unroll
      for (int e = 0; e < 4; ++e)
        s += __uint_as_float(qf[nt][i][e] << 16) + __uint_as_float(qf[nt][i][e] & 0xffff0000u);
      s += __shfl_xor_sync(0xffffffffu, s, 1);
      s += __shfl_xor_sync(0xffffffffu, s, 2);  // row g's sum, on its four lanes
      qs[nt][i][0] = __shfl_sync(0xffffffffu, s, (2 * t) * 4);
      qs[nt][i][1] = __shfl_sync(0xffffffffu, s, (2 * t + 1) * 4);
    }
  }
  // last and first visible key of the rows 2t, 2t + 1
  int key_hi[NT][2], key_lo[NT][2];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const int r = row0 + nt * 8 + 2 * t + x;
      const long long pos = p0 + r % p.Nq;
      key_hi[nt][x] = pos < len ? (pos < -1 ? -1 : (int)pos) : len - 1;
      const long long l2 = p.window ? pos - p.window + 1 : 0;
      key_lo[nt][x] = l2 <= 0 ? 0 : (l2 < 0x7fffffff ? (int)l2 : 0x7fffffff);
    }
  const long long all_hi = p0 < len - 1 ? p0 : (long long)len - 1;  // seen by every row
  const long long all_lo = p.window ? p0 + p.Nq - p.window : 0;

  float o[NT][D / 16][4] = {};
  float zo[NT][kG][2] = {};
  float m[NT][2], l[NT][2];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      m[nt][x] = -INFINITY;
      l[nt][x] = 0.f;
    }

  __syncthreads();  // the abort flag is initialised
  int slot = 0, phase = 0, waited = 0;
  bool ok = true;
  for (int s = s_first; s < n_stages; s += step) {
    ok = mbar_wait(bar0 + 8 * slot, phase, abort_flag, p.status);
    ok = __all_sync(0xffffffffu, ok);
    if (!ok) break;
    ++waited;
    const uint8_t* stage = ring + slot * C::kStageBytes;
    const uint32_t present = (masks >> (4 * slot)) & 0xfu;

    // ---- scores
    float sc[C::kSB][NT][4];
#pragma unroll
    for (int j = 0; j < C::kSB; ++j) {
      const int bi = s * C::kSB + j;
      if (!((present >> j) & 1u)) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int x = 0; x < 4; ++x) sc[j][nt][x] = -INFINITY;
        continue;
      }
      const uint32_t* blk = reinterpret_cast<const uint32_t*>(stage + j * L::kBytes);
      uint32_t w[2][kG], par[2][kG];
      if constexpr (D == 128) {
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const uint4 a = *reinterpret_cast<const uint4*>(blk + (r * 32 + lane) * 4);
          const uint4 q = *reinterpret_cast<const uint4*>(blk + L::kKParams + (8 * r + g) * 4);
          w[r][0] = a.x, w[r][1] = a.y, w[r][2] = a.z, w[r][3] = a.w;
          par[r][0] = q.x, par[r][1] = q.y, par[r][2] = q.z, par[r][3] = q.w;
        }
      } else {
        const uint4 a = *reinterpret_cast<const uint4*>(blk + lane * 4);
        w[0][0] = a.x, w[0][1] = a.y, w[1][0] = a.z, w[1][1] = a.w;
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const uint2 q = *reinterpret_cast<const uint2*>(blk + L::kKParams + (8 * r + g) * 2);
          par[r][0] = q.x, par[r][1] = q.y;
        }
      }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int x = 0; x < 4; ++x) sc[j][nt][x] = 0.f;
#pragma unroll
      for (int i = 0; i < kG; ++i) {
        uint32_t a[2][4];
#pragma unroll
        for (int r = 0; r < 2; ++r)
#pragma unroll
          for (int e = 0; e < 4; ++e) a[r][e] = codes_plus_128(w[r][i] >> (4 * e));
        const float s0 = param_scale(par[0][i]), s1 = param_scale(par[1][i]);
        const float z0 = fmaf(-128.f, s0, param_zero(par[0][i]));
        const float z1 = fmaf(-128.f, s1, param_zero(par[1][i]));
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          float c[4] = {0.f, 0.f, 0.f, 0.f};
          mma16816(c, a[0][0], a[1][0], a[0][1], a[1][1], qf[nt][i][0], qf[nt][i][1]);
          mma16816(c, a[0][2], a[1][2], a[0][3], a[1][3], qf[nt][i][2], qf[nt][i][3]);
          float(&y)[4] = sc[j][nt];
          y[0] = fmaf(s0, c[0], fmaf(z0, qs[nt][i][0], y[0]));
          y[1] = fmaf(s0, c[1], fmaf(z0, qs[nt][i][1], y[1]));
          y[2] = fmaf(s1, c[2], fmaf(z1, qs[nt][i][0], y[2]));
          y[3] = fmaf(s1, c[3], fmaf(z1, qs[nt][i][1], y[3]));
        }
      }
      const int lb = bi < n_s ? bi : w0 + bi - n_s;
      const int k0 = lb * 16;
      if (k0 + 15 > all_hi || (k0 < all_lo && k0 + 15 >= p.sinks)) {  // the same for the warp
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const int key = k0 + g + 8 * (x >> 1);
            const bool see = key <= key_hi[nt][x & 1] &&
                             (key >= key_lo[nt][x & 1] || key < p.sinks);
            if (!see) sc[j][nt][x] = -INFINITY;
          }
      }
    }

    // ---- bases: moved only when a score exceeds one by more than 8 (log2 units), so the
    // maximum over the warp's lanes is rarely needed
    bool grows = false;
    float mx[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        float y = -INFINITY;
#pragma unroll
        for (int j = 0; j < C::kSB; ++j) y = fmaxf(y, fmaxf(sc[j][nt][x], sc[j][nt][x + 2]));
        mx[nt][x] = y == -INFINITY ? y : y * p.scale_log2;
        grows |= mx[nt][x] > m[nt][x] + 8.f;
      }
    if (__any_sync(0xffffffffu, grows)) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          float y = mx[nt][x];
#pragma unroll
          for (int d = 4; d < 32; d *= 2) y = fmaxf(y, __shfl_xor_sync(0xffffffffu, y, d));
          if (y > m[nt][x] + 8.f) {
            const float a = ex2_approx(m[nt][x] - y);  // 0 from -inf
            m[nt][x] = y;
            l[nt][x] *= a;
#pragma unroll
            for (int i = 0; i < kG; ++i) zo[nt][i][x] *= a;
#pragma unroll
            for (int i = 0; i < D / 16; ++i) {
              o[nt][i][x] *= a;
              o[nt][i][x + 2] *= a;
            }
          }
        }
    }

    // ---- P, and O^T += V^T P^T block by block
#pragma unroll
    for (int j = 0; j < C::kSB; ++j) {
      if (!((present >> j) & 1u)) continue;
      const uint32_t* blk = reinterpret_cast<const uint32_t*>(stage + j * L::kBytes);
      const int bi = s * C::kSB + j;
      const int lb = bi < n_s ? bi : w0 + bi - n_s;
      float pr[NT][4];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const float base = m[nt][x & 1] == -INFINITY ? 0.f : m[nt][x & 1];
          pr[nt][x] = ex2_approx(fmaf(sc[j][nt][x], p.scale_log2, -base));  // 0 where masked
          l[nt][x & 1] += pr[nt][x];
        }
      uint32_t par[2][kG];
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        if constexpr (D == 128) {
          const uint4 q = *reinterpret_cast<const uint4*>(blk + L::kVParams + (8 * r + g) * 4);
          par[r][0] = q.x, par[r][1] = q.y, par[r][2] = q.z, par[r][3] = q.w;
        } else {
          const uint2 q = *reinterpret_cast<const uint2*>(blk + L::kVParams + (8 * r + g) * 2);
          par[r][0] = q.x, par[r][1] = q.y;
        }
        // rows past the request's length may hold any bits: 0 * NaN is not 0
        if (lb * 16 + 8 * r + g >= len)
#pragma unroll
          for (int i = 0; i < kG; ++i) par[r][i] = 0u;
      }
      uint32_t bp[NT][kG][2];
#pragma unroll
      for (int i = 0; i < kG; ++i) {
        const float s0 = param_scale(par[0][i]), s1 = param_scale(par[1][i]);
        const float z0 = fmaf(8.f, s0, param_zero(par[0][i]));
        const float z1 = fmaf(8.f, s1, param_zero(par[1][i]));
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const float(&y)[4] = pr[nt];
          bp[nt][i][0] = transpose_b16(pack_bf16x2(y[0] * s0, y[1] * s0));
          bp[nt][i][1] = transpose_b16(pack_bf16x2(y[2] * s1, y[3] * s1));
          zo[nt][i][0] = fmaf(y[0], z0, fmaf(y[2], z1, zo[nt][i][0]));
          zo[nt][i][1] = fmaf(y[1], z0, fmaf(y[3], z1, zo[nt][i][1]));
        }
      }
#pragma unroll
      for (int h = 0; h < D / 64; ++h) {
        const uint4 a = *reinterpret_cast<const uint4*>(blk + L::kVCodes + (h * 32 + lane) * 4);
        // codes e of the keys (2t, 2t + 1) and (2t + 8, 2t + 9), side by side
        const uint32_t u0[2] = {__byte_perm(a.x, a.y, 0x5410), __byte_perm(a.x, a.y, 0x7632)};
        const uint32_t u1[2] = {__byte_perm(a.z, a.w, 0x5410), __byte_perm(a.z, a.w, 0x7632)};
#pragma unroll
        for (int mm = 0; mm < 4; ++mm) {
          const int sh = 8 * (mm & 1);
          const uint32_t x = u0[mm >> 1] >> sh, y = u1[mm >> 1] >> sh;
          const uint32_t a0 = codes_centred(x), a1 = codes_centred(x >> 4);
          const uint32_t a2 = codes_centred(y), a3 = codes_centred(y >> 4);
          const int mt = 4 * h + mm;
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
            mma16816(o[nt][mt], a0, a1, a2, a3, bp[nt][mt / 2][0], bp[nt][mt / 2][1]);
        }
      }
    }

    __syncwarp();  // every lane has read the slot
    if (s_next < n_stages) {
      issue(s_next, slot, page_next);
      s_next += step;
      ++n_issued;
      page_next = s_next < n_stages ? page_of(s_next) : -1;
    }
    if (++slot == C::kStages) {
      slot = 0;
      phase ^= 1;
    }
  }
  if (!ok) {
    // a wait ran out: let the copies still in flight land before the ring is reused
    for (; waited < n_issued; ++waited) {
      mbar_wait_drain(bar0 + 8 * slot, phase, 100000000ull);
      if (++slot == C::kStages) {
        slot = 0;
        phase ^= 1;
      }
    }
    __syncwarp();
  }

  // ---- this warp's rows to shared memory, then the join
  float* mine = reinterpret_cast<float*>(ring);  // [8 NT][D]
  float* stats = reinterpret_cast<float*>(smem + C::kMergeOff);
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      float y = l[nt][x];
#pragma unroll
      for (int d = 4; d < 32; d *= 2) y += __shfl_xor_sync(0xffffffffu, y, d);
      const int r = nt * 8 + 2 * t + x;
      if (g == 0) {
        stats[warp * 8 * NT + r] = m[nt][x];
        stats[(C::kWarps + warp) * 8 * NT + r] = y;
      }
#pragma unroll
      for (int i = 0; i < kG; ++i) {
        float z = zo[nt][i][x];
#pragma unroll
        for (int d = 4; d < 32; d *= 2) z += __shfl_xor_sync(0xffffffffu, z, d);
#pragma unroll
        for (int h = 0; h < 2; ++h) {  // channels 16 mt + g and + 8
          mine[r * D + 32 * i + 16 * h + g] = o[nt][2 * i + h][x] + z;
          mine[r * D + 32 * i + 16 * h + 8 + g] = o[nt][2 * i + h][x + 2] + z;
        }
      }
    }
  C::Merge::run(stats, [&](int w) { return reinterpret_cast<const float*>(smem + w * C::kWarpBytes); },
                p.splits, rows, q_row0, p.o, p.o_bf16, p.lse);
}

}  // namespace osx
