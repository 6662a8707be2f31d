// kv4_fwd_kernel.cuh - attention of the newest tokens over the paged 4-bit cache.
//
// For request b, the query rows of one key/value head (group heads x Nq tokens) against
// the keys j < lens[b] with j <= p_i (p_i: the row's position), and with a window W > 0
// only j > p_i - W or j < sinks. Online softmax, one division at the end; returns O and
// LSE like the other attention calls.
//
// Bound: memory, 1.25 d bytes a token and head (keys, values and their parameters), and
// close behind it instruction issue: the codes have to become matrix operands. So
//   * a unit of work is one request and key/value head with 4 NT query rows; its keys
//     are shared by all of them (a group of 8 heads reads the cache once);
//   * a warp runs its own stages of kSB blocks of 16 tokens: one lane per block fetches
//     it with one bulk copy (a block is contiguous), through a ring of kStages slots, and
//     no warp waits for another;
//   * products run as S^T = K Q^T and O^T = V^T P^T on mma.m16n8k16 with the keys (the
//     values' channels) as the 16 rows and the query rows as columns, so a few query rows
//     waste little. (tcgen05 would need 128 rows of unpacked bf16 keys in shared memory:
//     four times the traffic that the cache itself costs there.) The cache's word order
//     is the operand order;
//   * a code becomes a bf16 operand by masking alone: the bit pattern 0x000c is the
//     (subnormal) bf16 number c 2^-133 and 0x00c0 is c 2^-129, both exact for c = 0..15 (a
//     bf16 number is linear in its bits below 2^8 of them), so a word of eight codes costs
//     one shift and four masks. The other operand carries the power of two: query rows are
//     scaled to a largest value in [2^119, 2^120), weights P by 2^64; powers of two change
//     no bit of a result;
//   * a group's scale and zero point are applied to the fp32 sums for the keys,
//       s_j = sum over groups of scale_j (sum_i c_i q_i) + zero_j (sum_i q_i),
//     (a parameter word is itself a pair of bf16 numbers, scale and zero point: the second
//     sum is one more product, with the sums of q cut into three bf16 parts), and for the
//     values the scale goes to the weight:
//       O = sum_j (P_j scale_j) c_j + sum_j P_j zero_j, the second sum in fp32.
//     P_j scale_j enters as the sum of two bf16 numbers (16 bits of it), the high part in
//     the even and the low part in the odd column of a query row: four query rows per
//     8-column tile. One bf16 part alone would be off by 2^-8 of scale * c, several times
//     the value itself where the zero point cancels most of it;
//   * the stages of all units, one after another, are dealt evenly to all warps of a grid
//     of one block per SM, however ragged the batch and however few the units: a warp
//     takes a run of consecutive stages, and where it leaves a unit that others share it
//     writes that unit's partial (base, denominator, rows) to the workspace; a second
//     kernel joins them by the log-sum-exp rule of attn_merge, in stage order (no atomics:
//     results do not depend on timing). A unit that lies within one warp's run is finished
//     there. Warp w's partial of unit u has slot w + u: both only grow along the stages.
// Statistics and sums are fp32.
// Measured (32 query heads on 8, d = 128): 131 072 tokens 40 us (168 MB; the attention launch
// by itself 39 us, 4.4 TB/s); 32 requests of up to 8 192 tokens 53 to 57 us (224 MB; by itself 51
// us). 270 warp instructions a block of 16 tokens and head; instructions issue in 46% of the
// cycles and the ALU pipe is busy in 47%: what bounds it is latency, since a warp fetches
// into a slot only once it has computed on it.
//
// Pages are looked up in the table and checked against n_pages: keys on a page outside
// the cache are invisible. Rows of a page past a request's length may hold anything. Lengths,
// positions and the table are plain loads: the launch before this one (the plan, say) may
// write them while this kernel's blocks are already resident, which the read-only path
// (ld.global.nc) does not allow for.
#pragma once

#include <cuda_bf16.h>

#include <cstdint>
#include <type_traits>

#include "decode_common.cuh"
#include "kv4_layout.cuh"
#include "serve_params.h"
#include "serve_ptx.cuh"

namespace osx {

template <int D, int NT>
struct Kv4FwdCfg {
  // Eight warps of 255 registers, so that a stage's blocks run interleaved. Measured at
  // NT = 1, d = 128 (128k tokens / ragged batch of 32, us): 8 warps, stages of 4 blocks 40.7
  // / 56.0; 16 warps, stages of 2 (a block at a time in registers) 42.8 / 57.2; 12 warps,
  // stages of 3 42.0 / 56.5.
  static constexpr int kWarps = 8;
  static constexpr int kRows = 4 * NT;
  static constexpr int kSB = D == 128 && NT == 2 ? 2 : 4;  // blocks of 16 tokens per stage
  static constexpr int kStages = D == 128 && NT == 1 ? 2 : 4;
  // Two row tiles leave no registers for blocks side by side: a branch per block, taken or
  // not, keeps the next block's operands out of them.
  static constexpr bool kBlockBranch = NT == 2;
  static constexpr uint32_t kStageBytes = kSB * Kv4<D>::kBytes;
  static constexpr uint32_t kWarpBytes = kStages * kStageBytes;
  // each warp's queries as B operands, 16 bytes a lane, tile and group
  static constexpr uint32_t kQBytes = NT * Kv4<D>::kGroups * 512;
  static constexpr uint32_t kQOff = kWarps * kWarpBytes;
  static constexpr uint32_t kBarOff = kQOff + kWarps * kQBytes;
  static constexpr uint32_t kScanOff = kBarOff + kWarps * kStages * 8;  // [threads] + [warps]
  static constexpr uint32_t kCursorOff = kScanOff;  // [2 warps], after the scan
  static constexpr uint32_t kMiscOff = kScanOff + (kWarps * 32 + kWarps) * 8;
  static_assert(kWarps * 2 * 64 <= kWarps * 32 * 8, "cursors fit the scan's place");
  static constexpr uint32_t kSmemBytes = kMiscOff + kWarps * 4;
  static_assert(kStages * kSB <= 31, "block masks");
  static_assert(kSmemBytes <= 232448, "shared memory per block");
};

constexpr uint32_t kLowNibbles = 0x000f000fu;   // c 2^-133 in each half
constexpr uint32_t kHighNibbles = 0x00f000f0u;  // c 2^-129
constexpr float kPShift = 64.f;                 // weights carry 2^64

// The blocks of 16 tokens that request b's rows see: [0, n_s) of the sinks, then n_w from
// w0 on.
struct Kv4Span {
  int len, n_s, w0, n_blocks;
  long long p0;  // position of the first query token
  __device__ int block(int i) const { return i < n_s ? i : w0 + i - n_s; }
};

__device__ __forceinline__ Kv4Span kv4_span(const Kv4FwdParams& p, int b) {
  Kv4Span s;
  const long long room = (long long)p.width * p.blocks_per_page * 16;
  int len = p.lens[b];
  if (len < 0) len = 0;
  if (len > room) len = (int)room;
  s.len = len;
  s.p0 = p.q_pos ? (long long)p.q_pos[b] : (long long)len - p.Nq;
  const long long hi_l = s.p0 + p.Nq < len ? s.p0 + p.Nq : len;  // keys below may be seen
  const int hi = hi_l > 0 ? (int)hi_l : 0;
  const long long lo_l = p.window ? s.p0 - p.window + 1 : 0;
  const int lo = lo_l <= 0 ? 0 : (lo_l < hi ? (int)lo_l : hi);
  const int sink_end = p.window ? (p.sinks < hi ? p.sinks : hi) : 0;
  s.w0 = lo / 16;
  const int n_w = hi > lo ? (hi - 1) / 16 - s.w0 + 1 : 0;
  s.n_s = (sink_end + 15) / 16;
  if (n_w > 0 && s.n_s > s.w0) s.n_s = s.w0;
  s.n_blocks = s.n_s + n_w;
  return s;
}

// a / n for 0 <= a < 2^31, with magic = floor(2^32 / n) (2^32 - 1 for n = 1): the product's
// high word is the quotient or one less, since a (2^32 / n - magic) < 2^32
__device__ __forceinline__ int quotient(int a, int n, uint32_t magic) {
  const int q = (int)__umulhi((uint32_t)a, magic);
  return q + (a - q * n >= n ? 1 : 0);
}

// Stages of n blocks: 2^stage_shift blocks each.
__device__ __forceinline__ int kv4_stages(const Kv4FwdParams& p, int n) {
  return (n + (1 << p.stage_shift) - 1) >> p.stage_shift;
}

// A place in the stages: unit = (b Hkv + h) row_tiles + rt, and a stage of it.
struct Kv4Cursor {
  int unit, stage, n_stages;
  int h, rt, b;
  Kv4Span s;
};

__device__ __forceinline__ void kv4_enter(const Kv4FwdParams& p, Kv4Cursor& c) {
  c.s = kv4_span(p, c.b);
  c.n_stages = kv4_stages(p, c.s.n_blocks);
}

// Inclusive prefix sums over the block's threads; *total gets the sum. scan: [kWarps] words.
template <int kWarps>
__device__ __forceinline__ long long block_scan(long long x, long long* scan, long long* total) {
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
#pragma unroll
  for (int s = 1; s < 32; s *= 2) {
    const long long y = __shfl_up_sync(0xffffffffu, x, s);
    if (lane >= s) x += y;
  }
  __syncthreads();  // scan may still be read from a round before
  if (lane == 31) scan[warp] = x;
  __syncthreads();
  long long all = 0, before = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    if (w == warp) before = all;
    all += scan[w];
  }
  *total = all;
  return x + before;
}

template <int D, int NT>
__global__ void __launch_bounds__(Kv4FwdCfg<D, NT>::kWarps * 32, 1)
kv4_fwd_kernel(const __grid_constant__ Kv4FwdParams p) {
  using C = Kv4FwdCfg<D, NT>;
  using L = Kv4<D>;
  constexpr int kG = L::kGroups;
  constexpr int kThreads = C::kWarps * 32;
  extern __shared__ __align__(128) uint8_t smem[];
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, g = lane >> 2, t = lane & 3;
  uint8_t* ring = smem + warp * C::kWarpBytes;
  const uint32_t ring_u = smem_u32(ring);
  const uint32_t bar0 = smem_u32(smem + C::kBarOff) + warp * C::kStages * 8;
  long long* scan = reinterpret_cast<long long*>(smem + C::kScanOff);
  // (each warp has a flag of its own: no warp waits for another)
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::kMiscOff) + warp;
  if (lane == 0) {
    *abort_flag = 0;
    for (int s = 0; s < C::kStages; ++s) mbar_init(bar0 + 8 * s, 1);
    fence_mbar_init();
  }
  __syncwarp();
  grid_dependents_launch();
  grid_dependency_wait();

  // ---- this warp's run of stages: [t0, t1) of the units' stages, one unit after another
  // (no more runs than stages; neighbouring runs lie on different SMs, so that few of them
  // spread over the card)
  const long long wg = (long long)warp * gridDim.x + blockIdx.x;
  const int per_b = p.Hkv * p.row_tiles;  // units of a request
  const int warps = gridDim.x * C::kWarps;
  auto stages_of = [&](int bb) {  // of all of request bb's units
    return bb < p.B ? (long long)kv4_stages(p, kv4_span(p, bb).n_blocks) * per_b : 0ll;
  };
  long long total = 0, t0 = 0, t1 = 0, pre = 0;
  int b = 0;
  auto cut = [&]() {
    const long long runs = decode_runs(total, warps);
    if (wg < runs) {
      t0 = divide(total * wg, runs);
      t1 = divide(total * (wg + 1), runs);
    }
  };
  if (p.B <= 32) {  // within the warp
    const long long n = stages_of(lane);
    long long incl = n;
#pragma unroll
    for (int s = 1; s < 32; s *= 2) {
      const long long y = __shfl_up_sync(0xffffffffu, incl, s);
      if (lane >= s) incl += y;
    }
    total = __shfl_sync(0xffffffffu, incl, 31);
    if (blockIdx.x == 0 && warp == 0) {  // for the join
      if (lane < p.B) p.ws_prefix[lane] = incl - n;
      if (lane == 0) p.ws_prefix[p.B] = total;
    }
    cut();
    // the first request whose stages end behind t0
    const uint32_t behind = __ballot_sync(0xffffffffu, incl > t0);
    if (t0 < t1) {
      b = __ffs(behind) - 1;
      pre = __shfl_sync(0xffffffffu, incl - n, b);
    }
  } else {
    for (int pass = p.B > kThreads ? 0 : 1; pass < 2; ++pass) {
      // (more requests than threads: a first pass for the total)
      long long carry = 0;
      bool found = false;
      for (int base = 0; base < p.B; base += kThreads) {
        const int bb = base + threadIdx.x;
        const long long n = stages_of(bb);
        long long sum;
        const long long incl = carry + block_scan<C::kWarps>(n, scan + kThreads, &sum);
        if (pass == 1) {
          if (p.B <= kThreads) total = sum;
          if (blockIdx.x == 0 && bb < p.B) p.ws_prefix[bb] = incl - n;
          if (base == 0) cut();
          scan[threadIdx.x] = incl;
          __syncthreads();
          if (!found && t0 < t1 && t0 < carry + sum) {
            int lo = 0, hi = kThreads - 1;
            while (lo < hi) {
              const int mid = (lo + hi) / 2;
              if (scan[mid] > t0) hi = mid; else lo = mid + 1;
            }
            b = base + lo;
            pre = lo > 0 ? scan[lo - 1] : carry;
            found = true;
          }
        }
        carry += sum;
      }
      if (pass == 0) total = carry;
      if (pass == 1 && blockIdx.x == 0 && threadIdx.x == 0) p.ws_prefix[p.B] = total;
    }
    __syncthreads();  // the cursors take the scan's place
  }
  if (t0 >= t1) return;

  // ---- two cursors over the run: where to compute, and where to fetch. They live in shared
  // memory: registers are what the products need
  Kv4Cursor& cur = reinterpret_cast<Kv4Cursor*>(smem + C::kCursorOff)[2 * warp];
  Kv4Cursor& fet = (&cur)[1];
  {
    Kv4Cursor c;
    c.b = b;
    kv4_enter(p, c);
    const int in_b = (int)divide(t0 - pre, c.n_stages);  // unit within the request
    c.stage = (int)((t0 - pre) - (long long)in_b * c.n_stages);
    c.h = in_b / p.row_tiles;
    c.rt = in_b - c.h * p.row_tiles;
    c.unit = b * per_b + in_b;
    if (lane == 0) cur = fet = c;
    __syncwarp();
  }
  int left = (int)(t1 - t0);  // stages to compute
  int to_fetch = left;
  // a cursor to the next unit (the run goes on, so there is one)
  auto next_unit = [&](Kv4Cursor& at) {
    Kv4Cursor c = at;
    ++c.unit;
    c.stage = 0;
    if (++c.rt == p.row_tiles) {
      c.rt = 0;
      if (++c.h == p.Hkv) {
        c.h = 0;
        do {  // the next request that has a stage
          ++c.b;
          kv4_enter(p, c);
          if (c.n_stages == 0) c.unit += per_b;
        } while (c.n_stages == 0 && c.b + 1 < p.B);
      }
    }
    __syncwarp();
    if (lane == 0) at = c;
    __syncwarp();
  };

  // ---- this lane's page of the fetch cursor's stage (a lane per block), -1: none
  int page_next = -1, in_page = 0;
  auto look_up = [&](int stage) {
    const int bi = (stage << p.stage_shift) + lane;
    page_next = -1;
    if (lane < 1 << p.stage_shift && bi < fet.s.n_blocks) {
      const int lb = fet.s.block(bi);
      const int pg = quotient(lb, p.blocks_per_page, p.page_magic);
      in_page = lb - pg * p.blocks_per_page;
      page_next = p.table[(long long)fet.b * p.width + pg];
    }
  };
  int fetch_stage = fet.stage;
  uint32_t masks = 0;  // blocks present, kSB bits per slot
  auto fetch = [&](int slot) {  // the fetch cursor's stage into a slot; then on to the next
    const bool ok = page_next >= 0 && page_next < p.n_pages;
    const uint32_t mk = __ballot_sync(0xffffffffu, ok);
    masks = (masks & ~(((1u << C::kSB) - 1u) << (C::kSB * slot))) | (mk << (C::kSB * slot));
    if (lane == 0) mbar_arrive_expect_tx(bar0 + 8 * slot, __popc(mk) * L::kBytes);
    __syncwarp();
    if (ok) {
      const uint32_t* src =
          p.cache +
          (((long long)page_next * p.Hkv + fet.h) * p.blocks_per_page + in_page) * L::kWords;
      bulk_load(ring_u + slot * C::kStageBytes + lane * L::kBytes, src, L::kBytes, bar0 + 8 * slot);
    }
    if (--to_fetch > 0) {
      if (++fetch_stage == fet.n_stages) {
        next_unit(fet);
        fetch_stage = 0;
      }
      look_up(fetch_stage);
    }
  };
  look_up(fetch_stage);
  int n_issued = 0, waited = 0;
#pragma unroll
  for (int k = 0; k < C::kStages; ++k)
    if (to_fetch > 0) {
      fetch(k);
      ++n_issued;
    }

  uint4* qsm = reinterpret_cast<uint4*>(smem + C::kQOff + warp * C::kQBytes);
  int slot = 0, phase = 0;
  bool ok = true;
  while (left > 0) {
    // ================================================================ one unit (or a part)
    const int first_stage = cur.stage;

    // ---- queries: B operands. Column n of tile nt is row 4 nt + n / 2; its odd column (the
    // weights' low part) has no part in the scores. Lane (g, t) holds, for column g and each
    // group i, values 32 i + 8 t + (0..7) paired as the codes come out of a word: (0, 4),
    // (1, 5), (2, 6), (3, 7), the second and last pair against codes that carry 2^4
    const int row0 = cur.rt * C::kRows;
    const int rows = p.rows - row0 < C::kRows ? p.rows - row0 : C::kRows;
    const long long q_row0 = ((long long)cur.b * p.Hkv + cur.h) * p.rows + row0;  // (b Hq + h) Nq + i
    // (in shared memory, for the registers' sake)
    // the sum of column n's row over group t (with the scores' power of two) in three bf16
    // parts, each against the zero point of a parameter word
    uint32_t qz[NT][3];
    float c_row[NT];      // score to log2 units, row 4 nt + t
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int r = nt * 4 + (g >> 1);
      uint4 u[kG];
      uint32_t top = 0;  // largest exponent field of the row
#pragma unroll
      for (int i = 0; i < kG; ++i) {
        u[i] = make_uint4(0, 0, 0, 0);
        if (r < rows)
          u[i] = *reinterpret_cast<const uint4*>(p.q + (q_row0 + r) * D + 32 * i + 8 * t);
        const uint32_t w[4] = {u[i].x, u[i].y, u[i].z, u[i].w};
#pragma unroll
        for (int e = 0; e < 4; ++e)
          top = max(top, max(w[e] & 0x7f80u, (w[e] >> 16) & 0x7f80u));
      }
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
      // q 2^k, k = 119 - E for a largest value in [2^E, 2^(E + 1)); at most 2^127
      const int E = (int)(top >> 7) - 127;
      const int k = 119 - E < 127 ? 119 - E : 127;
      const float up = __uint_as_float((uint32_t)(k + 127) << 23);
      const float up4 = up * 0.0625f;
      float sum[kG];
#pragma unroll
      for (int i = 0; i < kG; ++i) {
        uint32_t qf[4];
        // u: pairs (0,1) (2,3) (4,5) (6,7)
        const uint32_t pr[4] = {
            __byte_perm(u[i].x, u[i].z, 0x5410), __byte_perm(u[i].x, u[i].z, 0x7632),
            __byte_perm(u[i].y, u[i].w, 0x5410), __byte_perm(u[i].y, u[i].w, 0x7632)};
        sum[i] = 0.f;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float lo = __uint_as_float(pr[e] << 16), hi = __uint_as_float(pr[e] & 0xffff0000u);
          const float f = (e & 1) ? up4 : up;
          qf[e] = (g & 1) ? 0u : pack_bf16x2(lo * f, hi * f);
          sum[i] += lo + hi;
        }
        qsm[(nt * kG + i) * 32 + lane] = make_uint4(qf[0], qf[1], qf[2], qf[3]);
        sum[i] += __shfl_xor_sync(0xffffffffu, sum[i], 1);
        sum[i] += __shfl_xor_sync(0xffffffffu, sum[i], 2);  // the row's sum, on its four lanes
      }
      // row 4 nt + t is column 2 t: lanes 8 t ..
      const int kt = __shfl_sync(0xffffffffu, k, 8 * t);
      const float down = __uint_as_float((uint32_t)(kt > 6 ? kt - 6 : 0) << 23);  // 2^(k - 133)
      {
        const float own = __uint_as_float((uint32_t)(k > 6 ? k - 6 : 0) << 23);
        float x = 0.f;
#pragma unroll
        for (int i = 0; i < kG; ++i)
          if (i == t) x = (g & 1) ? 0.f : sum[i] * own;
#pragma unroll
        for (int e = 0; e < 3; ++e) {
          qz[nt][e] = pack_bf16x2(0.f, x);
          x -= __uint_as_float(qz[nt][e] & 0xffff0000u);
        }
      }
      c_row[nt] = p.scale_log2 * (down > 0.f ? 1.f / down : 0.f);
    }
    // stages [in_lo, in_hi) lie inside what every row sees (keys all_lo .. all_hi): past the
    // sinks' blocks, and no block of them past the request's length
    int in_lo, in_hi;
    {
      const Kv4Span& sp = cur.s;
      const int all_hi = sp.p0 < sp.len - 1 ? (sp.p0 < -1 ? -1 : (int)sp.p0) : sp.len - 1;
      const long long al = p.window ? sp.p0 + p.Nq - p.window : 0;
      const int all_lo = al <= 0 ? 0 : (al < 0x7fffffff - 15 ? (int)al : 0x7fffffff - 15);
      const int b_lo = (all_lo + 15) / 16, b_hi = (all_hi + 1) / 16;  // whole blocks
      const int i_lo = sp.n_s + (b_lo > sp.w0 ? b_lo - sp.w0 : 0);  // places in the unit's list
      const int i_hi = sp.n_s + b_hi - sp.w0;
      in_lo = kv4_stages(p, i_lo);
      in_hi = i_hi > 0 ? i_hi >> p.stage_shift : 0;
    }

    // columns 2t and 2t + 1 (high and low parts) of channels 16 mt + g and 16 mt + 8 + g
    float o[NT][D / 16][4] = {};
    float zo[NT][kG] = {};
    float m[NT], l[NT];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      m[nt] = -INFINITY;
      l[nt] = 0.f;
    }

    const int stop = cur.n_stages - first_stage < left ? cur.n_stages : first_stage + left;
    left -= stop - first_stage;
    for (int st = first_stage; st < stop; ++st) {
      ok = mbar_wait(bar0 + 8 * slot, phase, abort_flag, p.status);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      ++waited;
      const uint8_t* stage = ring + slot * C::kStageBytes;
      const uint32_t present = masks >> (C::kSB * slot);
      constexpr uint32_t kAll = (1u << C::kSB) - 1u;
      const bool inside = st >= in_lo && st < in_hi && (present & kAll) == kAll;
      auto compute = [&](auto edge) {
        constexpr bool kEdge = decltype(edge)::value;
        // ---- scores
        float sc[C::kSB][NT][2];  // keys g and g + 8 of a block
#pragma unroll
        for (int j = 0; j < C::kSB; ++j) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) sc[j][nt][0] = sc[j][nt][1] = -INFINITY;
          if ((kEdge || C::kBlockBranch) && !((present >> j) & 1u)) continue;
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
          // zero points against the sums of q: slots 2t, 2t + 1 are (scale, zero) of group t
          float y[NT][4];
          {
            const uint32_t* kp = blk + L::kKParams + (t & (kG - 1));
            const uint32_t za = kp[g * kG], zb = kp[(g + 8) * kG];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              mma16816_zero(y[nt], za, zb, za, zb, qz[nt][0], qz[nt][1]);
              mma1688(y[nt], za, zb, qz[nt][2]);
            }
          }
#pragma unroll
          for (int i = 0; i < kG; ++i) {
            uint32_t a[2][4];
#pragma unroll
            for (int r = 0; r < 2; ++r) {
              const uint32_t w8 = w[r][i] >> 8;
              a[r][0] = w[r][i] & kLowNibbles;
              a[r][1] = w[r][i] & kHighNibbles;
              a[r][2] = w8 & kLowNibbles;
              a[r][3] = w8 & kHighNibbles;
            }
            const float s0 = param_scale(par[0][i]), s1 = param_scale(par[1][i]);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              float c[4];
              const uint4 q = qsm[(nt * kG + i) * 32 + lane];  // this lane's own
              mma16816_zero(c, a[0][0], a[1][0], a[0][1], a[1][1], q.x, q.y);
              mma16816(c, a[0][2], a[1][2], a[0][3], a[1][3], q.z, q.w);
              y[nt][0] = fmaf(s0, c[0], y[nt][0]);
              y[nt][2] = fmaf(s1, c[2], y[nt][2]);
            }
          }
          if constexpr (kEdge) {
            const int k0 = cur.s.block((st << p.stage_shift) + j) * 16;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              const long long pos = cur.s.p0 + (row0 + nt * 4 + t) % p.Nq;
#pragma unroll
              for (int x = 0; x < 2; ++x) {
                const int key = k0 + g + 8 * x;
                if (key < cur.s.len && key <= pos &&
                    (!p.window || key > pos - p.window || key < p.sinks))
                  sc[j][nt][x] = y[nt][2 * x];
              }
            }
          } else {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) sc[j][nt][0] = y[nt][0], sc[j][nt][1] = y[nt][2];
          }
        }

        // ---- bases: moved only when a score exceeds one by more than 8 (log2 units), so the
        // maximum over the warp's lanes is rarely needed
        bool grows = false;
        float mx[NT];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          float y = -INFINITY;
#pragma unroll
          for (int j = 0; j < C::kSB; ++j) y = fmax3(y, sc[j][nt][0], sc[j][nt][1]);
          mx[nt] = y == -INFINITY ? y : y * c_row[nt];
          grows |= mx[nt] > m[nt] + 8.f;
        }
        if (__any_sync(0xffffffffu, grows)) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            float y = mx[nt];
#pragma unroll
            for (int d = 4; d < 32; d *= 2) y = fmaxf(y, __shfl_xor_sync(0xffffffffu, y, d));
            if (y > m[nt] + 8.f) {
              const float a = ex2_approx(m[nt] - y);  // 0 from -inf
              m[nt] = y;
              l[nt] *= a;
#pragma unroll
              for (int i = 0; i < kG; ++i) zo[nt][i] *= a;
#pragma unroll
              for (int i = 0; i < D / 16; ++i)
#pragma unroll
                for (int x = 0; x < 4; ++x) o[nt][i][x] *= a;
            }
          }
        }

        // ---- P, and O^T += V^T P^T block by block
#pragma unroll
        for (int j = 0; j < C::kSB; ++j) {
          if ((kEdge || C::kBlockBranch) && !((present >> j) & 1u)) continue;
          const uint32_t* blk = reinterpret_cast<const uint32_t*>(stage + j * L::kBytes);
          float pr[NT][2];
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            const float base = (m[nt] == -INFINITY ? 0.f : m[nt]) - kPShift;
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              pr[nt][x] = ex2_approx(fmaf(sc[j][nt][x], c_row[nt], -base));  // 0 where masked
              l[nt] += pr[nt][x];
            }
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
          }
          uint32_t bp[NT][kG][2];
#pragma unroll
          for (int i = 0; i < kG; ++i) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
              for (int r = 0; r < 2; ++r) {
                // a token that the row does not see may hold any bits: 0 * NaN is not 0
                const uint32_t pm = kEdge && sc[j][nt][r] == -INFINITY ? 0u : par[r][i];
                const float x = pr[nt][r] * param_scale(pm);
                const float high = __uint_as_float(__float_as_uint(x) & 0xffff0000u);
                // (the low part is rounded, not cut: cut ones would all err to one side, and
                // over a long context the small sums that are left show it)
                bp[nt][i][r] = transpose_b16(pack_bf16x2(high, x - high));
                zo[nt][i] = fmaf(pr[nt][r], param_zero(pm), zo[nt][i]);
              }
            }
          }
#pragma unroll
          for (int h = 0; h < D / 64; ++h) {
            const uint4 a = *reinterpret_cast<const uint4*>(blk + L::kVCodes + (h * 32 + lane) * 4);
            // codes of the keys (2t, 2t + 1) and (2t + 8, 2t + 9), side by side
            const uint32_t u0[2] = {__byte_perm(a.x, a.y, 0x5410), __byte_perm(a.x, a.y, 0x7632)};
            const uint32_t u1[2] = {__byte_perm(a.z, a.w, 0x5410), __byte_perm(a.z, a.w, 0x7632)};
#pragma unroll
            for (int mm = 0; mm < 4; ++mm) {
              const uint32_t x = u0[mm >> 1] >> (8 * (mm & 1)), y = u1[mm >> 1] >> (8 * (mm & 1));
              const int mt = 4 * h + mm;
#pragma unroll
              for (int nt = 0; nt < NT; ++nt)  // rows g: c 2^-133, rows g + 8: c 2^-129
                mma16816(o[nt][mt], x & kLowNibbles, x & kHighNibbles, y & kLowNibbles,
                         y & kHighNibbles, bp[nt][mt / 2][0], bp[nt][mt / 2][1]);
            }
          }
        }
      };
      if (inside)
        compute(std::false_type{});
      else
        compute(std::true_type{});
      __syncwarp();  // every lane has read the slot
      if (to_fetch > 0) {
        fetch(slot);
        ++n_issued;
      }
      if (++slot == C::kStages) {
        slot = 0;
        phase ^= 1;
      }
    }
    if (!ok) break;

    // ---- rows out: finished if the unit began and ended here, else a partial
    const bool whole = first_stage == 0 && stop == cur.n_stages;
    float* ws_o = p.ws_o + (wg + cur.unit) * (C::kRows * D);
    float* ws_ml = p.ws_ml + (wg + cur.unit) * (C::kRows * 2);
    constexpr float kDown = 0x1p-64f;                   // the weights' power of two
    constexpr float kLow = 0x1p+69f, kHigh = 0x1p+65f;  // 2^133 and 2^129, less that
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      float sum = l[nt];
#pragma unroll
      for (int d = 4; d < 32; d *= 2) sum += __shfl_xor_sync(0xffffffffu, sum, d);
      sum *= kDown;
      const int r = nt * 4 + t;
      const float inv = whole ? (sum > 0.f ? 1.f / sum : 0.f) : 1.f;
      if (g == 0) {
        if (!whole)
          *reinterpret_cast<float2*>(ws_ml + 2 * r) = make_float2(m[nt], sum);
        else if (r < rows)
          p.lse[q_row0 + r] =
              sum > 0.f ? (m[nt] + lg2_approx(sum)) * 0.69314718055994530942f : -INFINITY;
      }
#pragma unroll
      for (int i = 0; i < kG; ++i) {
        float z = zo[nt][i];
#pragma unroll
        for (int d = 4; d < 32; d *= 2) z += __shfl_xor_sync(0xffffffffu, z, d);
        z *= kDown;
#pragma unroll
        for (int h = 0; h < 2; ++h) {  // channels 16 mt + g and + 8
          const float(&x)[4] = o[nt][2 * i + h];
          const float y0 = fmaf(x[0] + x[1], kLow, z) * inv;
          const float y1 = fmaf(x[2] + x[3], kHigh, z) * inv;
          const int at = 32 * i + 16 * h + g;
          if (!whole) {
            ws_o[r * D + at] = y0;
            ws_o[r * D + at + 8] = y1;
          } else if (r < rows) {
            const long long e = (q_row0 + r) * D + at;
            if (p.o_bf16) {
              static_cast<__nv_bfloat16*>(p.o)[e] = __float2bfloat16_rn(y0);
              static_cast<__nv_bfloat16*>(p.o)[e + 8] = __float2bfloat16_rn(y1);
            } else {
              static_cast<float*>(p.o)[e] = y0;
              static_cast<float*>(p.o)[e + 8] = y1;
            }
          }
        }
      }
    }
    if (left > 0) next_unit(cur);
  }
  if (!ok) {
    // a wait ran out: let the copies still in flight land before the block ends
    for (; waited < n_issued; ++waited) {
      mbar_wait_drain(bar0 + 8 * slot, phase, 100000000ull);
      if (++slot == C::kStages) {
        slot = 0;
        phase ^= 1;
      }
    }
  }
}

}  // namespace osx
