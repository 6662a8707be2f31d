// window_token_kernel.cuh - attention with a sliding window and sinks for a few newest
// tokens: the form of attn_window_fwd whose query rows would leave a 128-row tensor-core
// tile almost empty.
//
// Bound: memory, 4 d bytes a key and key/value head. A warp takes a run of 16-key blocks
// (decode_common.cuh), all query rows of the key/value head (the group's heads times the
// tokens, 4 NT at a time) against each, and no warp waits for another. Keys and values go
// from global memory straight to the registers that feed mma.m16n8k16, 16 bytes a lane:
// no shared memory, no exchange, whole sectors. That works because the order of the
// summed index of a product is free:
//   S^T = K Q^T (rows: keys): lane (g, t) loads values 32 i + 8 t + (0..7) of keys g and
//     g + 8 as they lie, and holds the same values of its query rows;
//   O^T = V^T P^T (rows: channels): lane (g, t) loads channels 8 g + (0..7) (and 64 more)
//     of keys 2t, 2t + 1, 2t + 8, 2t + 9; tile e takes channel e of each, two keys side by
//     side after one byte permutation.
// Half of a block's registers are always in flight: the next block's keys are fetched once
// this one's scores are formed, its values once this one's products are issued.
//
// Measured: 4 requests, 32 query heads on 8, d = 128, window 4096: 14.5 us (67 MB, 4.6 TB/s),
// 17.0 us with the join; on 128-row tiles the same call took 65 us.
//
// A weight P enters as the sum of two bf16 numbers (16 bits of it), the high part in the
// even and the low part in the odd column of a query row: with four query rows to an
// 8-column tile the second part costs nothing, and the result is as exact as fp32 weights
// leave it.
#pragma once

#include <cuda_bf16.h>

#include <cstdint>

#include "decode_common.cuh"

namespace osx {

template <int NT>
struct TokenCfg {
  static constexpr int kRows = 4 * NT;
  static constexpr int kWarps = NT == 1 ? 12 : 8;  // 168 or 255 registers a thread
};

template <int D, int NT>
__global__ void __launch_bounds__(TokenCfg<NT>::kWarps * 32, 1)
window_token_kernel(const __grid_constant__ TokenParams p) {
  using C = TokenCfg<NT>;
  constexpr int kI = D / 32;  // 32-value pieces of a row
  constexpr int kH = D / 64;  // 64-channel halves
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, g = lane >> 2, t = lane & 3;
  grid_dependents_launch();

  // ---- this warp's run of blocks
  const int n = p.n_blocks;
  const int per_b = p.Hkv * p.row_tiles;
  const long long total = (long long)p.B * per_b * n;
  const long long runs = decode_runs(total, gridDim.x * C::kWarps);
  const long long wg = (long long)warp * gridDim.x + blockIdx.x;
  if (wg >= runs) return;
  const long long t0 = divide(total * wg, runs), t1 = divide(total * (wg + 1), runs);
  int left = (int)(t1 - t0);
  int unit = (int)divide(t0, n);
  int blk = (int)(t0 - (long long)unit * n);

  auto first_key = [&](int i) { return (i < p.n_sink_blocks ? i : p.w0 + i - p.n_sink_blocks) * 16; };
  uint4 kr[2][kI], vr[4][kH];
  auto head_of = [&](int u) { return u / p.row_tiles; };  // b Hkv + h
  auto load_k = [&](int u, int i) {
    const int k0 = first_key(i);
    const __nv_bfloat16* row = p.k + ((long long)head_of(u) * p.kv_ld + k0 + g) * D + 8 * t;
#pragma unroll
    for (int r = 0; r < 2; ++r)
#pragma unroll
      for (int x = 0; x < kI; ++x)
        kr[r][x] = k0 + g + 8 * r < p.Nkv
                       ? __ldcs(reinterpret_cast<const uint4*>(row + 8 * r * D + 32 * x))
                       : make_uint4(0, 0, 0, 0);
  };
  auto load_v = [&](int u, int i) {
    const int k0 = first_key(i);
    const __nv_bfloat16* row = p.v + ((long long)head_of(u) * p.kv_ld + k0 + 2 * t) * D + 8 * g;
#pragma unroll
    for (int kk = 0; kk < 4; ++kk) {
      const int key = 8 * (kk >> 1) + (kk & 1);  // beyond 2t
#pragma unroll
      for (int h = 0; h < kH; ++h)
        vr[kk][h] = k0 + 2 * t + key < p.Nkv
                        ? __ldcs(reinterpret_cast<const uint4*>(row + key * D + 64 * h))
                        : make_uint4(0, 0, 0, 0);
    }
  };
  grid_dependency_wait();
  load_k(unit, blk);
  load_v(unit, blk);

  while (left > 0) {
    // ================================================================ one unit (or a part)
    const int first = blk;
    const int stop = n - first < left ? n : first + left;
    const int head = head_of(unit), row0 = (unit - head * p.row_tiles) * C::kRows;
    const int rows = p.rows - row0 < C::kRows ? p.rows - row0 : C::kRows;
    // queries: column n of tile nt is row 4 nt + n / 2; its odd column has no part in scores
    uint4 qr[NT][kI];
    long long pos[NT];  // position of row 4 nt + t, in key rows
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int r = nt * 4 + (g >> 1);
      const int rg = row0 + r;  // row of the head: (head of the group, token)
#pragma unroll
      for (int x = 0; x < kI; ++x) {
        qr[nt][x] = make_uint4(0, 0, 0, 0);
        if (r < rows && !(g & 1)) {
          const long long hq = (long long)head * (p.rows / p.Nq) + rg / p.Nq;  // b Hq + head
          qr[nt][x] = *reinterpret_cast<const uint4*>(p.q + (hq * p.q_ld + rg % p.Nq) * D + 32 * x +
                                                      8 * t);
        }
      }
      pos[nt] = p.rel + (row0 + nt * 4 + t) % p.Nq;
    }
    float o[NT][D / 16][4] = {};
    float m[NT], l[NT];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      m[nt] = -INFINITY;
      l[nt] = 0.f;
    }

    for (int i = first; i < stop; ++i) {
      // where the run goes on
      const bool last = i + 1 == stop;
      const int u2 = last && stop == n ? unit + 1 : unit;
      const int i2 = last && stop == n ? 0 : i + 1;
      const bool more = !last || left > stop - first;
      const int k0 = first_key(i);

      // ---- scores of keys g and g + 8
      float y[NT][4];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        mma16816_zero(y[nt], kr[0][0].x, kr[1][0].x, kr[0][0].y, kr[1][0].y, qr[nt][0].x, qr[nt][0].y);
        mma16816(y[nt], kr[0][0].z, kr[1][0].z, kr[0][0].w, kr[1][0].w, qr[nt][0].z, qr[nt][0].w);
#pragma unroll
        for (int x = 1; x < kI; ++x) {
          mma16816(y[nt], kr[0][x].x, kr[1][x].x, kr[0][x].y, kr[1][x].y, qr[nt][x].x, qr[nt][x].y);
          mma16816(y[nt], kr[0][x].z, kr[1][x].z, kr[0][x].w, kr[1][x].w, qr[nt][x].z, qr[nt][x].w);
        }
      }
      if (more) load_k(u2, i2);
      float sc[NT][2];
      // (the same for the warp) is the block inside what every row sees?
      const bool inside = k0 + 15 <= p.rel && k0 + 15 < p.Nkv &&
                          (k0 > p.rel + p.Nq - 1 - p.window || k0 + 15 < p.sinks);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const int key = k0 + g + 8 * x;
          const bool see = inside || (key < p.Nkv && key <= pos[nt] &&
                                      (key > pos[nt] - p.window || key < p.sinks));
          sc[nt][x] = see ? y[nt][2 * x] : -INFINITY;
        }

      // ---- bases: moved only when a score exceeds one by more than 8 (log2 units)
      bool grows = false;
      float mx[NT];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const float top = fmaxf(sc[nt][0], sc[nt][1]);
        mx[nt] = top == -INFINITY ? top : top * p.scale_log2;
        grows |= mx[nt] > m[nt] + 8.f;
      }
      if (__any_sync(0xffffffffu, grows)) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          float top = mx[nt];
#pragma unroll
          for (int d = 4; d < 32; d *= 2) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
          if (top > m[nt] + 8.f) {
            const float a = ex2_approx(m[nt] - top);  // 0 from -inf
            m[nt] = top;
            l[nt] *= a;
#pragma unroll
            for (int e = 0; e < D / 16; ++e)
#pragma unroll
              for (int x = 0; x < 4; ++x) o[nt][e][x] *= a;
          }
        }
      }

      // ---- P and O^T += V^T P^T
      uint32_t b0[NT], b1[NT];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const float base = m[nt] == -INFINITY ? 0.f : m[nt];
        uint32_t part[2];
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const float w = ex2_approx(fmaf(sc[nt][x], p.scale_log2, -base));  // 0 where masked
          l[nt] += w;
          const float high = __uint_as_float(__float_as_uint(w) & 0xffff0000u);
          part[x] = pack_bf16x2(high, w - high);
        }
        b0[nt] = transpose_b16(part[0]);
        b1[nt] = transpose_b16(part[1]);
      }
#pragma unroll
      for (int e = 0; e < D / 16; ++e) {
        // channel of rows g and g + 8: e of both halves (d = 128), e and e + 4 (d = 64)
        const int e1 = kH == 2 ? e : e + 4;
        auto word = [](const uint4& u, int w) { return w == 0 ? u.x : w == 1 ? u.y : w == 2 ? u.z : u.w; };
        const uint32_t s0 = (e & 1) ? 0x7632 : 0x5410, s1 = (e1 & 1) ? 0x7632 : 0x5410;
        const uint32_t a0 = __byte_perm(word(vr[0][0], e / 2), word(vr[1][0], e / 2), s0);
        const uint32_t a1 = __byte_perm(word(vr[0][kH - 1], e1 / 2), word(vr[1][kH - 1], e1 / 2), s1);
        const uint32_t a2 = __byte_perm(word(vr[2][0], e / 2), word(vr[3][0], e / 2), s0);
        const uint32_t a3 = __byte_perm(word(vr[2][kH - 1], e1 / 2), word(vr[3][kH - 1], e1 / 2), s1);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) mma16816(o[nt][e], a0, a1, a2, a3, b0[nt], b1[nt]);
      }
      if (more) load_v(u2, i2);
    }
    left -= stop - first;

    // ---- rows out: finished if the unit began and ended here, else a partial
    const bool whole = first == 0 && stop == n;
    const long long slot = wg + unit;
    const long long out0 = (long long)head * p.rows + row0;  // dense rows of O and LSE
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      float sum = l[nt];
#pragma unroll
      for (int d = 4; d < 32; d *= 2) sum += __shfl_xor_sync(0xffffffffu, sum, d);
      const int r = nt * 4 + t;
      const float inv = whole ? (sum > 0.f ? 1.f / sum : 0.f) : 1.f;
      if (g == 0) {
        if (!whole)
          *reinterpret_cast<float2*>(p.ws_ml + (slot * C::kRows + r) * 2) = make_float2(m[nt], sum);
        else if (r < rows)
          p.lse[out0 + r] = sum > 0.f ? (m[nt] + lg2_approx(sum)) * 0.69314718055994530942f : -INFINITY;
      }
      // channels 8 g + (0..7) of each half
#pragma unroll
      for (int h = 0; h < kH; ++h) {
        float y[8];
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          const float(&x)[4] = o[nt][kH == 2 ? c : c & 3];
          const int lo = (kH == 2 ? h : c >> 2) * 2;  // rows g + 8
          y[c] = (x[lo] + x[lo + 1]) * inv;
        }
        const int at = 64 * h + 8 * g;
        if (!whole || (r < rows && !p.o_bf16)) {
          float* dst = whole ? static_cast<float*>(p.o) + (out0 + r) * D + at
                             : p.ws_o + (slot * C::kRows + r) * D + at;
          reinterpret_cast<float4*>(dst)[0] = make_float4(y[0], y[1], y[2], y[3]);
          reinterpret_cast<float4*>(dst)[1] = make_float4(y[4], y[5], y[6], y[7]);
        } else if (r < rows) {
          *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.o) + (out0 + r) * D + at) =
              make_uint4(pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]), pack_bf16x2(y[4], y[5]),
                         pack_bf16x2(y[6], y[7]));
        }
      }
    }
    ++unit;
    blk = 0;
  }
}

}  // namespace osx
