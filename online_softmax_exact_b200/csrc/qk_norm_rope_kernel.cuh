// qk_norm_rope_kernel.cuh - norms of queries and keys for each head with the position
// rotation in the same pass, from the packed projection to head-major tensors.
//
// For a head's row x of d values (queries and keys):
//   y = x * rsqrt(mean(x^2) + eps) * w,
//   (u, v) -> (u cos a - v sin a, v cos a + u sin a),  a = position * inv_freq[j],
// over the pairs j of the first r = 2 * n_freq values: (y[j], y[j + r/2]), or interleaved
// (y[2j], y[2j + 1]); the other values stay. Value rows are copied. Everything is in fp32
// and rounded to bf16 once.
//
// Bound: memory (each value is read once and written once; the projection is token-major
// and attention takes head-major rows, so this pass is also the transposition). What
// stands beside it is instruction issue, which the layout keeps down: a warp runs through
// a token's heads (or through 1/split of them, where tokens are few) with the norm weights
// already multiplied into the token's cosines and sines, rows ahead in flight up to the
// next token's; no warp waits for another. A lane holds four values and their four
// rotation partners of a row (d/8 lanes a row, 8-byte accesses that join to whole 128-byte
// lines), so a rotation needs no exchange between lanes; arithmetic is in packed fp32
// pairs.
//
// Measured: 32 768 tokens of 32 + 2 * 8 heads, d = 128 (805 MB): 140 us in a short run, 145
// us under power, 5.6 TB/s; a block per token with whole-block barriers took 190. One token
// of 32 requests: 4.1 us.
//
// Angles: position * inv_freq in 64 bits, reduced to [-pi, pi] in 64 bits, and only then
// sine and cosine in fp32. An fp32 product would be off by 2^-24 of an angle of up to
// 10^5 radians, several times the bf16 spacing of the result.
#pragma once

#include <cuda_bf16.h>

#include <cstdint>

#include "serve_params.h"
#include "serve_ptx.cuh"

namespace osx {

constexpr int kRopeThreads = 256;

__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  uint32_t d;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}

__device__ __forceinline__ uint64_t widen2(uint32_t w) {  // two bf16 to a pair
  return f2_pack(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}
__device__ __forceinline__ uint32_t narrow2(uint64_t v) {
  float a, b;
  f2_unpack(v, a, b);
  return pack2(a, b);
}

// position * inv_freq reduced to [-pi, pi], and its cosine and sine
__device__ __forceinline__ void rope_angle(int position, float inv_freq, float* c, float* s) {
  const double a = (double)position * (double)inv_freq;
  const double turns = rint(a * 0.15915494309189535);  // a / (2 pi)
  // 2 pi as a sum of two doubles; the first product is exact up to one rounding by fma
  const float r = (float)fma(-turns, 2.4492935982947064e-16, fma(-turns, 6.283185307179586, a));
  __sincosf(r, s, c);  // within 2^-21 on [-pi, pi]
}

template <int D, bool kInterleaved>
__global__ void __launch_bounds__(kRopeThreads, 4) qk_norm_rope_kernel(
    const __grid_constant__ RopeParams p, int split) {
  constexpr int kLanes = D / 8;         // lanes per row
  constexpr int kRows = 32 / kLanes;    // rows of a warp's pass
  constexpr int kAhead = 3;             // passes in flight (2: 167 us, 3: 140, 4: 146, 6: 149)
  constexpr int kWarps = kRopeThreads / 32;
  __shared__ __align__(16) float s_cos[kWarps][D / 2], s_sin[kWarps][D / 2];
  __shared__ __align__(16) float s_w[2][D];
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int c = lane % kLanes, sub = lane / kLanes;
  const int total = p.B * p.N, half = p.n_freq;
  float* cosw = s_cos[warp];
  float* sinw = s_sin[warp];

  // this lane's two runs of four values of a row: rotation partners i and i + half, eight
  // neighbours (interleaved pairs), or eight values that stay
  const bool turned = c < half / 4;
  const int at0 = kInterleaved ? 8 * c : (turned ? 4 * c : 2 * half + 8 * (c - half / 4));
  const int at1 = !kInterleaved && turned ? half + 4 * c : at0 + 4;

  // The warps that share a token take turns with its rows (heads in the projection's order),
  // kRows at a time: this lane's rows are first, first + per, ...
  const long long gw = (long long)blockIdx.x * kWarps + warp;  // this warp among all
  const int H = p.Hq + 2 * p.Hkv, n_qk = p.Hq + p.Hkv;
  const int per = kRows * split, first = (int)(gw % split) * kRows + sub;
  const int passes = (H + per - 1) / per;
  auto token_rows = [&](int token) {  // this lane's first row
    const int b = token / p.N;
    return p.qkv + (b * p.stride_b + (token - b * p.N) * p.stride_n + first * D);
  };
  uint2 x[kAhead][2];
  auto load = [&](int a, const __nv_bfloat16* row, int h) {
    if (h < H) {
      x[a][0] = __ldcs(reinterpret_cast<const uint2*>(row + at0));
      x[a][1] = __ldcs(reinterpret_cast<const uint2*>(row + at1));
    }
  };

  const int step = (int)((long long)gridDim.x * kWarps / split);
  int token = (int)(gw / split);
  const __nv_bfloat16* src = nullptr;
  int pos = 0;
#pragma unroll
  for (int a = 0; a < kAhead; ++a) x[a][0] = x[a][1] = make_uint2(0, 0);
  grid_dependents_launch();
  grid_dependency_wait();
  if (token < total) {
    src = token_rows(token);
    pos = p.positions[token];
#pragma unroll
    for (int a = 0; a < kAhead; ++a) load(a, src + a * per * D, first + a * per);
  }
  for (int i = threadIdx.x; i < 2 * D; i += kRopeThreads) {
    const void* w = i < D ? p.wq : p.wk;
    s_w[i / D][i % D] = p.w_fp32 ? static_cast<const float*>(w)[i % D]
                                 : __bfloat162float(static_cast<const __nv_bfloat16*>(w)[i % D]);
  }
  __syncthreads();

  const long long head_bytes = (long long)p.N * (D * 2);  // from head to head of an output
  while (token < total) {
    const int next = token < total - step ? token + step : total;
    const __nv_bfloat16* src_next = next < total ? token_rows(next) : nullptr;
    __syncwarp();
#pragma unroll
    for (int j = lane; j < D / 2; j += 32)
      if (j < half) rope_angle(pos, p.inv_freq[j], cosw + j, sinw + j);
    if (next < total) pos = p.positions[next];
    __syncwarp();
    const int b = token / p.N;
    const long long n = token - (long long)b * p.N;

    // (u, v) -> inv (u A + v M, u K + v E) for this lane's pairs, in its row's section
    // (queries, keys or values; rows of a warp may lie in two)
    uint64_t A[2], M[2], K[2], E[2];
    char* dst = nullptr;  // this lane's row of the output
    int sec_end = 0;      // first row behind the section
    int h = first;
    const __nv_bfloat16* ahead = src + (long long)kAhead * per * D;  // row to fetch next
    for (int base = 0; base < passes; base += kAhead) {
#pragma unroll
      for (int a = 0; a < kAhead; ++a) {
        uint2 r0 = x[a][0], r1 = x[a][1];
        if (base + kAhead < passes)
          load(a, ahead + a * per * D, h + kAhead * per);
        else if (src_next)
          load(a, src_next + a * per * D, first + a * per);
        if (h >= sec_end && h < H) {
          const int sec = h < p.Hq ? 0 : (h < n_qk ? 1 : 2);
          const int begin = sec == 0 ? 0 : (sec == 1 ? p.Hq : n_qk);
          const int heads = sec == 0 ? p.Hq : p.Hkv;
          sec_end = begin + heads;
          __nv_bfloat16* out = sec == 0 ? p.q : (sec == 1 ? p.k : p.v);
          dst = reinterpret_cast<char*>(out + (((long long)b * heads + (h - begin)) * p.N + n) * D);
          if (sec < 2) {
            const float4 w0 = *reinterpret_cast<const float4*>(&s_w[sec][at0]);
            const float4 w1 = *reinterpret_cast<const float4*>(&s_w[sec][at1]);
            float4 cc = make_float4(1.f, 1.f, 1.f, 1.f), ss = make_float4(0.f, 0.f, 0.f, 0.f);
            if (turned) {
              cc = *reinterpret_cast<const float4*>(cosw + 4 * c);
              ss = *reinterpret_cast<const float4*>(sinw + 4 * c);
            }
            const uint64_t C0 = f2_pack(cc.x, cc.y), C1 = f2_pack(cc.z, cc.w);
            const uint64_t S0 = f2_pack(ss.x, ss.y), S1 = f2_pack(ss.z, ss.w);
            const uint64_t N0 = f2_pack(-ss.x, -ss.y), N1 = f2_pack(-ss.z, -ss.w);
            uint64_t u0, u1, v0, v1;
            if (kInterleaved) {
              u0 = f2_pack(w0.x, w0.z), v0 = f2_pack(w0.y, w0.w);
              u1 = f2_pack(w1.x, w1.z), v1 = f2_pack(w1.y, w1.w);
            } else {
              u0 = f2_pack(w0.x, w0.y), u1 = f2_pack(w0.z, w0.w);
              v0 = f2_pack(w1.x, w1.y), v1 = f2_pack(w1.z, w1.w);
            }
            A[0] = f2_mul(u0, C0), A[1] = f2_mul(u1, C1);
            K[0] = f2_mul(u0, S0), K[1] = f2_mul(u1, S1);
            M[0] = f2_mul(v0, N0), M[1] = f2_mul(v1, N1);
            E[0] = f2_mul(v0, C0), E[1] = f2_mul(v1, C1);
          }
        }
        if (!__all_sync(0xffffffffu, h >= n_qk)) {
          uint64_t U[2], V[2];
          if (kInterleaved) {
            U[0] = f2_pack(__uint_as_float(r0.x << 16), __uint_as_float(r0.y << 16));
            U[1] = f2_pack(__uint_as_float(r1.x << 16), __uint_as_float(r1.y << 16));
            V[0] = f2_pack(__uint_as_float(r0.x & 0xffff0000u), __uint_as_float(r0.y & 0xffff0000u));
            V[1] = f2_pack(__uint_as_float(r1.x & 0xffff0000u), __uint_as_float(r1.y & 0xffff0000u));
          } else {
            U[0] = widen2(r0.x), U[1] = widen2(r0.y), V[0] = widen2(r1.x), V[1] = widen2(r1.y);
          }
          uint64_t sq = f2_mul(U[0], U[0]);
          sq = f2_fma(U[1], U[1], sq);
          sq = f2_fma(V[0], V[0], sq);
          sq = f2_fma(V[1], V[1], sq);
          float s0, s1;
          f2_unpack(sq, s0, s1);
          s0 += s1;
#pragma unroll
          for (int m = kLanes / 2; m > 0; m /= 2) s0 += __shfl_xor_sync(0xffffffffu, s0, m);
          const float inv = rsqrtf(s0 * (1.f / D) + p.eps);
          const uint64_t I = f2_pack(inv, inv);
          uint64_t Y[2], Z[2];
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const uint64_t u = f2_mul(U[k], I), v = f2_mul(V[k], I);
            Y[k] = f2_fma(v, M[k], f2_mul(u, A[k]));
            Z[k] = f2_fma(u, K[k], f2_mul(v, E[k]));
          }
          if (h < n_qk) {
            if (kInterleaved) {
              float u0, u1, v0, v1;
              f2_unpack(Y[0], u0, u1), f2_unpack(Z[0], v0, v1);
              r0 = make_uint2(pack2(u0, v0), pack2(u1, v1));
              f2_unpack(Y[1], u0, u1), f2_unpack(Z[1], v0, v1);
              r1 = make_uint2(pack2(u0, v0), pack2(u1, v1));
            } else {
              r0 = make_uint2(narrow2(Y[0]), narrow2(Y[1]));
              r1 = make_uint2(narrow2(Z[0]), narrow2(Z[1]));
            }
          }
        }
        if (h < H) {
          *reinterpret_cast<uint2*>(dst + at0 * 2) = r0;
          *reinterpret_cast<uint2*>(dst + at1 * 2) = r1;
          dst += per * head_bytes;
        }
        h += per;
      }
      ahead += kAhead * per * D;
    }
    token = next;
    src = src_next;
  }
}

}  // namespace osx
