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
// and attention takes head-major rows, so this pass is also the transposition). One block
// per token: its angles are the same for every head, so they are computed once per token
// and kept in registers, as are the norm weights. A row is held by d/8 lanes with 16
// bytes each, so rows move as whole 128-byte lines; a rotation partner r/2 values away
// is r/16 lanes away (one shuffle per value).
//
// Angles: position * inv_freq in 64 bits, reduced to [-pi, pi] in 64 bits, and only then
// sine and cosine in fp32. An fp32 product would be off by 2^-24 of an angle of up to
// 10^5 radians, several times the bf16 spacing of the result.
#pragma once

#include <cuda_bf16.h>

#include <cstdint>

#include "serve_params.h"

namespace osx {

constexpr int kRopeThreads = 256;

__device__ __forceinline__ void unpack8(const uint4& u, float (&x)[8]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}

__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  uint32_t d;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}

__device__ __forceinline__ void load_weights8(const void* w, int w_fp32, int at, float (&x)[8]) {
  if (w_fp32) {
    const float* f = static_cast<const float*>(w) + at;
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = f[i];
  } else {
    const __nv_bfloat16* h = static_cast<const __nv_bfloat16*>(w) + at;
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = __bfloat162float(h[i]);
  }
}

template <int D, bool kInterleaved>
__global__ void __launch_bounds__(kRopeThreads) qk_norm_rope_kernel(const RopeParams p) {
  constexpr int kLanes = D / 8;                    // lanes per row
  constexpr int kRows = kRopeThreads / kLanes;     // rows a block moves at a time
  constexpr int kAhead = 3;                        // of a thread's rows, loads in flight
  __shared__ float s_cos[D / 2], s_sin[D / 2];
  const long long token = blockIdx.x;
  const int b = (int)(token / p.N), n = (int)(token - (long long)b * p.N);
  const int c = threadIdx.x % kLanes, row0 = threadIdx.x / kLanes;
  const int H = p.Hq + 2 * p.Hkv;
  const __nv_bfloat16* src = p.qkv + b * p.stride_b + n * p.stride_n + c * 8;

  // the first rows' loads fly while the angles are computed
  uint4 x[kAhead];
#pragma unroll
  for (int a = 0; a < kAhead; ++a) {
    const int h = row0 + a * kRows;
    if (h < H) x[a] = __ldcs(reinterpret_cast<const uint4*>(src + (long long)h * D));
  }
  float wq[8], wk[8];
  load_weights8(p.wq, p.w_fp32, c * 8, wq);
  load_weights8(p.wk, p.w_fp32, c * 8, wk);
  if (threadIdx.x < p.n_freq) {
    const double a = (double)p.positions[token] * (double)p.inv_freq[threadIdx.x];
    const double turns = rint(a * 0.15915494309189535);           // a / (2 pi)
    // 2 pi as a sum of two doubles; the first product is exact up to one rounding by fma
    const float r = (float)fma(-turns, 2.4492935982947064e-16, fma(-turns, 6.283185307179586, a));
    sincosf(r, &s_sin[threadIdx.x], &s_cos[threadIdx.x]);
  }
  __syncthreads();

  // this lane's angles: values 8c .. 8c + 7 of a row (for pairs of halves, the sine of a
  // value in the first half carries the minus sign)
  const int half = p.n_freq;
  const bool turned = c * 8 < 2 * half;
  float cs[8], sn[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int e = c * 8 + i;
    const int j = kInterleaved ? e / 2 : (e < half ? e : e - half);
    cs[i] = turned ? s_cos[j] : 1.f;
    sn[i] = turned ? s_sin[j] : 0.f;
    if (kInterleaved ? (i & 1) == 0 : e < half) sn[i] = -sn[i];
  }
  // lane that holds the rotation partner of this lane's values (halves)
  const int shift = half / 8;
  const int lane = threadIdx.x % 32;
  const int partner = !turned ? lane : (c < shift ? lane + shift : lane - shift);

  for (int base = 0; base < H; base += kAhead * kRows) {
#pragma unroll
    for (int a = 0; a < kAhead; ++a) {
      const int h = base + row0 + a * kRows;
      const uint4 raw = x[a];
      const int hn = h + kAhead * kRows;
      if (hn < H) x[a] = __ldcs(reinterpret_cast<const uint4*>(src + (long long)hn * D));
      // rows of one warp: a shuffle below needs every lane, so none leaves early
      const bool is_q = h < p.Hq, is_v = h >= p.Hq + p.Hkv;
      float f[8];
      unpack8(h < H ? raw : make_uint4(0, 0, 0, 0), f);
      float ss = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) ss = fmaf(f[i], f[i], ss);
#pragma unroll
      for (int s = kLanes / 2; s > 0; s /= 2) ss += __shfl_xor_sync(0xffffffffu, ss, s);
      const float inv = rsqrtf(ss * (1.f / D) + p.eps);
      float y[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) y[i] = f[i] * inv * (is_q ? wq[i] : wk[i]);
      float z[8];
      if (kInterleaved) {
#pragma unroll
        for (int i = 0; i < 8; ++i) z[i] = fmaf(y[i ^ 1], sn[i], y[i] * cs[i]);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float other = __shfl_sync(0xffffffffu, y[i], partner);
          z[i] = fmaf(other, sn[i], y[i] * cs[i]);
        }
      }
      if (h >= H) continue;
      uint4 out = make_uint4(pack2(z[0], z[1]), pack2(z[2], z[3]), pack2(z[4], z[5]),
                             pack2(z[6], z[7]));
      __nv_bfloat16* dst;
      if (is_q) {
        dst = p.q + (((long long)b * p.Hq + h) * p.N + n) * D;
      } else if (!is_v) {
        dst = p.k + (((long long)b * p.Hkv + (h - p.Hq)) * p.N + n) * D;
      } else {
        dst = p.v + (((long long)b * p.Hkv + (h - p.Hq - p.Hkv)) * p.N + n) * D;
        out = raw;
      }
      *reinterpret_cast<uint4*>(dst + c * 8) = out;
    }
  }
}

}  // namespace osx
