// kv4_layout.cuh - the paged 4-bit cache of keys and values: layout and conversions.
//
// A token's keys (and its values) of one head are cut into groups of 32 values. A group
// is stored as 32 codes of 4 bits, a scale and a zero point (bf16 each):
//   zero = min, scale = bf16((max - min) / 15), code = rint((x - zero) / scale) in 0..15,
//   value = code * scale + zero,
// 5 bits a value in all. The inputs are bf16, so the zero point is exact; the scale is
// rounded to the nearest bf16 (a relative change of the step by up to 2^-8, and the codes are
// taken against the rounded scale, so no value moves by more than half a step plus that).
// Differences are taken in fp32.
//
// Pages hold page_size tokens (a multiple of 16) of every key/value head:
//   cache[page][kv head][block], block = 16 tokens = 20 d bytes (2560 at d = 128):
//     words [0, 2d)       codes of the keys
//     words [2d, 4d)      codes of the values
//     words [4d, 4.5d)    key parameters  [token][group]: scale in the low half, zero high
//     words [4.5d, 5d)    value parameters
// A word (32 bits) holds eight codes, the first in its low bits. The codes of a block are
// in the order in which the lanes of a warp feed them to mma.m16n8k16 as its A operand
// (lane = 4 g + t), so that a lane's words are 16 contiguous bytes:
//   keys    word (r, g, t, i) (at d = 64: (g, t, r, i)): token 8r + g,
//           values 32 i + 8 t + e, e = 0..7
//   values  word (h, g, t, b, a): token 8b + 2t + a, values 64 h + 8 e + g, e = 0..7
// A block is contiguous, so one bulk copy brings 16 tokens of a head, keys, values and
// parameters, into shared memory.
#pragma once

#include <cuda_bf16.h>

#include <cstdint>

#include "serve_ptx.cuh"

namespace osx {

template <int D>
struct Kv4 {
  static constexpr int kGroups = D / 32;            // groups of a token's row
  static constexpr int kWords = 5 * D;              // 32-bit words of a block
  static constexpr int kBytes = 20 * D;
  static constexpr int kVCodes = 2 * D;             // word offsets in a block
  static constexpr int kKParams = 4 * D;
  static constexpr int kVParams = 4 * D + D / 2;

  __device__ static int k_word(int row, int t, int i) {
    const int r = row >> 3, g = row & 7;
    return D == 128 ? (r * 32 + g * 4 + t) * 4 + i : ((g * 4 + t) * 2 + r) * 2 + i;
  }
  __device__ static int v_word(int row, int h, int g) {
    return kVCodes + (h * 32 + g * 4 + ((row & 7) >> 1)) * 4 + (row >> 3) * 2 + (row & 1);
  }
};

// 8x8 transposition of nibbles across 8 lanes: on entry lane e (bits kShift.. of the lane
// number) holds nibbles j; on exit lane j holds nibbles e. Three exchange steps.
template <int kShift>
__device__ __forceinline__ uint32_t transpose_nibbles(uint32_t w, int e) {
#pragma unroll
  for (int k = 1; k < 8; k *= 2) {
    const uint32_t m = k == 1 ? 0x0f0f0f0fu : (k == 2 ? 0x00ff00ffu : 0x0000ffffu);
    const uint32_t p = __shfl_xor_sync(0xffffffffu, w, k << kShift);
    w = (e & k) ? ((w & ~m) | ((p >> (4 * k)) & m)) : ((w & m) | ((p & m) << (4 * k)));
  }
  return w;
}

// Division by multiplication and fma: with r = RN(1/b), q = RN(a r) and e = a - q b (exact
// by fma), RN(q + e r) is RN(a / b) away from under- and overflow (Markstein's theorem, for
// b whose significand is not all ones; here 15, and scales of 8 significant bits, for all of
// which one Newton step from an approximation within 2 units in the last place gives RN(1/b)).
__device__ __forceinline__ float divide_fma(float a, float b, float r) {
  const float q = a * r;
  return fmaf(fmaf(-q, b, a), r, q);
}

// A group's scale and the codes of eight of its values, in plain divisions: for ranges
// outside 2^-90 .. 2^90, where the products above could leave the normal numbers.
__device__ __noinline__ uint32_t quant8_wide(uint4 raw, float zero, float range, float* scale_out) {
  const float scale = __bfloat162float(__float2bfloat16_rn(__fdiv_rn(range, 15.f)));
  *scale_out = scale;
  const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
  uint32_t codes = 0;
  if (!(scale > 0.f)) return codes;
  for (int i = 0; i < 8; ++i) {
    const float f = __uint_as_float((i & 1) ? w[i / 2] & 0xffff0000u : w[i / 2] << 16);
    const float q = fminf(fmaxf(rintf(__fdiv_rn(f - zero, scale)), 0.f), 15.f);
    codes |= (uint32_t)q << (4 * i);
  }
  return codes;
}

// The eight codes of a lane's values (bf16, raw) as one word, against the zero point and the
// range (maximum - minimum) of their group, and the group's parameter word. A quotient is
// the correctly rounded one, so a tie is a tie of the true quotient and goes to the even
// code: adding 1.5 * 2^23 rounds it to the integer in the low bits. The sum of the shifted
// words carries eight copies of that constant's own bits, subtracted at the end (modulo
// 2^32). The quotient stays below 15.5 (the scale is at most 2^-8 below range / 15).
__device__ __forceinline__ uint32_t quant8(const uint4& raw, float zero, float range,
                                           uint32_t* par) {
  float scale;
  uint32_t codes;
  if (range >= 0x1p-90f && range <= 0x1p+90f) {
    scale = __bfloat162float(__float2bfloat16_rn(divide_fma(range, 15.f, 1.f / 15.f)));
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(scale));
    r = fmaf(fmaf(-scale, r, 1.f), r, r);  // one Newton step
    const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
    codes = 0;
    // as divide_fma, two values at a time in packed fp32
    const uint64_t Z = f2_pack(zero, zero), R = f2_pack(r, r), NS = f2_pack(-scale, -scale);
    const uint64_t ROUND = f2_pack(12582912.0f, 12582912.0f);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint64_t Y =
          f2_sub(f2_pack(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u)), Z);
      const uint64_t Q = f2_mul(Y, R);
      float a, b;
      f2_unpack(f2_add(f2_fma(f2_fma(Q, NS, Y), R, Q), ROUND), a, b);
      codes += (__float_as_uint(a) << (8 * i)) + (__float_as_uint(b) << (8 * i + 4));
    }
    constexpr uint32_t kBits = 0x4B400000u;
    codes -= kBits + (kBits << 4) + (kBits << 8);  // higher shifts leave the word
  } else {
    codes = quant8_wide(raw, zero, range, &scale);
  }
  *par = (__float_as_uint(scale) >> 16) | (__float_as_uint(zero) & 0xffff0000u);
  return codes;
}

// Minimum and maximum of eight bf16 values (raw) and of the lanes at kStep and 2 kStep from
// this one: a group of 32.
template <int kStep>
__device__ __forceinline__ void group_range(const uint4& raw, float* lo, float* range) {
  uint32_t mx, mn, a, b;
  asm("max.bf16x2 %0, %1, %2;" : "=r"(a) : "r"(raw.x), "r"(raw.y));
  asm("max.bf16x2 %0, %1, %2;" : "=r"(b) : "r"(raw.z), "r"(raw.w));
  asm("max.bf16x2 %0, %1, %2;" : "=r"(mx) : "r"(a), "r"(b));
  asm("min.bf16x2 %0, %1, %2;" : "=r"(a) : "r"(raw.x), "r"(raw.y));
  asm("min.bf16x2 %0, %1, %2;" : "=r"(b) : "r"(raw.z), "r"(raw.w));
  asm("min.bf16x2 %0, %1, %2;" : "=r"(mn) : "r"(a), "r"(b));
  mn ^= 0x80008000u;  // as maxima of the negated values
  // low halves in one word, high halves in another: their maximum is (maximum, -minimum)
  a = __byte_perm(mx, mn, 0x5410);
  b = __byte_perm(mx, mn, 0x7632);
  asm("max.bf16x2 %0, %0, %1;" : "+r"(a) : "r"(b));
#pragma unroll
  for (int s = kStep; s <= 2 * kStep; s *= 2) {
    b = __shfl_xor_sync(0xffffffffu, a, s);
    asm("max.bf16x2 %0, %0, %1;" : "+r"(a) : "r"(b));
  }
  const float hi = __uint_as_float(a << 16);
  // a minimum of -0 counts as +0: which of the two a minimum of both is, is not defined
  *lo = 0.f - __uint_as_float(a & 0xffff0000u);
  *range = hi - *lo;
}

// scale (low half) and zero point (high half) of a parameter word
__device__ __forceinline__ float param_scale(uint32_t p) { return __uint_as_float(p << 16); }
__device__ __forceinline__ float param_zero(uint32_t p) {
  return __uint_as_float(p & 0xffff0000u);
}

}  // namespace osx
