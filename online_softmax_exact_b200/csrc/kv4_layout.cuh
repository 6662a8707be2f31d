// kv4_layout.cuh - the paged 4-bit cache of keys and values: layout and conversions.
//
// A token's keys (and its values) of one head are cut into groups of 32 values. A group
// is stored as 32 codes of 4 bits, a scale and a zero point (bf16 each):
//   zero = min, scale = bf16((max - min) / 15), code = rint((x - zero) / scale) in 0..15,
//   value = code * scale + zero,
// 5 bits a value in all. The inputs are bf16, so the zero point is exact; the scale is
// rounded to the nearest bf16 (a 2^-9 relative change of the step, and the codes are
// taken against the rounded scale, so no value moves by more than half a step plus that).
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

#include <cstdint>

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

// The eight codes of f against (zero, scale) as one word. The quotient is the correctly
// rounded one: with r = RN(1/s), q = RN(y r) and e = y - q s (exact by fma), RN(q + e r)
// is RN(y / s) unless the significand of s is all ones (Markstein's theorem on division
// by multiplication and fma; s has 8 significant bits here), away from under- and
// overflow; scales outside that range take a plain division. So a tie is a tie of the
// true quotient and goes to the even code. Adding 1.5 * 2^23 rounds to the integer in
// the low bits; the sum of the shifted words carries eight copies of the constant's own
// bits, which are subtracted at the end (modulo 2^32).
__device__ __forceinline__ uint32_t quant8(const float (&f)[8], float zero, float scale) {
  if (!(scale > 0.f)) return 0u;
  uint32_t w = 0;
  if (scale >= 0x1p-100f && scale <= 0x1p+100f) {
    const float r = __frcp_rn(scale);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float y = f[i] - zero;
      const float q0 = y * r;
      const float q = fmaf(fmaf(-q0, scale, y), r, q0);
      w += __float_as_uint(q + 12582912.0f) << (4 * i);
    }
    constexpr uint32_t kBits = 0x4B400000u;
    return w - (kBits + (kBits << 4) + (kBits << 8));  // higher shifts leave the word
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float q = fminf(fmaxf(rintf(__fdiv_rn(f[i] - zero, scale)), 0.f), 15.f);
    w |= (uint32_t)q << (4 * i);
  }
  return w;
}

// scale (low half) and zero point (high half) of a parameter word
__device__ __forceinline__ float param_scale(uint32_t p) { return __uint_as_float(p << 16); }
__device__ __forceinline__ float param_zero(uint32_t p) {
  return __uint_as_float(p & 0xffff0000u);
}

}  // namespace osx
