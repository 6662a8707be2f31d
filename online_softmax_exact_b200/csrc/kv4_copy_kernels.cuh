// kv4_copy_kernels.cuh - tokens into the paged 4-bit cache, and back out as bf16.
//
// Both are memory passes. A warp takes a window of 16 tokens of one head, keys or values,
// and works in the cache's own word order (see kv4_layout.cuh): lane (g, t) converts the
// words that it will feed to, or has read from, the cache, so a whole block moves as
// 16-byte accesses of consecutive lanes and the bf16 side as runs of 64 (keys) or 128
// (values) bytes of a row. Windows are cut where the cache's blocks are, so in a prompt
// all but the first and last of a request's windows fill a block exactly; the others
// (and single tokens) store word by word.
// Measured (24.6k tokens of 8 heads, d = 128): append 46 us (131 MB, 2.8 TB/s: instructions
// issue in 63% of the cycles, and 32 warps an SM do not hide all of the loads' latency), read
// 35 us (165 MB, 4.7 TB/s: issue 66%, ALU pipe 64%), both in a stream, overlapping, 69 to 71
// us. Plain divisions and slots resolved value by value took half as long again, items found
// in 64-bit divisions 1 us.
#pragma once

#include <cuda_bf16.h>

#include <cstdint>

#include "serve_params.h"

#include "kv4_layout.cuh"
#include "qk_norm_rope_kernel.cuh"

namespace osx {

// Warps of a block, and blocks of the append kernel kept on an SM: 64 registers a thread. Both
// kernels on the tokens above, blocks of 8 / 4 / 2 warps: 70.7 / 68.8 / 73.4 us; 8 warps at
// 72 registers (3 blocks) 75.1 us, at 48 (5 blocks, spilling) 72.8 us.
constexpr int kKv4CopyWarps = 4;
constexpr int kKv4AppendBlocks = 8;

// Warp -> (request, window, head, keys or values); neighbouring warps take neighbouring
// heads of one window. False past the end.
__device__ __forceinline__ bool kv4_copy_item(const Kv4CopyParams& p, int& b, int& c, int& h,
                                              int& which) {
  uint32_t w = blockIdx.x * kKv4CopyWarps + threadIdx.x / 32;
  if (w >= p.items) return false;
  which = (int)(w & 1);
  w >>= 1;
  const uint32_t q = w / (uint32_t)p.Hkv;
  h = (int)(w - q * (uint32_t)p.Hkv);
  b = (int)(q / (uint32_t)p.windows);
  c = (int)(q - (uint32_t)b * (uint32_t)p.windows);
  return true;
}

template <int D>
__global__ void __launch_bounds__(kKv4CopyWarps * 32, kKv4AppendBlocks)
    kv4_append_kernel(const Kv4CopyParams p) {
  using L = Kv4<D>;
  int b, c, h, which;
  if (!kv4_copy_item(p, b, c, h, which)) return;
  const int lane = threadIdx.x % 32, g = lane >> 2, t = lane & 3;
  grid_dependents_launch();
  grid_dependency_wait();
  const int* slots = p.slots + (long long)b * p.N;
  const long long limit = (long long)p.n_pages * p.page_size;
  // the window's first token: aligned with the cache's blocks if slots run on from the first
  // (fewer tokens than a block has fill none, and need not wait for the first slot)
  const int s_first = p.N < 16 ? 0 : slots[0];
  const int i0 = c * 16 - (s_first > 0 ? s_first % 16 : 0);
  auto slot_of = [&](int row) {
    const int i = i0 + row;
    const int s = i >= 0 && i < p.N ? slots[i] : -1;
    return s < limit ? s : -1;
  };
  const int blocks = p.page_size / 16;
  auto block_of = [&](int slot) {
    const int page = slot / p.page_size, off = slot - page * p.page_size;
    return p.cache + (((long long)page * p.Hkv + h) * blocks + off / 16) * L::kWords;
  };
  const __nv_bfloat16* src =
      (which ? p.v : p.k) + (((long long)b * p.Hkv + h) * p.N + i0) * (long long)D;
  // the whole window in one block, row for row (lane l < 16 asks for row l)
  const int mine = slot_of(lane & 15);
  const int base = __shfl_sync(0xffffffffu, mine, 0);
  const bool whole = __all_sync(0xffffffffu, base >= 0 && base % 16 == 0 &&
                                                 mine == base + (lane & 15));
  if (!whole && __all_sync(0xffffffffu, mine < 0)) return;

  if (which == 0) {
    // keys: rows g and g + 8, words i: values 32 i + 8 t ..
    uint4 raw[2][L::kGroups];
    int slot[2];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      slot[r] = __shfl_sync(0xffffffffu, mine, 8 * r + g);
#pragma unroll
      for (int i = 0; i < L::kGroups; ++i)
        raw[r][i] = slot[r] < 0 ? make_uint4(0, 0, 0, 0)
                                : __ldcs(reinterpret_cast<const uint4*>(
                                      src + (8 * r + g) * D + 32 * i + 8 * t));
    }
    uint32_t word[2][L::kGroups] = {}, par[2][L::kGroups] = {};
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      if (!__any_sync(0xffffffffu, slot[r] >= 0)) continue;
#pragma unroll
      for (int i = 0; i < L::kGroups; ++i) {
        float lo, range;
        group_range<1>(raw[r][i], &lo, &range);
        word[r][i] = quant8(raw[r][i], lo, range, &par[r][i]);
      }
    }
    if (whole) {
      uint32_t* blk = block_of(base);
      if constexpr (D == 128) {
#pragma unroll
        for (int r = 0; r < 2; ++r)
          *reinterpret_cast<uint4*>(blk + (r * 32 + lane) * 4) =
              make_uint4(word[r][0], word[r][1], word[r][2], word[r][3]);
      } else {
        *reinterpret_cast<uint4*>(blk + lane * 4) =
            make_uint4(word[0][0], word[0][1], word[1][0], word[1][1]);
      }
      // a row's parameters are on all of its lanes
      if (t < 2) {
        uint32_t* row = blk + L::kKParams + (8 * t + g) * L::kGroups;
        if constexpr (D == 128)
          *reinterpret_cast<uint4*>(row) = make_uint4(
              t ? par[1][0] : par[0][0], t ? par[1][1] : par[0][1], t ? par[1][2] : par[0][2],
              t ? par[1][3] : par[0][3]);
        else
          *reinterpret_cast<uint2*>(row) =
              make_uint2(t ? par[1][0] : par[0][0], t ? par[1][1] : par[0][1]);
      }
    } else {
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        if (slot[r] < 0) continue;
        uint32_t* blk = block_of(slot[r]);
        const int row = slot[r] % 16;  // page_size is a multiple of 16
#pragma unroll
        for (int i = 0; i < L::kGroups; ++i) {
          blk[L::k_word(row, t, i)] = word[r][i];
          if (t == i) blk[L::kKParams + row * L::kGroups + i] = par[r][i];
        }
      }
    }
  } else {
    // values: rows 8 bb + 2 t + a (kk = 2 bb + a), chunk e = g of the 64-value half h2
    uint4 raw[4][D / 64];
    int slot[4];
#pragma unroll
    for (int kk = 0; kk < 4; ++kk) {
      const int row = 8 * (kk >> 1) + 2 * t + (kk & 1);
      slot[kk] = __shfl_sync(0xffffffffu, mine, row);
#pragma unroll
      for (int h2 = 0; h2 < D / 64; ++h2)
        raw[kk][h2] = slot[kk] < 0 ? make_uint4(0, 0, 0, 0)
                                   : __ldcs(reinterpret_cast<const uint4*>(src + row * D +
                                                                           64 * h2 + 8 * g));
    }
    uint32_t word[4][D / 64] = {}, par[4][D / 64] = {};
#pragma unroll
    for (int kk = 0; kk < 4; ++kk) {
      if (!__any_sync(0xffffffffu, slot[kk] >= 0)) continue;
#pragma unroll
      for (int h2 = 0; h2 < D / 64; ++h2) {
        float lo, range;
        group_range<4>(raw[kk][h2], &lo, &range);
        word[kk][h2] = transpose_nibbles<2>(quant8(raw[kk][h2], lo, range, &par[kk][h2]), g);
      }
    }
    // parameters: lanes g = 0 and 4 of a group's four
    if (whole) {
      uint32_t* blk = block_of(base);
#pragma unroll
      for (int h2 = 0; h2 < D / 64; ++h2) {
        *reinterpret_cast<uint4*>(blk + L::kVCodes + (h2 * 32 + lane) * 4) =
            make_uint4(word[0][h2], word[1][h2], word[2][h2], word[3][h2]);
        if ((g & 3) == 0)
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            blk[L::kVParams + (8 * (kk >> 1) + 2 * t + (kk & 1)) * L::kGroups + 2 * h2 + (g >> 2)] =
                par[kk][h2];
      }
    } else {
#pragma unroll
      for (int kk = 0; kk < 4; ++kk) {
        if (slot[kk] < 0) continue;
        uint32_t* blk = block_of(slot[kk]);
        const int row = slot[kk] % 16;
#pragma unroll
        for (int h2 = 0; h2 < D / 64; ++h2) {
          blk[L::v_word(row, h2, g)] = word[kk][h2];
          if ((g & 3) == 0) blk[L::kVParams + row * L::kGroups + 2 * h2 + (g >> 2)] = par[kk][h2];
        }
      }
    }
  }
}

// eight codes of a word as values, packed to bf16
__device__ __forceinline__ uint4 dequant8(uint32_t w, uint32_t par) {
  const float s = param_scale(par), z = param_zero(par);
  float y[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float c = __uint_as_float(((w >> (4 * i)) & 15u) | 0x4B000000u) - 8388608.0f;
    y[i] = fmaf(c, s, z);  // c s is exact (4 by 8 bits): one rounding
  }
  return make_uint4(pack2(y[0], y[1]), pack2(y[2], y[3]), pack2(y[4], y[5]), pack2(y[6], y[7]));
}

template <int D>
__global__ void __launch_bounds__(kKv4CopyWarps * 32) kv4_read_kernel(const Kv4CopyParams p) {
  using L = Kv4<D>;
  int b, c, h, which;
  if (!kv4_copy_item(p, b, c, h, which)) return;
  const int lane = threadIdx.x % 32, g = lane >> 2, t = lane & 3;
  grid_dependents_launch();
  grid_dependency_wait();
  const int start = p.start[b], len = p.lens[b];
  const int blocks = p.page_size / 16;
  const long long pb = (long long)(start > 0 ? start : 0) / 16 + c;  // block of the request
  const long long i0 = pb * 16 - start;                              // its first token's output row
  const uint32_t* blk = nullptr;
  if (start >= 0 && pb * 16 < len && pb / blocks < p.width) {
    const int page = p.table[(long long)b * p.width + pb / blocks];
    if (page >= 0 && page < p.n_pages)
      blk = p.cache + (((long long)page * p.Hkv + h) * blocks + pb % blocks) * L::kWords;
  }
  __nv_bfloat16* dst = (which ? p.v_out : p.k_out) + ((long long)b * p.Hkv + h) * p.N * (long long)D;
  auto put = [&](int row, int at, uint32_t w, uint32_t par) {
    const long long i = (start < 0 ? (long long)c * 16 : i0) + row;
    if (i < 0 || i >= p.N) return;
    const uint4 y = blk && pb * 16 + row < len ? dequant8(w, par) : make_uint4(0, 0, 0, 0);
    *reinterpret_cast<uint4*>(dst + i * D + at) = y;
  };
  if (which == 0) {
    uint32_t word[2][L::kGroups] = {}, par[2][L::kGroups] = {};
    if (blk) {
      if constexpr (D == 128) {
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const uint4 w = *reinterpret_cast<const uint4*>(blk + (r * 32 + lane) * 4);
          const uint4 q = *reinterpret_cast<const uint4*>(blk + L::kKParams + (8 * r + g) * 4);
          word[r][0] = w.x, word[r][1] = w.y, word[r][2] = w.z, word[r][3] = w.w;
          par[r][0] = q.x, par[r][1] = q.y, par[r][2] = q.z, par[r][3] = q.w;
        }
      } else {
        const uint4 w = *reinterpret_cast<const uint4*>(blk + lane * 4);
        word[0][0] = w.x, word[0][1] = w.y, word[1][0] = w.z, word[1][1] = w.w;
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const uint2 q = *reinterpret_cast<const uint2*>(blk + L::kKParams + (8 * r + g) * 2);
          par[r][0] = q.x, par[r][1] = q.y;
        }
      }
    }
#pragma unroll
    for (int r = 0; r < 2; ++r)
#pragma unroll
      for (int i = 0; i < L::kGroups; ++i) put(8 * r + g, 32 * i + 8 * t, word[r][i], par[r][i]);
  } else {
#pragma unroll
    for (int h2 = 0; h2 < D / 64; ++h2) {
      uint32_t word[4] = {0, 0, 0, 0};
      if (blk) {
        const uint4 w =
            *reinterpret_cast<const uint4*>(blk + L::kVCodes + (h2 * 32 + lane) * 4);
        word[0] = w.x, word[1] = w.y, word[2] = w.z, word[3] = w.w;
      }
#pragma unroll
      for (int kk = 0; kk < 4; ++kk) {
        const int row = 8 * (kk >> 1) + 2 * t + (kk & 1);
        const uint32_t w = transpose_nibbles<2>(word[kk], g);
        const uint32_t par =
            blk ? blk[L::kVParams + row * L::kGroups + 2 * h2 + (g >> 2)] : 0u;
        put(row, 64 * h2 + 8 * g, w, par);
      }
    }
  }
}

}  // namespace osx
