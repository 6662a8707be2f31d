// decode_merge.cuh - joining the partial results of the warps and blocks that share one
// key/value head's queries.
//
// Each warp ends with, for its 8 NT query rows: a base m (log2 units), a denominator l
// and an unnormalised output row of D values, over the keys it has seen. They are joined
// by the log-sum-exp rule of attn_merge in two steps, always in the same order (no
// atomics, so results do not depend on timing): the block's warps through shared memory,
// then the cluster's blocks through distributed shared memory, each block finishing a
// slice of the rows' values. One launch, no workspace, nothing left over between calls.
#pragma once

#include <cuda_bf16.h>

#include <cstdint>

#include "serve_ptx.cuh"

namespace osx {

template <int D, int NT, int kWarps>
struct DecodeMerge {
  static constexpr int kRows = 8 * NT;
  // shared memory of the block: its own joined rows, statistics of warps, and weights
  static constexpr uint32_t kStatFloats = 2 * kWarps * kRows;           // m, l by warp
  static constexpr uint32_t kJoinFloats = kRows * D + 2 * kRows;        // o, m, l
  static constexpr uint32_t kWeightFloats = 16 * kRows + kRows;         // by rank; 1 / l
  static constexpr uint32_t kBytes = (kStatFloats + kJoinFloats + kWeightFloats) * 4;

  // warp_o(w): shared-memory rows [kRows][D] of warp w. rows: valid rows of the tile.
  // o_row0: first row's index in o ([..][D]) and lse.
  template <class WarpO>
  __device__ static void run(float* smem, WarpO warp_o, int splits, int rows, long long o_row0,
                             void* o, int o_bf16, float* lse) {
    float* sm = smem;                     // [kWarps][kRows]
    float* sl = sm + kWarps * kRows;
    float* jo = sl + kWarps * kRows;      // [kRows][D]
    float* jm = jo + kRows * D;
    float* jl = jm + kRows;
    float* wt = jl + kRows;               // [16][kRows]
    float* inv = wt + 16 * kRows;
    const int tid = threadIdx.x;
    __syncthreads();
    for (int x = tid; x < kRows * D; x += kWarps * 32) {
      const int r = x / D;
      float M = -INFINITY;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) M = fmaxf(M, sm[w * kRows + r]);
      float acc = 0.f, l = 0.f;
      if (M != -INFINITY) {
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
          const float a = ex2_approx(sm[w * kRows + r] - M);  // 0 for a warp without keys
          acc = fmaf(a, warp_o(w)[x], acc);
          l = fmaf(a, sl[w * kRows + r], l);
        }
      }
      jo[x] = acc;
      if (x % D == 0) {
        jm[r] = M;
        jl[r] = l;
      }
    }
    int rank = 0;
    if (splits > 1) {
      rank = (int)cluster_rank();
      cluster_barrier();
      if (tid < 32) {
        for (int r = tid; r < kRows; r += 32) {
          float m[16], l[16];
          float M = -INFINITY;
#pragma unroll
          for (int k = 0; k < 16; ++k) {
            m[k] = k < splits ? ld_cluster_f32(smem_u32(&jm[r]), k) : -INFINITY;
            l[k] = k < splits ? ld_cluster_f32(smem_u32(&jl[r]), k) : 0.f;
          }
#pragma unroll
          for (int k = 0; k < 16; ++k) M = fmaxf(M, m[k]);
          float L = 0.f;
#pragma unroll
          for (int k = 0; k < 16; ++k) {
            const float a = M == -INFINITY ? 0.f : ex2_approx(m[k] - M);
            wt[k * kRows + r] = a;
            L = fmaf(a, l[k], L);
          }
          inv[r] = L > 0.f ? 1.f / L : 0.f;
          if (rank == 0 && r < rows)
            lse[o_row0 + r] = L > 0.f ? (M + lg2_approx(L)) * 0.69314718055994530942f : -INFINITY;
        }
      }
      __syncthreads();
    } else {
      __syncthreads();
      if (tid < kRows) {
        const float L = jl[tid];
        inv[tid] = L > 0.f ? 1.f / L : 0.f;
        if (tid < rows)
          lse[o_row0 + tid] =
              L > 0.f ? (jm[tid] + lg2_approx(L)) * 0.69314718055994530942f : -INFINITY;
      }
      __syncthreads();
    }
    // this block's slice, two values a thread
    const int pairs = kRows * D / 2 / splits;
    for (int x = tid; x < pairs; x += kWarps * 32) {
      const int e = 2 * (rank * pairs + x), r = e / D;
      if (r >= rows) continue;
      float a = 0.f, c = 0.f;
      if (splits > 1) {
#pragma unroll 4
        for (int k = 0; k < splits; ++k) {
          const float w = wt[k * kRows + r];
          a = fmaf(w, ld_cluster_f32(smem_u32(&jo[e]), k), a);
          c = fmaf(w, ld_cluster_f32(smem_u32(&jo[e + 1]), k), c);
        }
      } else {
        a = jo[e];
        c = jo[e + 1];
      }
      a *= inv[r];
      c *= inv[r];
      const long long at = o_row0 * D + e;
      if (o_bf16)
        *reinterpret_cast<uint32_t*>(static_cast<__nv_bfloat16*>(o) + at) = pack_bf16x2(a, c);
      else
        *reinterpret_cast<float2*>(static_cast<float*>(o) + at) = make_float2(a, c);
    }
    if (splits > 1) cluster_barrier();  // no block leaves while another reads its rows
  }
};

}  // namespace osx
