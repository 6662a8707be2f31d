// decode_common.cuh - how the decode kernels share their work, and the join of its parts.
//
// A unit is the query rows (a tile of kRows) of one request and key/value head; its keys
// are cut into stages. The stages of all units, one after another, are cut into `runs`
// runs of equal length (to one stage), one per warp: run w is [total w / runs,
// total (w + 1) / runs). A warp that begins and ends a unit within its run finishes it;
// every other part of a unit leaves a partial (base m in log2 units, denominator l,
// unnormalised rows) in slot w + unit of the workspace: both only grow along the stages,
// so no two parts share a slot. The join combines a unit's partials by the log-sum-exp
// rule of attn_merge, in an order that does not depend on timing.
#pragma once

#include <cuda_bf16.h>

#include <cstdint>

#include "serve_params.h"
#include "serve_ptx.cuh"

namespace osx {

// a / b of non-negative numbers, in 32 bits where they fit (a 64-bit division costs about
// five times as much, and several of them lie in the path of a short call)
__device__ __forceinline__ long long divide(long long a, long long b) {
  if (((a | b) >> 32) == 0) return (uint32_t)a / (uint32_t)b;
  return a / b;
}

// Runs that `total` stages are cut into on a grid of `warps` warps: none is empty.
__device__ __forceinline__ long long decode_runs(long long total, int warps) {
  return total < warps ? total : warps;
}

// Joins the partials of one row of one unit, kHalf of its values: kLanes lanes per partial,
// the partials dealt to the block's groups of lanes, in two steps whose order does not
// depend on timing. kThreads goes by the number of partials (launch_join).
template <int D, int kRows, int kThreads>
__global__ void __launch_bounds__(kThreads) decode_join_kernel(
    const __grid_constant__ JoinParams p) {
  constexpr int kHalf = 64, kParts = D / kHalf;  // values of a block, blocks of a row
  constexpr int kLanes = kHalf / 4, kGroups = kThreads / kLanes;
  __shared__ float4 part[kGroups][kLanes];
  __shared__ float2 stat[kGroups];
  const int half = blockIdx.x % kParts;
  const int unit = blockIdx.x / kParts / kRows, r = blockIdx.x / kParts % kRows;
  const int per_b = p.Hkv * p.row_tiles;
  const int b = unit / per_b, in_b = unit - b * per_b;
  const int h = in_b / p.row_tiles, rt = in_b - h * p.row_tiles;
  if (rt * kRows + r >= p.rows) return;
  const long long row = ((long long)b * p.Hkv + h) * p.rows + rt * kRows + r;
  grid_dependents_launch();
  const int lane = threadIdx.x % kLanes, grp = threadIdx.x / kLanes;
  auto store = [&](float4 y) {
    const long long at = row * (D / 4) + half * kLanes + lane;
    if (p.o_bf16)
      reinterpret_cast<uint2*>(p.o)[at] = make_uint2(pack_bf16x2(y.x, y.y), pack_bf16x2(y.z, y.w));
    else
      reinterpret_cast<float4*>(p.o)[at] = y;
  };
  grid_dependency_wait();  // the attention launch's writes are visible from here on
  // stages before request b's units, of all units, and of each of b's
  long long pre, total, n;
  if (p.prefix) {
    pre = p.prefix[b];
    total = p.prefix[p.B];
    n = divide(p.prefix[b + 1] - pre, per_b);
  } else {
    n = p.n_stages;
    pre = (long long)b * per_b * n;
    total = (long long)p.B * per_b * n;
  }
  if (n == 0) {  // no key is seen
    if (grp == 0) store(make_float4(0.f, 0.f, 0.f, 0.f));
    if (half == 0 && threadIdx.x == 0) p.lse[row] = -INFINITY;
    return;
  }
  // runs of the unit's first and last stage: run w has stages [total w / runs, ..)
  const long long first = pre + in_b * n, last = first + n - 1;
  const long long runs = decode_runs(total, p.n_warps);
  const int w0 = (int)divide((first + 1) * runs - 1, total);
  const int w1 = (int)divide((last + 1) * runs - 1, total);
  if (w0 == w1) return;  // finished by that warp
  const int parts = w1 - w0 + 1;
  const float* ml = p.ml + ((long long)w0 + unit) * (kRows * 2) + 2 * r;
  const float4* po = reinterpret_cast<const float4*>(p.parts + ((long long)w0 + unit) * (kRows * D) +
                                                     r * D + half * kHalf) + lane;
  // this group's partials against their own running maximum
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  float M = -INFINITY, l = 0.f;
  for (int k0 = grp; k0 < parts; k0 += 5 * kGroups) {
    float2 st[5];
    float4 x[5];
#pragma unroll
    for (int j = 0; j < 5; ++j) {
      const long long k = k0 + j * kGroups;
      st[j] = make_float2(-INFINITY, 0.f);
      x[j] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (k < parts) {
        st[j] = *reinterpret_cast<const float2*>(ml + k * (kRows * 2));
        x[j] = po[k * (kRows * (D / 4))];
      }
    }
    float top = M;
#pragma unroll
    for (int j = 0; j < 5; ++j) top = fmaxf(top, st[j].x);
    if (top == -INFINITY) continue;  // no keys so far
    const float keep = ex2_approx(M - top);
    M = top;
    l *= keep;
    acc.x *= keep, acc.y *= keep, acc.z *= keep, acc.w *= keep;
#pragma unroll
    for (int j = 0; j < 5; ++j) {
      const float a = ex2_approx(st[j].x - top);  // 0 for a part without keys
      l = fmaf(a, st[j].y, l);
      acc.x = fmaf(a, x[j].x, acc.x);
      acc.y = fmaf(a, x[j].y, acc.y);
      acc.z = fmaf(a, x[j].z, acc.z);
      acc.w = fmaf(a, x[j].w, acc.w);
    }
  }
  part[grp][lane] = acc;
  if (lane == 0) stat[grp] = make_float2(M, l);
  __syncthreads();
  if (grp != 0) return;
  M = -INFINITY;
#pragma unroll
  for (int k = 0; k < kGroups; ++k) M = fmaxf(M, stat[k].x);
  const float base = M == -INFINITY ? 0.f : M;
  float sum = 0.f;
  acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
  for (int k = 0; k < kGroups; ++k) {
    const float a = ex2_approx(stat[k].x - base);
    const float4 x = part[k][lane];
    sum = fmaf(a, stat[k].y, sum);
    acc.x = fmaf(a, x.x, acc.x);
    acc.y = fmaf(a, x.y, acc.y);
    acc.z = fmaf(a, x.z, acc.z);
    acc.w = fmaf(a, x.w, acc.w);
  }
  const float inv = sum > 0.f ? 1.f / sum : 0.f;
  store(make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv));
  if (half == 0 && lane == 0)
    p.lse[row] = sum > 0.f ? (M + lg2_approx(sum)) * 0.69314718055994530942f : -INFINITY;
}

}  // namespace osx
