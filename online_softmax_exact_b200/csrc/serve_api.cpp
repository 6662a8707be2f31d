// serve_api.cpp - the C ABI of the serving operators: argument checks and dispatch. Every
// check runs before any CUDA call, so invalid arguments are reported without touching a
// device.
#include <cmath>
#include <cstdint>

#include "../../include/attn.h"
#include "api_checks.h"
#include "attn_internal.h"
#include "serve_params.h"

namespace {

using osx::aligned;
using osx::overlap;
using osx::Span;
using osx::span;

constexpr int64_t kMaxRows = (int64_t(1) << 31) - 512;
constexpr int64_t kMaxOffset = int64_t(1) << 60;

// Every output apart from every input and from every other output.
bool apart(const Span* out, int n_out, const Span* in, int n_in) {
  for (int i = 0; i < n_out; ++i) {
    for (int j = 0; j < i; ++j)
      if (overlap(out[i], out[j])) return false;
    for (int j = 0; j < n_in; ++j)
      if (overlap(out[i], in[j])) return false;
  }
  return true;
}

// Heads, head size and page geometry shared by the cache calls.
attn_status_t check_cache(const void* cache, int Hkv, int d, int page_size, int n_pages) {
  if (!cache || !aligned(cache, 16)) return ATTN_ERR_INVALID_ARG;
  if (Hkv < 1 || page_size < 16 || page_size % 16 != 0 || n_pages < 1) return ATTN_ERR_INVALID_ARG;
  if (d != 64 && d != 128) return ATTN_ERR_UNSUPPORTED;
  if ((int64_t)n_pages * page_size > INT32_MAX) return ATTN_ERR_UNSUPPORTED;  // 32-bit slots
  return ATTN_OK;
}

uint64_t cache_bytes(int Hkv, int d, int page_size, int n_pages) {
  return (uint64_t)n_pages * Hkv * (page_size / 16) * 20 * d;
}

bool too_many(int64_t a, int64_t b, int64_t limit) { return a > limit / b; }

// Windows of 16 tokens that N tokens can touch, wherever they start, and the copy kernels'
// items, two per window and head; 0 where they leave 32 bits (over 500 GB of rows).
int copy_windows(int N) { return (int)(((int64_t)N + 30) / 16); }

unsigned copy_items(int B, int N, int Hkv) {
  const int64_t per = 2 * (int64_t)copy_windows(N) * Hkv;
  return too_many(per, B, 0xffffff00LL) ? 0u : (unsigned)(per * B);
}

}  // namespace

extern "C" {

attn_status_t attn_kv_plan(const int32_t* lens, const int32_t* new_lens, int32_t* table,
                           const int32_t* free_pages, const int32_t* free_head, int32_t* slots,
                           int32_t* positions, int32_t* lens_out, int32_t* head_out,
                           int32_t* served, int B, int n_new, int width, int page_size,
                           int n_free, void* stream) {
  if (!lens || !new_lens || !table || !free_pages || !free_head || !slots || !positions ||
      !lens_out || !head_out || !served)
    return ATTN_ERR_INVALID_ARG;
  if (B < 1 || n_new < 1 || width < 1 || page_size < 1 || n_free < 0) return ATTN_ERR_INVALID_ARG;
  const void* all[10] = {lens,  new_lens,  table,    free_pages, free_head,
                         slots, positions, lens_out, head_out,   served};
  for (const void* p : all)
    if (!aligned(p, 4)) return ATTN_ERR_INVALID_ARG;
  if (too_many(B, n_new, 1 << 30) || too_many(width, page_size, INT32_MAX))
    return ATTN_ERR_UNSUPPORTED;
  const uint64_t b4 = (uint64_t)B * 4;
  const Span in[4] = {span(lens, b4), span(new_lens, b4), span(free_pages, (uint64_t)n_free * 4),
                      span(free_head, 4)};
  const Span out[6] = {span(table, b4 * width), span(slots, b4 * n_new),
                       span(positions, b4 * n_new), span(lens_out, b4), span(head_out, 4),
                       span(served, b4)};
  if (!apart(out, 6, in, 4)) return ATTN_ERR_INVALID_ARG;
  const int inj = osx::take_injected();
  if (inj != ATTN_OK) return static_cast<attn_status_t>(inj);
  const osx::PlanParams p{lens,     new_lens, table, free_pages, free_head, slots,
                          positions, lens_out, head_out, served, B, n_new, width, page_size, n_free};
  return static_cast<attn_status_t>(osx::launch_kv_plan(p, static_cast<cudaStream_t>(stream)));
}

attn_status_t attn_qk_norm_rope(const void* qkv, int64_t stride_b, int64_t stride_n,
                                const void* wq, const void* wk, int w_fp32,
                                const float* inv_freq, int n_freq, const int32_t* positions,
                                void* q, void* k, void* v, int B, int N, int Hq, int Hkv, int d,
                                float eps, int interleaved, void* stream) {
  if (!qkv || !wq || !wk || !inv_freq || !positions || !q || !k || !v) return ATTN_ERR_INVALID_ARG;
  if (B < 1 || N < 1 || Hq < 1 || Hkv < 1) return ATTN_ERR_INVALID_ARG;
  if ((w_fp32 != 0 && w_fp32 != 1) || (interleaved != 0 && interleaved != 1))
    return ATTN_ERR_INVALID_ARG;
  if (!std::isfinite(eps) || eps < 0.f) return ATTN_ERR_INVALID_ARG;
  if (!aligned(qkv, 16) || !aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) ||
      !aligned(wq, w_fp32 ? 4 : 2) || !aligned(wk, w_fp32 ? 4 : 2) || !aligned(inv_freq, 4) ||
      !aligned(positions, 4))
    return ATTN_ERR_INVALID_ARG;
  if (d != 64 && d != 128) return ATTN_ERR_UNSUPPORTED;
  if (n_freq < 1 || 2 * (int64_t)n_freq > d) return ATTN_ERR_INVALID_ARG;
  if (n_freq % 8 != 0) return ATTN_ERR_UNSUPPORTED;
  if (too_many(B, N, 1 << 30) || (int64_t)Hq + 2 * (int64_t)Hkv > (1 << 20))
    return ATTN_ERR_UNSUPPORTED;
  const int64_t row = ((int64_t)Hq + 2 * (int64_t)Hkv) * d;
  if (stride_b < 0 || stride_n < 0 || stride_b % 8 != 0 || stride_n % 8 != 0 ||
      (N > 1 && stride_n < row) || (B > 1 && stride_b < row) || stride_b > kMaxOffset / B ||
      stride_n > kMaxOffset / N)
    return ATTN_ERR_INVALID_ARG;
  const uint64_t bn = (uint64_t)B * N * d * 2;
  const Span in[5] = {span(qkv, ((uint64_t)(B - 1) * stride_b + (uint64_t)(N - 1) * stride_n + row) * 2),
                      span(wq, (uint64_t)d * (w_fp32 ? 4 : 2)), span(wk, (uint64_t)d * (w_fp32 ? 4 : 2)),
                      span(inv_freq, (uint64_t)n_freq * 4), span(positions, (uint64_t)B * N * 4)};
  const Span out[3] = {span(q, bn * Hq), span(k, bn * Hkv), span(v, bn * Hkv)};
  if (!apart(out, 3, in, 5)) return ATTN_ERR_INVALID_ARG;
  const int inj = osx::take_injected();
  if (inj != ATTN_OK) return static_cast<attn_status_t>(inj);
  const osx::RopeParams p{static_cast<const __nv_bfloat16*>(qkv), stride_b, stride_n, wq, wk,
                          inv_freq, positions, static_cast<__nv_bfloat16*>(q),
                          static_cast<__nv_bfloat16*>(k), static_cast<__nv_bfloat16*>(v),
                          B, N, Hq, Hkv, n_freq, w_fp32, eps};
  return static_cast<attn_status_t>(
      osx::launch_qk_norm_rope(p, d, interleaved, static_cast<cudaStream_t>(stream)));
}

attn_status_t attn_kv4_append(const void* k, const void* v, void* cache, const int32_t* slots,
                              int B, int Hkv, int N, int d, int page_size, int n_pages,
                              void* stream) {
  if (!k || !v || !slots || B < 1 || N < 1) return ATTN_ERR_INVALID_ARG;
  if (!aligned(k, 16) || !aligned(v, 16) || !aligned(slots, 4)) return ATTN_ERR_INVALID_ARG;
  const attn_status_t st = check_cache(cache, Hkv, d, page_size, n_pages);
  if (st != ATTN_OK) return st;
  if (too_many(B, N, 1 << 30) || !copy_items(B, N, Hkv)) return ATTN_ERR_UNSUPPORTED;
  const uint64_t bytes = (uint64_t)B * Hkv * N * d * 2;
  const Span in[3] = {span(k, bytes), span(v, bytes), span(slots, (uint64_t)B * N * 4)};
  const Span out[1] = {span(cache, cache_bytes(Hkv, d, page_size, n_pages))};
  if (!apart(out, 1, in, 3)) return ATTN_ERR_INVALID_ARG;
  const int inj = osx::take_injected();
  if (inj != ATTN_OK) return static_cast<attn_status_t>(inj);
  osx::Kv4CopyParams p = {};
  p.k = static_cast<const __nv_bfloat16*>(k);
  p.v = static_cast<const __nv_bfloat16*>(v);
  p.cache = static_cast<uint32_t*>(cache);
  p.slots = slots;
  p.B = B;
  p.N = N;
  p.Hkv = Hkv;
  p.page_size = page_size;
  p.n_pages = n_pages;
  p.windows = copy_windows(N);
  p.items = copy_items(B, N, Hkv);
  return static_cast<attn_status_t>(
      osx::launch_kv4_append(p, d, static_cast<cudaStream_t>(stream)));
}

attn_status_t attn_kv4_read(const void* cache, const int32_t* table, const int32_t* start,
                            const int32_t* lens, void* k, void* v, int B, int Hkv, int N, int d,
                            int page_size, int n_pages, int width, void* stream) {
  if (!table || !start || !lens || !k || !v || B < 1 || N < 1 || width < 1)
    return ATTN_ERR_INVALID_ARG;
  if (!aligned(k, 16) || !aligned(v, 16) || !aligned(table, 4) || !aligned(start, 4) ||
      !aligned(lens, 4))
    return ATTN_ERR_INVALID_ARG;
  const attn_status_t st = check_cache(cache, Hkv, d, page_size, n_pages);
  if (st != ATTN_OK) return st;
  if (too_many(B, N, 1 << 30) || too_many(width, page_size, INT32_MAX) || !copy_items(B, N, Hkv))
    return ATTN_ERR_UNSUPPORTED;
  const uint64_t bytes = (uint64_t)B * Hkv * N * d * 2;
  const Span in[4] = {span(cache, cache_bytes(Hkv, d, page_size, n_pages)),
                      span(table, (uint64_t)B * width * 4), span(start, (uint64_t)B * 4),
                      span(lens, (uint64_t)B * 4)};
  const Span out[2] = {span(k, bytes), span(v, bytes)};
  if (!apart(out, 2, in, 4)) return ATTN_ERR_INVALID_ARG;
  const int inj = osx::take_injected();
  if (inj != ATTN_OK) return static_cast<attn_status_t>(inj);
  osx::Kv4CopyParams p = {};
  p.k_out = static_cast<__nv_bfloat16*>(k);
  p.v_out = static_cast<__nv_bfloat16*>(v);
  p.cache = static_cast<uint32_t*>(const_cast<void*>(cache));
  p.table = table;
  p.start = start;
  p.lens = lens;
  p.B = B;
  p.N = N;
  p.Hkv = Hkv;
  p.page_size = page_size;
  p.n_pages = n_pages;
  p.width = width;
  p.windows = copy_windows(N);
  p.items = copy_items(B, N, Hkv);
  return static_cast<attn_status_t>(osx::launch_kv4_read(p, d, static_cast<cudaStream_t>(stream)));
}

int64_t attn_kv4_fwd_workspace(int B, int Hq, int Hkv, int Nq, int d) {
  if (B < 1 || Hq < 1 || Hkv < 1 || Hq % Hkv != 0 || Nq < 1 || (d != 64 && d != 128) ||
      too_many(B, Hq, 1 << 30) || too_many(Hq, Nq, 1 << 30))
    return 0;
  return osx::kv4_workspace(B, Hkv, Hq / Hkv * Nq, d).bytes;
}

attn_status_t attn_kv4_fwd(const void* q, const void* cache, const int32_t* table,
                           const int32_t* lens, const int32_t* q_pos, void* o, float* lse,
                           int o_bf16, int B, int Hq, int Hkv, int Nq, int d, int page_size,
                           int n_pages, int width, int64_t max_len, int window, int sinks,
                           float scale, void* workspace, int64_t workspace_bytes, void* stream) {
  if (!q || !table || !lens || !o || !lse || !workspace) return ATTN_ERR_INVALID_ARG;
  if (B < 1 || Hq < 1 || Hkv < 1 || Hq % Hkv != 0 || Nq < 1 || width < 1 || max_len < 0)
    return ATTN_ERR_INVALID_ARG;
  if ((o_bf16 != 0 && o_bf16 != 1) || window < 0 || sinks < 0) return ATTN_ERR_INVALID_ARG;
  if (!std::isfinite(scale) || !(scale > 0.f)) return ATTN_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(o, 16) || !aligned(lse, 4) || !aligned(table, 4) ||
      !aligned(lens, 4) || !aligned(q_pos, 4) || !aligned(workspace, 16))
    return ATTN_ERR_INVALID_ARG;
  const attn_status_t st = check_cache(cache, Hkv, d, page_size, n_pages);
  if (st != ATTN_OK) return st;
  if (too_many(B, Hq, 1 << 30) || too_many(Hq, Nq, 1 << 30) ||
      too_many(width, page_size, INT32_MAX))
    return ATTN_ERR_UNSUPPORTED;
  // blocks of 16 tokens over all query tiles: a warp's share has to fit 31 bits
  const int64_t tiles = (int64_t)B * Hkv * (((int64_t)Hq / Hkv * Nq + 3) / 4);
  if (too_many(tiles, ((int64_t)width * page_size + 15) / 16, int64_t(1) << 40))
    return ATTN_ERR_UNSUPPORTED;
  const uint64_t rows = (uint64_t)B * Hq * Nq;
  const Span in[5] = {span(q, rows * d * 2), span(cache, cache_bytes(Hkv, d, page_size, n_pages)),
                      span(table, (uint64_t)B * width * 4), span(lens, (uint64_t)B * 4),
                      span(q_pos ? q_pos : lens, (uint64_t)B * 4)};
  const osx::Kv4Workspace ws = osx::kv4_workspace(B, Hkv, Hq / Hkv * Nq, d);
  if (workspace_bytes < ws.bytes) return ATTN_ERR_INVALID_ARG;
  const Span out[3] = {span(o, rows * d * (o_bf16 ? 2 : 4)), span(lse, rows * 4),
                       span(workspace, (uint64_t)ws.bytes)};
  if (!apart(out, 3, in, 5)) return ATTN_ERR_INVALID_ARG;
  const int inj = osx::take_injected();
  if (inj != ATTN_OK) return static_cast<attn_status_t>(inj);
  const int64_t room = (int64_t)width * page_size;
  osx::Kv4FwdParams p = {};
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.cache = static_cast<const uint32_t*>(cache);
  p.table = table;
  p.lens = lens;
  p.q_pos = q_pos;
  p.o = o;
  p.lse = lse;
  p.o_bf16 = o_bf16;
  p.ws_prefix = static_cast<long long*>(workspace);
  p.ws_ml = reinterpret_cast<float*>(static_cast<char*>(workspace) + ws.ml);
  p.ws_o = reinterpret_cast<float*>(static_cast<char*>(workspace) + ws.o);
  p.B = B;
  p.Hkv = Hkv;
  p.Nq = Nq;
  p.rows = Hq / Hkv * Nq;
  p.blocks_per_page = page_size / 16;
  p.page_magic = p.blocks_per_page == 1
                     ? 0xffffffffu
                     : static_cast<uint32_t>((uint64_t(1) << 32) / p.blocks_per_page);
  p.n_pages = n_pages;
  p.width = width;
  p.window = window;
  p.sinks = sinks;
  p.scale_log2 = static_cast<float>(static_cast<double>(scale) * 1.4426950408889634);
  return static_cast<attn_status_t>(
      osx::launch_kv4_fwd(p, d, max_len > 0 && max_len < room ? max_len : room,
                          static_cast<cudaStream_t>(stream)));
}

int64_t attn_window_fwd_workspace(int B, int Hq, int Hkv, int64_t Nq, int d) {
  if (B < 1 || Hq < 1 || Hkv < 1 || Hq % Hkv != 0 || Nq < 1 || Nq > kMaxRows ||
      (d != 64 && d != 128) || too_many(B, Hq, 1 << 30) || !osx::window_is_token(B, Hq, Hkv, Nq))
    return 0;
  return osx::token_workspace(B, Hkv, (int)(Hq / Hkv * Nq), d).bytes;
}

attn_status_t attn_window_fwd(const void* q, const void* k, const void* v, void* o, float* lse,
                              int o_bf16, int B, int Hq, int Hkv, int64_t Nq, int64_t Nkv,
                              int64_t q_ld, int64_t kv_ld, int64_t q_off, int64_t kv_off, int d,
                              int window, int sinks, float scale, void* workspace,
                              int64_t workspace_bytes, void* stream) {
  if (!q || !k || !v || !o || !lse) return ATTN_ERR_INVALID_ARG;
  if (B < 1 || Hq < 1 || Hkv < 1 || Hq % Hkv != 0) return ATTN_ERR_INVALID_ARG;
  if (Nq < 1 || Nkv < 1 || q_ld < Nq || kv_ld < Nkv || q_off < 0 || kv_off < 0)
    return ATTN_ERR_INVALID_ARG;
  if ((o_bf16 != 0 && o_bf16 != 1) || window < 1 || sinks < 0) return ATTN_ERR_INVALID_ARG;
  if (!std::isfinite(scale) || !(scale > 0.f)) return ATTN_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(o, 16) || !aligned(lse, 4))
    return ATTN_ERR_INVALID_ARG;
  if (d != 64 && d != 128) return ATTN_ERR_UNSUPPORTED;
  if (Nq > kMaxRows || Nkv > kMaxRows || q_ld > kMaxRows || kv_ld > kMaxRows ||
      too_many(B, Hq, 1 << 30) || q_off > kMaxOffset || kv_off > kMaxOffset)
    return ATTN_ERR_UNSUPPORTED;
  const uint64_t bh = (uint64_t)B * Hq, bhkv = (uint64_t)B * Hkv;
  const Span in[3] = {span(q, ((bh - 1) * q_ld + Nq) * d * 2),
                      span(k, ((bhkv - 1) * kv_ld + Nkv) * d * 2),
                      span(v, ((bhkv - 1) * kv_ld + Nkv) * d * 2)};
  const int64_t ws = attn_window_fwd_workspace(B, Hq, Hkv, Nq, d);
  if (workspace_bytes < ws || (ws > 0 && (!workspace || !aligned(workspace, 16))))
    return ATTN_ERR_INVALID_ARG;
  const Span out[3] = {span(o, bh * Nq * d * (o_bf16 ? 2 : 4)), span(lse, bh * Nq * 4),
                       span(workspace, (uint64_t)ws)};
  if (!apart(out, ws > 0 ? 3 : 2, in, 3)) return ATTN_ERR_INVALID_ARG;
  const int inj = osx::take_injected();
  if (inj != ATTN_OK) return static_cast<attn_status_t>(inj);
  const osx::WindowLaunch a{q,    k,     v,     o,      lse, o_bf16, B,     Hq,    Hkv, Nq, Nkv,
                            q_ld, kv_ld, q_off, kv_off, d,   window, sinks, scale,
                            static_cast<float*>(workspace)};
  return static_cast<attn_status_t>(osx::launch_window(a, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
