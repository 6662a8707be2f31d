// serve_params.h - kernel parameters of the serving operators, shared by the ABI layer,
// the launchers and the kernels.
#pragma once

#include <cuda_bf16.h>

#include <cstdint>

namespace osx {

struct PlanParams {
  const int* lens;        // [B]
  const int* new_lens;    // [B]
  int* table;             // [B][width], entries of new pages written
  const int* free_pages;  // [n_free]
  const int* free_head;   // [1]
  int* slots;             // [B][n_new]
  int* positions;         // [B][n_new]
  int* lens_out;          // [B]
  int* head_out;          // [1]
  int* served;            // [B]
  int B, n_new, width, page_size, n_free;
};

struct RopeParams {
  const __nv_bfloat16* qkv;  // [B][N][(Hq + 2 Hkv) * d], strides in elements
  long long stride_b, stride_n;
  const void* wq;            // [d] bf16 or fp32
  const void* wk;
  const float* inv_freq;     // [n_freq]
  const int* positions;      // [B][N]
  __nv_bfloat16* q;          // [B][Hq][N][d]
  __nv_bfloat16* k;          // [B][Hkv][N][d]
  __nv_bfloat16* v;
  int B, N, Hq, Hkv, n_freq;
  int w_fp32;
  float eps;
};

struct Kv4CopyParams {
  const __nv_bfloat16* k;   // append: [B][Hkv][N][d]
  const __nv_bfloat16* v;
  __nv_bfloat16* k_out;     // read: [B][Hkv][N][d]
  __nv_bfloat16* v_out;
  uint32_t* cache;
  const int* slots;         // append: [B][N]
  const int* table;         // read: [B][width]
  const int* start;         // read: [B]
  const int* lens;          // read: [B]
  int B, N, Hkv, page_size, n_pages, width, windows;
  unsigned items;  // a warp each: (request, window, head, keys or values)
};

struct Kv4FwdParams {
  const __nv_bfloat16* q;   // [B][Hq][Nq][D]
  const uint32_t* cache;
  const int* table;         // [B][width]
  const int* lens;          // [B]
  const int* q_pos;         // [B] position of the first query token, or null: lens - Nq
  void* o;                  // [B][Hq][Nq][D] fp32 or bf16
  float* lse;               // [B][Hq][Nq]
  unsigned* status;
  int o_bf16;
  float* ws_o;              // partials by slot: rows, (base, denominator) pairs
  float* ws_ml;
  long long* ws_prefix;     // [B + 1] stages before each request
  int B, Hkv, Nq, rows, row_tiles;   // rows = group * Nq
  int blocks_per_page, n_pages, width;
  uint32_t page_magic;      // floor(2^32 / blocks_per_page), 2^32 - 1 for one
  int window, sinks;
  int stage_shift;          // a stage has 2^stage_shift blocks
  float scale_log2;
};

// The join of a decode launch's partials (see decode_common.cuh).
struct JoinParams {
  const float* parts;       // [slot][kRows][D]
  const float* ml;          // [slot][kRows][2]
  const long long* prefix;  // [B + 1] stages before each request's units, or null:
  long long n_stages;       // every unit has this many
  void* o;                  // rows of unit (b, h, tile): ((b Hkv + h) rows + tile kRows ..)
  float* lse;
  int o_bf16, B, Hkv, rows, row_tiles, n_warps;
};

// A few query rows over bf16 keys with a window (the token form of attn_window_fwd).
struct TokenParams {
  const __nv_bfloat16* q;   // [B][Hq][q_ld][D]
  const __nv_bfloat16* k;   // [B][Hkv][kv_ld][D]
  const __nv_bfloat16* v;
  void* o;
  float* lse;
  float* ws_o;
  float* ws_ml;
  int o_bf16, B, Hkv, Nq, rows, row_tiles;  // rows = group * Nq
  int Nkv;
  long long q_ld, kv_ld, rel;
  int window, sinks, n_sink_blocks, w0, n_blocks;  // blocks of 16 keys: sinks', then from w0
  float scale_log2;
};

struct WindowLaunch {
  const void* q;  // bf16 [B][Hq][q_ld][d], rows [0, Nq)
  const void* k;  // bf16 [B][Hkv][kv_ld][d], rows [0, Nkv)
  const void* v;
  void* o;        // [B][Hq][Nq][d] fp32 or bf16
  float* lse;     // [B][Hq][Nq]
  int o_bf16, B, Hq, Hkv;
  long long Nq, Nkv, q_ld, kv_ld, q_off, kv_off;
  int d, window;
  long long sinks;
  float scale;
  float* workspace;  // of the token form (null where it is not used)
};

struct WindowParams {
  void* o;
  float* lse;
  unsigned* status;
  int o_bf16, Hq, Hkv, group;
  int Nq, Nkv;
  long long rel;     // position of query row 0 less that of key row 0
  int window, sinks; // sinks: key rows [0, sinks) of this chunk stay visible
  int pair;        // a unit is 128 rows of two neighbouring heads, else 256 rows of one
  int heads, row_blocks, units;  // heads (or pairs of them), row blocks of 128 or 256
  int cut_blocks;  // row blocks whose windows the sequence's start cuts
  float scale_log2;
};

}  // namespace osx
