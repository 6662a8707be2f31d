// serve_kernels.cu - device translation unit of the serving operators: instantiations and
// launchers.
#include <mutex>

#include "../../include/attn.h"
#include "attn_internal.h"
#include "attn_window_kernel.cuh"
#include "decode_common.cuh"
#include "kv4_copy_kernels.cuh"
#include "kv4_fwd_kernel.cuh"
#include "kv_plan_kernel.cuh"
#include "qk_norm_rope_kernel.cuh"
#include "tma_host.h"
#include "window_token_kernel.cuh"

namespace osx {

namespace {

int launched() {
  if (cudaGetLastError() != cudaSuccess) return ATTN_ERR_CUDA;
  count_launch();
  return ATTN_OK;
}

// A launch whose blocks may start before the launch before it in the stream has ended (each
// waits for that in the kernel before it touches global memory): its launch latency and
// set-up lie beside that one's end.
template <class... A>
int launch_dependent(void (*kernel)(A...), unsigned grid, unsigned threads, uint32_t smem,
                     cudaStream_t stream, const A&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, kernel, args...) != cudaSuccess) {
    cudaGetLastError();
    return ATTN_ERR_CUDA;
  }
  return launched();
}

// Blocks of a one-dimensional grid, or 0 when there are more than a grid can have.
unsigned grid_1d(long long blocks) {
  return blocks > 0 && blocks <= 0x7fffffffLL ? static_cast<unsigned>(blocks) : 0u;
}

// A kernel's shared memory limit, set once per device.
template <auto kKernel>
int prepare_kernel(uint32_t smem) {
  constexpr int kMaxDevices = 64;
  static std::mutex mutex;
  static bool ready[kMaxDevices];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return ATTN_ERR_CUDA;
  std::lock_guard<std::mutex> lock(mutex);
  if (ready[dev]) return ATTN_OK;
  if (cudaFuncSetAttribute(kKernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) !=
      cudaSuccess)
    return ATTN_ERR_CUDA;
  ready[dev] = true;
  return ATTN_OK;
}

// The join of a decode launch, 64 values of a row to a block. A unit has about warps / units
// partials, and no more than stages; a block takes up to five per group of 16 threads in one
// round of loads. (Measured with 128 / 256 / 512 threads: 55 partials a unit 18.0 / 17.2 /
// 18.4 us for the whole call, 148 partials 40.6 / 40.4 / 39.6 us.)
template <int D, int kRows>
int launch_join(const JoinParams& j, long long stages, cudaStream_t stream) {
  const long long units = (long long)j.B * j.Hkv * j.row_tiles;
  const unsigned grid = grid_1d(units * kRows * (D / 64));
  if (!grid) return ATTN_ERR_UNSUPPORTED;
  long long parts = j.n_warps / units + 1;
  if (stages < parts) parts = stages;
  if (parts <= 40)
    return launch_dependent(decode_join_kernel<D, kRows, 128>, grid, 128, 0, stream, j);
  if (parts <= 80)
    return launch_dependent(decode_join_kernel<D, kRows, 256>, grid, 256, 0, stream, j);
  return launch_dependent(decode_join_kernel<D, kRows, 512>, grid, 512, 0, stream, j);
}

template <int D, int NT>
int launch_kv4_fwd_dn(Kv4FwdParams p, long long max_len, int num_sms, cudaStream_t stream) {
  using C = Kv4FwdCfg<D, NT>;
  p.row_tiles = (p.rows + C::kRows - 1) / C::kRows;
  const long long items = (long long)p.B * p.Hkv * p.row_tiles;
  if (!grid_1d(items * C::kRows * (D / 64))) return ATTN_ERR_UNSUPPORTED;  // the join's blocks
  // one block per SM, or fewer where there cannot be a stage for each of their warps
  long long keys = max_len;
  if (p.window && (long long)p.window + p.Nq + p.sinks < keys)
    keys = (long long)p.window + p.Nq + p.sinks;
  int grid = num_sms < kKv4MaxBlocks ? num_sms : kKv4MaxBlocks;
  // one block to a stage where that gives every warp at most one (a short call's time is
  // that of its longest chain: 3 requests of up to 700 tokens, windowed, 10.2 -> 8.9 us)
  long long stages = keys / 16 + 2;  // of a unit, at most
  p.stage_shift = 0;
  if (items * stages > (long long)grid * C::kWarps) {
    stages = keys / (16 * C::kSB) + 2;
    p.stage_shift = C::kSB == 4 ? 2 : 1;
  }
  static_assert(C::kSB == 2 || C::kSB == 4, "blocks of a stage");
  if (items * stages < grid) grid = (int)(items * stages);
  const int rc = prepare_kernel<kv4_fwd_kernel<D, NT>>(C::kSmemBytes);
  if (rc != ATTN_OK) return rc;
  const int st =
      launch_dependent(kv4_fwd_kernel<D, NT>, grid, C::kWarps * 32, C::kSmemBytes, stream, p);
  if (st != ATTN_OK) return st;
  const JoinParams j{p.ws_o, p.ws_ml, p.ws_prefix, 0, p.o, p.lse, p.o_bf16, p.B, p.Hkv, p.rows,
                     p.row_tiles, grid * C::kWarps};
  return launch_join<D, C::kRows>(j, stages, stream);
}

template <int D, int NT>
Kv4Workspace kv4_workspace_dn(int B, int Hkv, int rows) {
  using C = Kv4FwdCfg<D, NT>;
  const long long items = (long long)B * Hkv * ((rows + C::kRows - 1) / C::kRows);
  const long long slots = (long long)kKv4MaxBlocks * C::kWarps + items;
  Kv4Workspace w;
  w.ml = ((long long)(B + 1) * 8 + 255) / 256 * 256;
  w.o = w.ml + (slots * C::kRows * 2 * 4 + 255) / 256 * 256;
  w.bytes = w.o + slots * C::kRows * D * 4;
  return w;
}

// Blocks of 16 keys that the rows at positions rel .. rel + Nq - 1 (in key rows) see: those
// of the sinks, then n_blocks - n_sink_blocks from w0 on.
void window_blocks(const WindowLaunch& a, TokenParams* p) {
  const long long rel = a.q_off - a.kv_off;
  const long long hi = rel + a.Nq < a.Nkv ? rel + a.Nq : a.Nkv;  // keys below may be seen
  long long lo = rel - a.window + 1;
  if (lo < 0) lo = 0;
  long long s = a.sinks - a.kv_off;
  s = s < 0 ? 0 : (s < a.Nkv ? s : a.Nkv);
  p->sinks = (int)s;
  if (s > hi) s = hi;
  const long long w0 = lo / 16, n_w = hi > lo ? (hi - 1) / 16 - w0 + 1 : 0;
  long long n_s = s > 0 ? (s + 15) / 16 : 0;
  if (n_w > 0 && n_s > w0) n_s = w0;
  p->n_sink_blocks = (int)n_s;
  p->w0 = (int)(n_w > 0 ? w0 : 0);
  p->n_blocks = (int)(n_s + n_w);
}

template <int D, int NT>
int launch_token_dn(const WindowLaunch& a, const DeviceProps& dp, cudaStream_t stream) {
  using C = TokenCfg<NT>;
  TokenParams p;
  p.q = static_cast<const __nv_bfloat16*>(a.q);
  p.k = static_cast<const __nv_bfloat16*>(a.k);
  p.v = static_cast<const __nv_bfloat16*>(a.v);
  p.o = a.o;
  p.lse = a.lse;
  p.o_bf16 = a.o_bf16;
  p.B = a.B;
  p.Hkv = a.Hkv;
  p.Nq = (int)a.Nq;
  p.rows = (int)(a.Hq / a.Hkv * a.Nq);
  p.row_tiles = (p.rows + C::kRows - 1) / C::kRows;
  p.Nkv = (int)a.Nkv;
  p.q_ld = a.q_ld;
  p.kv_ld = a.kv_ld;
  p.rel = a.q_off - a.kv_off;
  p.window = a.window;
  p.scale_log2 = static_cast<float>(static_cast<double>(a.scale) * 1.4426950408889634);
  window_blocks(a, &p);
  const long long units = (long long)a.B * a.Hkv * p.row_tiles;
  if (units > 0x7fffffffLL / C::kRows) return ATTN_ERR_UNSUPPORTED;
  const TokenWorkspace ws = token_workspace(a.B, a.Hkv, p.rows, D);
  p.ws_ml = a.workspace;
  p.ws_o = a.workspace + ws.o / 4;
  int grid = dp.num_sms < kTokenMaxBlocks ? dp.num_sms : kTokenMaxBlocks;
  if (units * p.n_blocks < grid) grid = (int)(units * p.n_blocks);
  if (p.n_blocks > 0) {
    const int st = launch_dependent(window_token_kernel<D, NT>, grid, C::kWarps * 32, 0, stream, p);
    if (st != ATTN_OK) return st;
  }
  const JoinParams j{p.ws_o,   p.ws_ml, nullptr, p.n_blocks, p.o,         p.lse,
                     p.o_bf16, p.B,     p.Hkv,   p.rows,     p.row_tiles, grid * C::kWarps};
  return launch_join<D, C::kRows>(j, p.n_blocks, stream);
}

template <int D>
int launch_window_d(const WindowLaunch& a, const DeviceProps& dp, cudaStream_t stream) {
  using C = WindowCfg<D>;
  CUtensorMap tq, tk, tv;
  if (!encode_rows_bf16(&tq, a.q, (uint64_t)a.B * a.Hq, a.Nq, a.q_ld, D, 128) ||
      !encode_rows_bf16(&tk, a.k, (uint64_t)a.B * a.Hkv, a.Nkv, a.kv_ld, D, 128) ||
      !encode_rows_bf16(&tv, a.v, (uint64_t)a.B * a.Hkv, a.Nkv, a.kv_ld, D, 128))
    return ATTN_ERR_UNSUPPORTED;
  WindowParams p;
  p.status = dp.status;
  p.o = a.o;
  p.lse = a.lse;
  p.o_bf16 = a.o_bf16;
  p.Hq = a.Hq;
  p.Hkv = a.Hkv;
  p.group = a.Hq / a.Hkv;
  p.Nq = (int)a.Nq;
  p.Nkv = (int)a.Nkv;
  p.rel = a.q_off - a.kv_off;
  p.window = a.window;
  const long long s = a.sinks - a.kv_off;
  p.sinks = (int)(s < 0 ? 0 : (s < a.Nkv ? s : a.Nkv));
  p.scale_log2 = static_cast<float>(static_cast<double>(a.scale) * 1.4426950408889634);
  p.pair = p.group % 2 == 0;
  const int per_block = p.pair ? 128 : 256;
  p.heads = p.pair ? a.B * a.Hq / 2 : a.B * a.Hq;
  p.row_blocks = (int)((a.Nq + per_block - 1) / per_block);
  const long long units = (long long)p.heads * p.row_blocks;
  if (units > 0x7fffffffLL) return ATTN_ERR_UNSUPPORTED;
  p.units = (int)units;
  // row blocks with per_block qp < window - 1 - rel
  const long long cut = a.window - 1 - p.rel;
  p.cut_blocks = (int)(cut <= 0 ? 0
                                : ((cut + per_block - 1) / per_block < p.row_blocks
                                       ? (cut + per_block - 1) / per_block
                                       : p.row_blocks));
  const int rc = prepare_kernel<attn_window_kernel<D>>(C::kSmemBytes);
  if (rc != ATTN_OK) return rc;
  const int grid = units < dp.num_sms ? (int)units : dp.num_sms;
  return launch_dependent(attn_window_kernel<D>, grid, C::kThreads, C::kSmemBytes, stream, tq, tk,
                          tv, p);
}

}  // namespace

int launch_window(const WindowLaunch& a, cudaStream_t stream) {
  DeviceProps dp;
  int rc = device_props(&dp);
  if (rc != ATTN_OK) return rc;
  if (window_is_token(a.B, a.Hq, a.Hkv, a.Nq)) {
    const bool few = a.Hq / a.Hkv * a.Nq <= 4;
    if (a.d == 128)
      return few ? launch_token_dn<128, 1>(a, dp, stream) : launch_token_dn<128, 2>(a, dp, stream);
    return few ? launch_token_dn<64, 1>(a, dp, stream) : launch_token_dn<64, 2>(a, dp, stream);
  }
  return a.d == 128 ? launch_window_d<128>(a, dp, stream) : launch_window_d<64>(a, dp, stream);
}

// The token form costs about 1.45 ns per 16-key block of a unit (8 query rows of a key/value
// head), the tile form about 1.95 us per 128-key tile and round of 256-row units over the
// SMs: the token form is the cheaper one up to some 168 units a round. Measured (us, token /
// tile form; window 4096 and d = 128 unless said): 1 x 8/1 heads, 1 row 10 / 62, 32 rows 21 /
// 64; 8 x 32/8 heads, 2 rows 42 / 129, 8 rows 101 / 129, 16 rows 192 / 129; 16 x 16/16, d =
// 64, window 2048, 4 rows 30 / 61, 16 rows 80 / 62; 4 x 32/8, window 128, 16 rows 18 / 12.
bool window_is_token(int B, int Hq, int Hkv, long long Nq) {
  constexpr long long kSms = 148, kUnitsPerRound = 160;
  const long long rows = Hq / Hkv * Nq;
  const long long units = (long long)B * Hkv * ((rows + 7) / 8);
  const long long rounds = ((long long)B * Hq * ((Nq + 255) / 256) + kSms - 1) / kSms;
  return units <= kUnitsPerRound * rounds;
}

TokenWorkspace token_workspace(int B, int Hkv, int rows, int d) {
  const int tile = rows <= 4 ? TokenCfg<1>::kRows : TokenCfg<2>::kRows;
  const int warps = rows <= 4 ? TokenCfg<1>::kWarps : TokenCfg<2>::kWarps;
  const long long units = (long long)B * Hkv * ((rows + tile - 1) / tile);
  const long long slots = (long long)kTokenMaxBlocks * warps + units;
  TokenWorkspace w;
  w.o = (slots * tile * 2 * 4 + 255) / 256 * 256;
  w.bytes = w.o + slots * tile * d * 4;
  return w;
}

int launch_kv_plan(const PlanParams& p, cudaStream_t stream) {
  DeviceProps dp;
  int rc = device_props(&dp);
  if (rc != ATTN_OK) return rc;
  const unsigned grid = grid_1d(((long long)p.B * p.n_new + kPlanChunk - 1) / kPlanChunk);
  if (!grid) return ATTN_ERR_UNSUPPORTED;
  return launch_dependent(kv_plan_kernel, grid, kPlanThreads, 0, stream, p);
}

int launch_qk_norm_rope(const RopeParams& p, int d, int interleaved, cudaStream_t stream) {
  DeviceProps dp;
  int rc = device_props(&dp);
  if (rc != ATTN_OK) return rc;
  // a warp per token, or up to eight where that would leave warps idle (four blocks an SM)
  constexpr int kWarps = kRopeThreads / 32;
  const long long tokens = (long long)p.B * p.N, warps = 4ll * dp.num_sms * kWarps;
  int split = 1;
  while (split < kWarps && tokens * split * 2 <= warps) split *= 2;
  const long long blocks = (tokens * split + kWarps - 1) / kWarps, most = 4ll * dp.num_sms;
  const unsigned grid = grid_1d(blocks < most ? blocks : most);
  auto* kernel = d == 128 ? (interleaved ? qk_norm_rope_kernel<128, true> : qk_norm_rope_kernel<128, false>)
                          : (interleaved ? qk_norm_rope_kernel<64, true> : qk_norm_rope_kernel<64, false>);
  return launch_dependent(kernel, grid, kRopeThreads, 0, stream, p, split);
}

static int launch_kv4_copy(void (*kernel)(Kv4CopyParams), const Kv4CopyParams& p,
                           cudaStream_t stream) {
  DeviceProps dp;
  const int rc = device_props(&dp);
  if (rc != ATTN_OK) return rc;
  const unsigned grid = grid_1d(((long long)p.items + kKv4CopyWarps - 1) / kKv4CopyWarps);
  if (!grid) return ATTN_ERR_UNSUPPORTED;
  return launch_dependent(kernel, grid, kKv4CopyWarps * 32, 0, stream, p);
}

int launch_kv4_append(const Kv4CopyParams& p, int d, cudaStream_t stream) {
  return launch_kv4_copy(d == 128 ? kv4_append_kernel<128> : kv4_append_kernel<64>, p, stream);
}

int launch_kv4_read(const Kv4CopyParams& p, int d, cudaStream_t stream) {
  return launch_kv4_copy(d == 128 ? kv4_read_kernel<128> : kv4_read_kernel<64>, p, stream);
}

// 4 query rows a unit, or 8 (the unpacked codes then serve twice the rows)
Kv4Workspace kv4_workspace(int B, int Hkv, int rows, int d) {
  if (d == 128)
    return rows <= 4 ? kv4_workspace_dn<128, 1>(B, Hkv, rows) : kv4_workspace_dn<128, 2>(B, Hkv, rows);
  return rows <= 4 ? kv4_workspace_dn<64, 1>(B, Hkv, rows) : kv4_workspace_dn<64, 2>(B, Hkv, rows);
}

int launch_kv4_fwd(const Kv4FwdParams& params, int d, long long max_len, cudaStream_t stream) {
  DeviceProps dp;
  int rc = device_props(&dp);
  if (rc != ATTN_OK) return rc;
  Kv4FwdParams p = params;
  p.status = dp.status;
  if (d == 128)
    return p.rows <= 4 ? launch_kv4_fwd_dn<128, 1>(p, max_len, dp.num_sms, stream)
                       : launch_kv4_fwd_dn<128, 2>(p, max_len, dp.num_sms, stream);
  return p.rows <= 4 ? launch_kv4_fwd_dn<64, 1>(p, max_len, dp.num_sms, stream)
                     : launch_kv4_fwd_dn<64, 2>(p, max_len, dp.num_sms, stream);
}

}  // namespace osx
