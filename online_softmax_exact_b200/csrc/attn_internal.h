// attn_internal.h - interface between the C ABI layer (attn_api.cu) and the kernel
// translation unit (attn_kernels.cu). Not installed; not part of the ABI.
#pragma once

#include <cuda_runtime.h>
#include <cstdint>

namespace osx {

// One (query chunk, key/value chunk) pair of a launch; rows are tensor-map rows.
struct PairLaunch {
  long long q_start, q_len, kv_start, kv_len, q_off, kv_off;
  float* o;
  float* lse;
};

// One attention launch over up to kMaxPairs pairs sharing the q/k/v tensor maps;
// arguments have already been validated by the ABI layer. The maps span q_rows
// (resp. kv_rows) rows of [B*H][rows][d] views with row strides q_ld / kv_ld.
struct FwdLaunch {
  const void* q;
  const void* k;
  const void* v;
  int B, Hq, Hkv;
  long long q_rows, kv_rows, q_ld, kv_ld;
  int d;
  int causal;
  float scale;
  int accumulate;  // o/lse are in/out accumulators (see attn_fwd_partial_acc)
  int n_pairs;
  const PairLaunch* pairs;
};

// Returns 0 (ATTN_OK) or an attn_status_t failure code.
int launch_fwd(const FwdLaunch& a, cudaStream_t stream);
int launch_merge(const float* const* o_parts, const float* const* lse_parts, int n_parts,
                 float* o, float* lse, long long rows, int d, cudaStream_t stream);
// Launches the failure-path check kernel (a bounded wait that must run out).
int launch_wait_probe(long long limit_cycles, cudaStream_t stream);
// Launches the exponential check kernel (y = 2^x by the polynomial or by ex2.approx).
int launch_exp2_probe(const float* x, float* y, long long n, int use_poly, cudaStream_t stream);
// Reads (and optionally clears) the device status word of the current device.
int read_device_status(unsigned* out, int reset);
uint64_t launch_count();

// Per-device properties of the current device (looked up once per device).
struct DeviceProps {
  int num_sms;
  unsigned* status;  // device address of the status word
};
int device_props(DeviceProps* out);
void count_launch();

// Serving operators (arguments already validated by the ABI layer).
struct PlanParams;
struct RopeParams;
struct Kv4CopyParams;
struct Kv4FwdParams;
struct WindowLaunch;
int launch_window(const WindowLaunch& a, cudaStream_t stream);
// Whether a windowed call runs in its token form, and that form's workspace (statistics at
// offset 0, rows at o).
constexpr int kTokenMaxBlocks = 160;  // blocks of the attention launch at most
struct TokenWorkspace {
  long long o, bytes;
};
bool window_is_token(int B, int Hq, int Hkv, long long Nq);
TokenWorkspace token_workspace(int B, int Hkv, int rows, int d);
int launch_kv_plan(const PlanParams& p, cudaStream_t stream);
int launch_qk_norm_rope(const RopeParams& p, int d, int interleaved, cudaStream_t stream);
int launch_kv4_append(const Kv4CopyParams& p, int d, cudaStream_t stream);
int launch_kv4_read(const Kv4CopyParams& p, int d, cudaStream_t stream);
// Workspace of launch_kv4_fwd: byte offsets of its parts, and its size. The prefix sums
// are at offset 0.
struct Kv4Workspace {
  long long ml, o, bytes;
};
constexpr int kKv4MaxBlocks = 160;  // blocks of the attention launch at most
Kv4Workspace kv4_workspace(int B, int Hkv, int rows, int d);
// max_len: the longest request's length as far as the caller knows it (only the number of
// blocks depends on it)
int launch_kv4_fwd(const Kv4FwdParams& p, int d, long long max_len, cudaStream_t stream);

}  // namespace osx
