/*
 * attn.h - C ABI of libattn: exact blockwise self-attention forward on NVIDIA B200
 * (sm_100a), and the merge of partial results.
 *
 * What is computed. For every batch b, query head h and query row i:
 *     s_j   = scale * <q[b,h,i,:], k[b,g,j,:]>   over the visible keys j,
 *     O_i   = sum_j softmax(s)_j * v[b,g,j,:],
 *     LSE_i = ln(sum_j exp(s_j)),
 * with g = h / (Hq / Hkv). This is the conventional three-step attention
 * ("FlashAttention by hand": logits, a softmax row that sums to one, weights times
 * values), reached exactly, up to floating-point rounding, by the tiled online
 * softmax the same page describes: key/value tiles streamed through on-chip
 * memory, a running maximum and denominator, rescaling of the partial output when
 * the maximum grows, and one final division. The score matrix never reaches
 * global memory.
 *
 * Masking. With causal != 0, key j is visible to query i when
 * kv_off + j <= q_off + i (global positions; HOF SWIFT Attention, section 3,
 * Transform stage names causal masking). A row with no visible key has O = 0 and
 * LSE = -inf.
 *
 * Layouts. q, k, v are bf16, row-major [B][H][N][d] (d contiguous). O is fp32
 * [B][Hq][Nq][d]; LSE is fp32 [B][Hq][Nq], natural log, scale included.
 *
 * Ownership and execution. The caller owns every buffer; the library allocates no
 * device memory. All pointers named "device" must be device (or managed) memory.
 * Calls enqueue work on `stream` (a cudaStream_t; NULL is the legacy default
 * stream) and return without waiting. Buffers must stay valid until that work has
 * finished. No call throws; every call returns an attn_status_t.
 *
 * Errors. Arguments are checked before anything is launched: null or misaligned
 * pointers, non-positive sizes, Hq not a multiple of Hkv, outputs overlapping
 * inputs, a negative or non-finite scale, and offsets/leading dimensions that do
 * not fit give ATTN_ERR_INVALID_ARG. Shapes the kernels are not built for (d other
 * than 64 or 128, more than ATTN_MAX_MERGE_PARTS parts, sizes beyond the tensor-map
 * limits) give ATTN_ERR_UNSUPPORTED. A failed CUDA call gives ATTN_ERR_CUDA. NaN or
 * Inf inside the rows a call attends is not checked and gives unspecified results.
 *
 * Device-side failures. Every wait inside the kernels is bounded (4 s of wall-clock
 * time). A wait that runs out stops the kernel early, leaves its outputs unspecified
 * and is recorded in a per-device status word; the launch itself has already returned
 * ATTN_OK by then. Results therefore count only once attn_device_status has reported
 * ATTN_OK for the stream they were computed on. Nothing traps or faults.
 */
#ifndef ATTN_H
#define ATTN_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  ATTN_OK = 0,
  ATTN_ERR_INVALID_ARG = 1,
  ATTN_ERR_UNSUPPORTED = 2,
  ATTN_ERR_CUDA = 3,
  ATTN_ERR_TIMEOUT = 4,
  ATTN_ERR_INJECTED = 5
} attn_status_t;

#define ATTN_MAX_MERGE_PARTS 64
#define ATTN_MAX_BATCH_PAIRS 48

/* One (query chunk, key/value chunk) pair of attn_fwd_partial_batch. Rows count in the
 * parent tensors; o and lse are the pair's own outputs (or accumulators). */
typedef struct {
  int64_t q_start, q_len;   /* query rows [q_start, q_start + q_len) */
  int64_t kv_start, kv_len; /* key/value rows [kv_start, kv_start + kv_len) */
  int64_t q_off, kv_off;    /* global positions of the first rows (causal test) */
  float* o;                 /* device, fp32 [B][Hq][q_len][d], 16-byte aligned */
  float* lse;               /* device, fp32 [B][Hq][q_len], 4-byte aligned */
} attn_pair_t;

/* Static description of a status code. Never NULL. */
const char* attn_status_string(int status);

/* ABI version: (major << 16) | minor. */
int attn_version(void);

/*
 * attn_fwd - single-pass attention over a whole sequence ("FlashAttention by hand",
 * paragraphs on the fused tiled computation, the running statistics, rescaling and
 * the final division).
 *
 *   q      device, bf16 [B][Hq][N][d], 16-byte aligned
 *   k, v   device, bf16 [B][Hkv][N][d], 16-byte aligned
 *   o      device, fp32 [B][Hq][N][d], 16-byte aligned (written)
 *   lse    device, fp32 [B][Hq][N], 4-byte aligned (written)
 *   B, Hq, Hkv >= 1 with Hq % Hkv == 0; N >= 1; d in {64, 128}
 *   causal 0 or 1 (key j visible to query i iff j <= i)
 *   scale  finite, >= 0 (normally 1/sqrt(d))
 *   stream cudaStream_t to enqueue on
 */
attn_status_t attn_fwd(const void* q, const void* k, const void* v, float* o, float* lse,
                       int B, int Hq, int Hkv, int64_t N, int d, int causal, float scale,
                       void* stream);

/*
 * attn_fwd_partial - attention of one query chunk against one key/value chunk: one
 * ring step of Ring Attention ("Ring Attention with Blockwise Parallel
 * Transformers", section 3: each device attends its query block to the key/value
 * block it currently holds), or one fragment of the ATTENTION2D query x key/value
 * grid (section 3: fragment-local statistics). The result is the NORMALISED
 * partial output over this chunk's visible keys plus its LSE, ready for
 * attn_merge.
 *
 *   q        device, bf16: &Q[0][0][q_start][0] of a parent tensor
 *            [B][Hq][q_ld][d]; the chunk is rows [q_start, q_start + Nq)
 *   k_chunk, v_chunk
 *            device, bf16: &K[0][0][kv_start][0] of parents [B][Hkv][kv_ld][d];
 *            the chunk is rows [kv_start, kv_start + Nkv); rows beyond it are
 *            never read
 *   o_part   device, fp32 dense [B][Hq][Nq][d] (written)
 *   lse_part device, fp32 dense [B][Hq][Nq] (written)
 *   q_ld >= Nq, kv_ld >= Nkv: allocated sequence length of the parents
 *   q_off, kv_off >= 0: global position of the chunks' first rows (used only for
 *            the causal test kv_off + j <= q_off + i)
 *   other arguments as for attn_fwd. All pointers 16-byte aligned (lse_part 4).
 */
attn_status_t attn_fwd_partial(const void* q, const void* k_chunk, const void* v_chunk,
                               float* o_part, float* lse_part, int B, int Hq, int Hkv,
                               int64_t Nq, int64_t Nkv, int64_t q_ld, int64_t kv_ld,
                               int64_t q_off, int64_t kv_off, int d, int causal,
                               float scale, void* stream);

/*
 * attn_fwd_partial_acc - attn_fwd_partial fused with the merge: o_acc and lse_acc
 * hold, on entry, a normalised partial result over keys disjoint from this chunk
 * (LSE = -inf with O = 0 where no key has been seen yet), and on exit the
 * combination of that partial with this chunk's, by the same log-sum-exp rule as
 * attn_merge. This is the running update a Ring Attention device applies at each
 * ring step ("Ring Attention with Blockwise Parallel Transformers", section 3) and the
 * rescale of the online softmax ("FlashAttention by hand", paragraphs on the running
 * statistics and rescaling) applied at chunk granularity; it needs no buffer for the
 * chunk's own partial and no separate merge launch. A chunk none of whose keys is
 * visible to a row leaves that row unchanged.
 *
 *   o_acc, lse_acc  device, fp32 [B][Hq][Nq][d] and [B][Hq][Nq], read and written
 *   other arguments exactly as for attn_fwd_partial.
 * Successive calls on one accumulator must be ordered (one stream); calls on
 * different accumulators may run concurrently.
 */
attn_status_t attn_fwd_partial_acc(const void* q, const void* k_chunk, const void* v_chunk,
                                   float* o_acc, float* lse_acc, int B, int Hq, int Hkv,
                                   int64_t Nq, int64_t Nkv, int64_t q_ld, int64_t kv_ld,
                                   int64_t q_off, int64_t kv_off, int d, int causal,
                                   float scale, void* stream);

/*
 * attn_fwd_partial_batch - several pairs of attn_fwd_partial (accumulate = 0) or of
 * attn_fwd_partial_acc (accumulate = 1) over the same parent tensors in ONE launch:
 * e.g. all the chunk pairs of a ring step, or of a whole emulated ring. Each pair's
 * result is exactly that of the single-pair call; the work units of all pairs share
 * one persistent grid, heaviest first, so the tail of one pair is filled by the next.
 *
 *   q      device, bf16 parent [B][Hq][q_ld][d];  k, v: parents [B][Hkv][kv_ld][d]
 *   pairs  HOST array of n_pairs (1 .. ATTN_MAX_BATCH_PAIRS) pair descriptions; every
 *          chunk must lie inside its parent; no two pairs' outputs may overlap
 *   other arguments as for attn_fwd_partial. Rows of a parent outside a pair's chunks
 *   may hold anything, NaN and Inf included (uninitialised memory, or a copy still in
 *   flight): a pair reads them into its last tiles but they never reach its result
 *   (keys there are masked, their value rows are zeroed on chip before P.V, and query
 *   rows there are not stored).
 */
attn_status_t attn_fwd_partial_batch(const void* q, const void* k, const void* v, int B,
                                     int Hq, int Hkv, int64_t q_ld, int64_t kv_ld, int d,
                                     int causal, float scale, const attn_pair_t* pairs,
                                     int n_pairs, int accumulate, void* stream);

/*
 * attn_merge - combine partial results computed over disjoint key sets
 * (ATTENTION2D, section 3: fragment-local statistics normalised and summed in
 * stages; section 2: the combination is commutative and associative, so no
 * approximation enters). Per row, with M = max_i LSE_i and w_i = exp(LSE_i - M):
 *     O = sum_i w_i O_i / sum_i w_i,   LSE = M + ln(sum_i w_i).
 * Parts with LSE = -inf contribute nothing; if all are -inf, O = 0, LSE = -inf.
 * n_parts = 1 copies. The result does not depend on the order of the parts beyond
 * fp32 rounding.
 *
 *   o_parts, lse_parts  HOST arrays of n_parts DEVICE pointers: fp32 [rows][d]
 *                       (32-byte aligned: rows move as 256-bit loads) and fp32
 *                       [rows] (4-byte aligned)
 *   n_parts             1 .. ATTN_MAX_MERGE_PARTS
 *   o, lse              device, fp32 [rows][d] (32-byte aligned) and [rows]
 *                       (written); must not overlap any part
 *   rows >= 1; d in {64, 128}
 */
attn_status_t attn_merge(const float* const* o_parts, const float* const* lse_parts,
                         int n_parts, float* o, float* lse, int64_t rows, int d,
                         void* stream);

/*
 * attn_ring_fwd_host - Ring Attention's schedule on one GPU, from HOST buffers to
 * HOST buffers ("Ring Attention with Blockwise Parallel Transformers", section 3:
 * the sequence is cut into blocks; at ring step s the holder of query block i
 * attends key/value block (i - s) mod n_chunks, and its partial results are
 * combined). The sequence is cut into n_chunks chunks of C = N / n_chunks rows;
 * query chunk i attends, in ring order, every key/value chunk (under the causal
 * mask only chunks 0..i); each pair is one partial (attn_fwd_partial_batch
 * launches) and a query chunk's partials are combined in ring order with
 * attn_merge. Results equal those of the same calls made on device buffers.
 *
 * The copies are pipelined with the compute: the chunks of q, k, v go to the device
 * on h2d_stream as strided copies (causal: Q_0, K_0 V_0, Q_1, K_1 V_1, ...; else all
 * of K, V first, then Q_0, Q_1, ...), every pair is launched as soon as both of its
 * chunks are in, and a query chunk's merged result goes back on d2h_stream as soon
 * as it is final. The call is asynchronous like the others; the work is ordered
 * after earlier work on `stream`, and later work on `stream` waits for all of it,
 * including the last copy back.
 *
 *   q_h, k_h, v_h   HOST, bf16 [B][Hq][N][d], [B][Hkv][N][d]; page-locked memory
 *                   lets the copies overlap (pageable memory works, unoverlapped)
 *   o_h, lse_h      HOST, fp32 chunk-major [n_chunks][B][Hq][C][d] and
 *                   [n_chunks][B][Hq][C] (written)
 *   q_d, k_d, v_d   DEVICE staging, same shapes as q_h, k_h, v_h (16-byte aligned);
 *                   their contents on entry do not matter (a pair may run before the
 *                   neighbouring chunk has arrived; see attn_fwd_partial_batch)
 *   o_d, lse_d      DEVICE, same shapes as o_h, lse_h (o_d 32-byte aligned)
 *   ws_o, ws_lse    DEVICE partial buffers, ws_slots slots of [B][Hq][C][d] and
 *                   [B][Hq][C] (ws_o 32-byte aligned); ws_slots must be at least
 *                   the number of chunks a query chunk visits when that is more than
 *                   one (n_chunks), else 0 and the pointers may be NULL
 *   n_chunks        1 .. ATTN_MAX_BATCH_PAIRS, dividing N
 *   h2d_stream, d2h_stream  streams for the two copy directions (NULL: `stream`)
 *   other arguments as for attn_fwd. Device buffers must not overlap each other.
 * The host buffers are read and written by copies that run after the call returns:
 * they must stay allocated (and q_h, k_h, v_h unchanged) until `stream` has passed
 * this call's work.
 */
attn_status_t attn_ring_fwd_host(const void* q_h, const void* k_h, const void* v_h,
                                 float* o_h, float* lse_h, void* q_d, void* k_d, void* v_d,
                                 float* o_d, float* lse_d, float* ws_o, float* ws_lse,
                                 int ws_slots, int B, int Hq, int Hkv, int64_t N, int d,
                                 int n_chunks, int causal, float scale, void* stream,
                                 void* h2d_stream, void* d2h_stream);

/*
 * attn_ring_fwd_host_noalloc - attn_ring_fwd_host for callers that cannot allocate
 * device memory. The pages have no counterpart of this call: it exists for programs in
 * which cudaMalloc is not an option, for example code in a process whose device memory
 * belongs to another allocator (a framework's caching allocator, a fixed per-component
 * budget), or code on a latency-critical path where an allocation would synchronise the
 * device. It takes the same host inputs and outputs as attn_ring_fwd_host and runs the
 * same kernels in the same order (results are identical), but its device staging
 * buffers and partial slots live in one fixed array of the library's own device data:
 * it calls no cudaMalloc, cudaFree or other allocating routine.
 *
 * The array holds ATTN_NOALLOC_SCRATCH_BYTES bytes, and every GPU on which the library
 * is loaded keeps it until the process exits. A call needs, each piece rounded up to
 * 256 bytes, with C = N / n_chunks and S = n_chunks if n_chunks > 1, else 0:
 *     B*Hq*N*d*2 + 2 * B*Hkv*N*d*2 + B*Hq*N*d*4 + B*Hq*N*4 + S*B*Hq*C*d*4 + S*B*Hq*C*4
 * bytes; a call that needs more returns ATTN_ERR_UNSUPPORTED before touching the
 * device. Invalid arguments give ATTN_ERR_INVALID_ARG as for attn_ring_fwd_host.
 *
 * The first call on a device, with that device current, looks up the array's device
 * address (once per device); make that first call before any stream capture. Every
 * call shares the array, which keeps what the last call left in it; no part of it
 * needs to start at zero, since a call writes every byte it uses before reading it.
 * Calls whose work overlaps on the GPU race on the array: issue them on one stream
 * (later calls on a stream wait for all the work of earlier ones, copies back
 * included) or otherwise order them.
 *
 *   q_h, k_h, v_h, o_h, lse_h, B, Hq, Hkv, N, d, n_chunks, causal, scale, stream,
 *   h2d_stream, d2h_stream: as for attn_ring_fwd_host
 */
#define ATTN_NOALLOC_SCRATCH_BYTES (64ull * 1024ull * 1024ull)
attn_status_t attn_ring_fwd_host_noalloc(const void* q_h, const void* k_h, const void* v_h,
                                         float* o_h, float* lse_h, int B, int Hq, int Hkv,
                                         int64_t N, int d, int n_chunks, int causal,
                                         float scale, void* stream, void* h2d_stream,
                                         void* d2h_stream);

/*
 * Serving operators: what a decoder layer does around its attention when it answers
 * requests token by token over a paged cache. The pages have no counterpart of these
 * calls. `lens`, `table`, `slots`, ... are int32 device arrays, so that no call needs the
 * host to know a request's length; values in them that make no sense (a page or slot
 * outside the cache, a length beyond the table) never lead to an access out of bounds:
 * each call states what it does with them.
 *
 * The 4-bit cache. Keys and values of one token and key/value head are stored in groups of
 * 32 values: zero = min (+0 for -0), scale = bf16((max - min) / 15), code =
 * rint((x - zero) / scale) (differences in fp32, quotients correctly rounded, ties to the
 * even code; 0 where the scale is 0), value = code * scale + zero; 4 bits a code and a bf16
 * scale and zero point a group, 5 bits a value. Inputs must be finite and at most 2^126 in
 * magnitude; a group with other values reads back as unspecified values, its neighbours
 * are not affected. The cache is one buffer of
 *     n_pages * Hkv * page_size / 16 * 20 * d  bytes, 16-byte aligned:
 * [page][kv head][block of 16 tokens], a block of 20 d bytes holding, in 32-bit words,
 *     [0, 2d)       key codes, eight to a word, the first in the low bits; word
 *                   (r, g, t, i) (d = 64: (g, t, r, i)), r < 2, g < 8, t < 4, i < d / 32:
 *                   token 8r + g, values 32 i + 8 t + (0..7)
 *     [2d, 4d)      value codes; word (h, g, t, b, a), h < d / 64, g < 8, t < 4, b, a < 2:
 *                   token 8b + 2t + a, values 64 h + 8 (0..7) + g
 *     [4d, 4.5d)    key parameters [token][group]: scale in the low 16 bits, zero point high
 *     [4.5d, 5d)    value parameters, likewise
 * (the order in which a warp feeds the codes to the tensor core). page_size is a multiple
 * of 16; slot s of the cache is row s % page_size of page s / page_size; n_pages *
 * page_size must fit 31 bits. d is 64 or 128. Pages need no initialisation.
 */

/*
 * attn_kv_plan - pages and slots for the tokens that a batch of requests is about to add:
 * request b holds lens[b] tokens in its pages table[b][0 .. ceil(lens[b] / page_size)) and
 * adds new_lens[b]. The pages it lacks are taken from the free list, in request order:
 * free_pages[free_head ..). Then
 *     positions[b][i] = lens[b] + i (modulo 2^32)                     for every i < n_new
 *     slots[b][i]     = table[b][pos / page_size] * page_size + pos % page_size
 *                                                  for i < new_lens[b], else -1
 *     lens_out[b] = lens[b] + new_lens[b],  head_out[0] = free_head[0] + pages taken.
 * A request is not served (served[b] = 0, its slots -1, lens_out[b] = lens[b], no page
 * taken) if its length, new_lens[b] < 0 or > n_new make no sense, if it would need more
 * than `width` pages, or if the free list ends before its last page (requests behind it
 * that need pages are then not served either). A held page that is negative in the table,
 * or a slot beyond 31 bits, gives slot -1.
 *
 *   table       [B][width], entries of new pages written, all others left as they were
 *   free_pages  [n_free] page numbers (n_free >= 0; NULL is refused even then)
 *   slots, positions [B][n_new]; lens_out, served [B]; free_head, head_out [1]
 * Outputs must not overlap each other or an input: the call may be repeated on the same
 * inputs with the same result.
 */
attn_status_t attn_kv_plan(const int32_t* lens, const int32_t* new_lens, int32_t* table,
                           const int32_t* free_pages, const int32_t* free_head, int32_t* slots,
                           int32_t* positions, int32_t* lens_out, int32_t* head_out,
                           int32_t* served, int B, int n_new, int width, int page_size,
                           int n_free, void* stream);

/*
 * attn_qk_norm_rope - norms of queries and keys for each head with the position rotation
 * in the same pass, from the packed projection to the head-major tensors the attention
 * calls take. Per query or key head row x: y = x * rsqrt(mean(x^2) + eps) * w, then the
 * pairs (y[j], y[j + n_freq]) (interleaved = 0) or (y[2j], y[2j + 1]) (interleaved = 1),
 * j < n_freq, turn by the angle positions[b][i] * inv_freq[j]; values from 2 n_freq on
 * stay. Value heads are copied. fp32 throughout (angles in fp64), rounded to bf16 once;
 * values of query and key rows below 2^60 in magnitude (their squares are summed in fp32).
 *
 *   qkv        device, bf16; row (b, i) at qkv + b * stride_b + i * stride_n (elements,
 *              multiples of 8) holds Hq query, Hkv key and Hkv value heads of d values;
 *              16-byte aligned
 *   wq, wk     device, [d] bf16 (w_fp32 = 0) or fp32 (w_fp32 = 1)
 *   inv_freq   device, fp32 [n_freq], n_freq a multiple of 8, 2 n_freq <= d
 *   positions  device, int32 [B][N]
 *   q, k, v    device, bf16 [B][Hq][N][d], [B][Hkv][N][d], 16-byte aligned (written)
 */
attn_status_t attn_qk_norm_rope(const void* qkv, int64_t stride_b, int64_t stride_n,
                                const void* wq, const void* wk, int w_fp32,
                                const float* inv_freq, int n_freq, const int32_t* positions,
                                void* q, void* k, void* v, int B, int N, int Hq, int Hkv, int d,
                                float eps, int interleaved, void* stream);

/*
 * attn_kv4_append - tokens into the 4-bit cache: row (b, i) of k and v (bf16
 * [B][Hkv][N][d], 16-byte aligned) goes to slot slots[b][i]. A slot that is negative or
 * outside the cache skips its row; everything else in the cache stays as it was. The slots
 * of one call must differ from each other.
 */
attn_status_t attn_kv4_append(const void* k, const void* v, void* cache, const int32_t* slots,
                              int B, int Hkv, int N, int d, int page_size, int n_pages,
                              void* stream);

/*
 * attn_kv4_read - tokens [start[b], start[b] + N) of each request out of the 4-bit cache,
 * as the bf16 tensors the attention calls take (k, v [B][Hkv][N][d], 16-byte aligned,
 * written; values in fp32, then rounded to bf16). Rows at or past lens[b], rows on a page outside
 * the cache or the table, and all rows of a request with a negative start are zero.
 */
attn_status_t attn_kv4_read(const void* cache, const int32_t* table, const int32_t* start,
                            const int32_t* lens, void* k, void* v, int B, int Hkv, int N, int d,
                            int page_size, int n_pages, int width, void* stream);

/*
 * attn_kv4_fwd - attention of the newest tokens over the 4-bit cache. Query token i of
 * request b has position p = q_pos[b] + i (q_pos NULL: lens[b] - Nq + i) and sees the
 * cached tokens j < lens[b] with j <= p and, when window > 0, (j > p - window or
 * j < sinks). Returns O and LSE as the other attention calls do (attn_merge joins them
 * with partials over other keys); rows that see no key give O = 0, LSE = -inf. What a token
 * that a row does not see holds in the cache, or whether it was ever written, does not
 * reach that row.
 *
 *   q        device, bf16 [B][Hq][Nq][d], 16-byte aligned
 *   table    device, int32 [B][width]; tokens on a page outside the cache are not seen
 *   lens     device, int32 [B]; a negative length counts as 0, one beyond the table
 *            (width * page_size) as the table's end
 *   q_pos    device, int32 [B], or NULL. Needed where the requests of a call add different
 *            numbers of tokens: their first new positions, the lengths before attn_kv_plan
 *            (rows behind a request's new tokens are padding)
 *   o        device, [B][Hq][Nq][d], fp32 (o_bf16 = 0) or bf16 (o_bf16 = 1), 16-byte aligned
 *   lse      device, fp32 [B][Hq][Nq]
 *   max_len  the longest request's length as far as the caller knows (0: unknown, the
 *            table's width counts). It guides how the work is split, never the result's
 *            definition.
 *   window   0 (none) or the window's length; sinks >= 0 counts only with a window
 *   scale    finite, > 0
 *   workspace  device, 16-byte aligned, at least attn_kv4_fwd_workspace(...) bytes (some 1 to
 *            6 MB, and 1 to 4 KB for each request, key/value head and tile of up to 8 rows,
 *            a row being a head of the group at a position). Its contents on entry do not
 *            matter, and nothing in it is kept. Calls whose work may overlap on the GPU need
 *            workspaces of their own.
 * Query rows, the scale, and their product may be of any size below 2^112 (the scale's factor
 * leaves fp32 beyond). Cached values may be up to 2^24 in magnitude, and the scales of the
 * values' groups 2^-40 or more (a group of values with a smaller one counts as its zero
 * point, about). The same inputs give the same bits.
 * The cache is read and unpacked once for every 4 (up to 4 rows a key/value head) or 8 rows, so
 * a long chunk over a cached history is better served by attn_kv4_read and a bf16 call,
 * merged with the chunk's own: over 32 768 tokens of one request, 32 heads on 8, d = 128, 64
 * query tokens take 414 us here and 513 us by attn_kv4_read and attn_fwd_partial, 128 tokens
 * 805 and 514 us, one token 29 and 513 us.
 */
attn_status_t attn_kv4_fwd(const void* q, const void* cache, const int32_t* table,
                           const int32_t* lens, const int32_t* q_pos, void* o, float* lse,
                           int o_bf16, int B, int Hq, int Hkv, int Nq, int d, int page_size,
                           int n_pages, int width, int64_t max_len, int window, int sinks,
                           float scale, void* workspace, int64_t workspace_bytes,
                           void* stream);

/* Bytes of workspace that attn_kv4_fwd needs for these sizes (0: sizes it would refuse). */
int64_t attn_kv4_fwd_workspace(int B, int Hq, int Hkv, int Nq, int d);

/*
 * attn_window_fwd - attention with a sliding window and a few first tokens that stay
 * visible: query row i (position q_off + i) sees key row j (position kv_off + j) when
 *     kv_off + j <= q_off + i  and  (kv_off + j > q_off + i - window  or  kv_off + j < sinks).
 * The work grows with window + sinks, not with the sequence. The chunk arguments are those
 * of attn_fwd_partial, so a prompt can run in pieces (q_off = kv_off + Nkv - Nq for the
 * newest Nq rows), down to single tokens, and results over disjoint key chunks merge with
 * attn_merge. Rows that see no key give O = 0, LSE = -inf.
 *
 *   q        device, bf16 parent [B][Hq][q_ld][d], rows [0, Nq) of it
 *   k, v     device, bf16 parents [B][Hkv][kv_ld][d], rows [0, Nkv): rows beyond are never
 *            read; rows within must be finite, also where no query row sees them (unlike
 *            attn_kv4_fwd's tokens: a row not seen enters products with weight 0)
 *   o        device, dense [B][Hq][Nq][d], fp32 (o_bf16 = 0) or bf16 (o_bf16 = 1)
 *   lse      device, fp32 [B][Hq][Nq]
 *   window >= 1, sinks >= 0; scale finite, > 0; d in {64, 128}
 *   workspace  device, 16-byte aligned, at least attn_window_fwd_workspace(...) bytes: a
 *            call of few query rows splits its keys and joins the parts there. May be NULL
 *            where that is 0. Its contents on entry do not matter, and nothing in it is
 *            kept; calls whose work may overlap on the GPU need workspaces of their own.
 * Sums and softmax statistics are fp32. The weights of V's rows are bf16 numbers: one each
 * (2^-8 of a weight) on 128-row tiles, as in attn_fwd, and the sum of two (2^-15 of it)
 * where few query rows take the form that needs a workspace.
 */
attn_status_t attn_window_fwd(const void* q, const void* k, const void* v, void* o, float* lse,
                              int o_bf16, int B, int Hq, int Hkv, int64_t Nq, int64_t Nkv,
                              int64_t q_ld, int64_t kv_ld, int64_t q_off, int64_t kv_off, int d,
                              int window, int sinks, float scale, void* workspace,
                              int64_t workspace_bytes, void* stream);

/* Bytes of workspace that attn_window_fwd needs for these sizes (0: none, or sizes it would
 * refuse). */
int64_t attn_window_fwd_workspace(int B, int Hq, int Hkv, int64_t Nq, int d);

/*
 * attn_device_status - synchronise `stream` and report whether any kernel of this
 * library on the current device recorded a device-side failure since the last
 * reset (ATTN_ERR_TIMEOUT: a bounded wait ran out; the kernel then stopped its
 * work and returned, leaving its outputs unspecified). reset != 0 clears the
 * record. Returns ATTN_ERR_CUDA if synchronising fails.
 */
attn_status_t attn_device_status(void* stream, int reset);

/*
 * attn_debug_inject - host-side fault injection for tests of error paths: the next
 * `count` calls of an entry point that launches work return `status`
 * (which must be a failure code) after argument checks and before any launch.
 * count = 0 disarms. Not thread-safe; for tests only.
 */
attn_status_t attn_debug_inject(int status, int count);

/*
 * attn_debug_wait_timeout - failure-path check for tests: launches one tiny kernel
 * whose single waiting thread waits, through the same bounded mbarrier wait the
 * attention kernel uses, on a barrier that nothing arrives on, with a limit of
 * limit_cycles SM clock cycles at the device's peak clock (1 .. 2^31; converted to
 * wall-clock time, as the kernels' own limit is). The wait runs out, the kernel
 * records ATTN_ERR_TIMEOUT in the device status word (see attn_device_status) and
 * returns; the device stays usable. Nothing traps or faults.
 */
attn_status_t attn_debug_wait_timeout(int64_t limit_cycles, void* stream);

/*
 * attn_debug_exp2 - check of the two exponentials the softmax uses, for tests:
 * y[i] = 2^x[i] through the FMA-pipe polynomial (use_poly = 1: Cody and Waite's
 * reduction to x = n + f, |f| <= 1/2, and a degree-3 minimax polynomial for 2^f, max
 * relative error 7.5e-5 for -125.5 <= x <= 127; just above -126 the result can come
 * out denormal, off by at most 2^-138 in absolute terms) or through the exp unit's
 * ex2.approx (use_poly = 0). The polynomial clamps x below at -126 (it gives at most
 * 2^-125 there, not 0). x, y: device fp32 arrays of n >= 1 values, not overlapping.
 */
attn_status_t attn_debug_exp2(const float* x, float* y, int64_t n, int use_poly, void* stream);

/* Number of CUDA kernels this library has launched in this process (all devices). */
uint64_t attn_launch_count(void);

#ifdef __cplusplus
}
#endif

#endif /* ATTN_H */
