"""Serving operators: pages and slots, normed and rotated heads, the paged 4-bit cache and
attention over it, and attention with a sliding window.

Thin bindings over the entry points of the same names in ``include/attn.h``: they check
torch tensors, allocate the outputs that are not given (and workspaces), and launch on the
tensors' device and its current stream (or ``stream``). The marshalling is native
(``csrc/serving_binding.cpp``): a decode step's kernels take microseconds, and so do calls.
``stream`` is a torch stream, or a handle as an integer (given tensors then have to live until
it is done with them); the caller orders it behind the work that makes the inputs. What the
call allocates comes from that stream's memory, never from what the current one still uses.
A whole prompt can run through ``attn_window_fwd(q, k, v, window=W, sinks=S)`` on the bf16
tensors. One decoder layer's step over a batch of requests, of which request b adds
new_lens[b] <= N tokens, the first at position lens[b]::

    slots, pos, grown, head, served = attn_kv_plan(lens, new_lens, table, free, head,
                                                   page_size=cache.shape[2] * 16, n_new=N)
    q, k, v = attn_qk_norm_rope(qkv, wq, wk, inv_freq, pos, n_heads=Hq, n_kv_heads=Hkv)
    attn_kv4_append(k, v, cache, slots)
    o, lse = attn_kv4_fwd(q, cache, table, grown, q_pos=lens)
    lens = grown
"""

from __future__ import annotations

import torch

from ._abi import load_serving as _native

__all__ = ["kv4_cache", "attn_kv_plan", "attn_qk_norm_rope", "attn_kv4_append", "attn_kv4_read",
           "attn_kv4_fwd", "attn_window_fwd"]


def _handle(stream, tensors):
    """The handle of a given stream (an integer is one already, None the current stream).
    Given tensors are recorded on a stream object, so that their memory is not reused too
    early; with an integer they have to live until the stream is done with them. What a
    call allocates comes from its stream's memory, recorded on the caller's stream."""
    if stream is None:
        return None
    if not hasattr(stream, "cuda_stream"):
        return int(stream)
    for t in tensors:
        if isinstance(t, torch.Tensor) and t.is_cuda:
            t.record_stream(stream)
    return int(stream.cuda_stream)


def kv4_cache(n_pages: int, n_kv_heads: int, d: int, *, page_size: int = 64,
              device=None) -> torch.Tensor:
    """An uninitialised paged 4-bit cache: uint8 [n_pages, n_kv_heads, page_size / 16, 20 d]
    (layout in attn.h)."""
    if n_pages < 1 or n_kv_heads < 1 or d not in (64, 128) or page_size < 16 or page_size % 16:
        raise ValueError("need n_pages, n_kv_heads >= 1, d 64 or 128, page_size a multiple of 16")
    return torch.empty((n_pages, n_kv_heads, page_size // 16, 20 * d), dtype=torch.uint8,
                       device=device if device is not None else "cuda")


def attn_kv_plan(lens: torch.Tensor, new_lens: torch.Tensor, table: torch.Tensor,
                 free_pages: torch.Tensor, free_head: torch.Tensor, *, page_size: int,
                 n_new: int, stream=None):
    """Pages and slots for new_lens[b] <= n_new tokens of each request that holds lens[b]
    tokens. lens, new_lens int32 [B]; table int32 [B, width], new pages entered in place;
    free_pages int32 [F], taken from free_head (int32 [1]) on. Returns (slots [B, n_new],
    positions [B, n_new], lens [B], free_head [1], served [B]), all int32: slots are -1
    behind a request's tokens and where it was not served (served 0, length unchanged). The
    five share one allocation: clone what outlives the step by long, or is to be saved."""
    h = _handle(stream, (lens, new_lens, table, free_pages, free_head))
    return _native().kv_plan(lens, new_lens, table, free_pages, free_head, page_size, n_new, h)


def attn_qk_norm_rope(qkv: torch.Tensor, wq: torch.Tensor, wk: torch.Tensor,
                      inv_freq: torch.Tensor, positions: torch.Tensor, *, n_heads: int,
                      n_kv_heads: int, eps: float = 1e-6, interleaved: bool = False,
                      q: torch.Tensor | None = None, k: torch.Tensor | None = None,
                      v: torch.Tensor | None = None, stream=None):
    """Per-head RMS norms of queries and keys and their rotation, in one pass.
    qkv bf16 [B, N, (n_heads + 2 n_kv_heads) d] (its rows may be strided); wq, wk [d] bf16
    or fp32; inv_freq fp32 [r / 2] for the first r values of a head (r / 2 a multiple of 8);
    positions int32 [B, N]. Returns bf16 (q [B, n_heads, N, d], k, v [B, n_kv_heads, N, d])."""
    h = _handle(stream, (qkv, wq, wk, inv_freq, positions, q, k, v))
    return _native().qk_norm_rope(qkv, wq, wk, inv_freq, positions, n_heads, n_kv_heads, eps,
                                  interleaved, q, k, v, h)


def attn_kv4_append(k: torch.Tensor, v: torch.Tensor, cache: torch.Tensor, slots: torch.Tensor, *,
                    stream=None) -> None:
    """Tokens into the 4-bit cache: k, v bf16 [B, Hkv, N, d], slots int32 [B, N] (distinct;
    a negative slot, or one outside the cache, skips its token)."""
    _native().kv4_append(k, v, cache, slots, _handle(stream, (k, v, cache, slots)))


def attn_kv4_read(cache: torch.Tensor, table: torch.Tensor, start: torch.Tensor,
                  lens: torch.Tensor, *, n: int, k: torch.Tensor | None = None,
                  v: torch.Tensor | None = None, stream=None):
    """Tokens [start[b], start[b] + n) of each request out of the 4-bit cache, as bf16
    (k, v [B, Hkv, n, d]); zeros at and past lens[b]. start, lens int32 [B]."""
    h = _handle(stream, (cache, table, start, lens, k, v))
    return _native().kv4_read(cache, table, start, lens, n, k, v, h)


def _is_bf16(o_dtype) -> bool:
    if o_dtype is torch.bfloat16:
        return True
    if o_dtype is torch.float32:
        return False
    raise ValueError("o_dtype must be torch.float32 or torch.bfloat16")


def attn_kv4_fwd(q: torch.Tensor, cache: torch.Tensor, table: torch.Tensor, lens: torch.Tensor, *,
                 q_pos: torch.Tensor | None = None, window: int = 0, sinks: int = 0,
                 scale: float | None = None, max_len: int = 0,
                 o_dtype: torch.dtype = torch.float32, o: torch.Tensor | None = None,
                 lse: torch.Tensor | None = None, stream=None):
    """Attention of each request's newest tokens over the 4-bit cache. q bf16
    [B, Hq, Nq, d]; table int32 [B, width]; lens int32 [B], the tokens cached (the queries'
    own among them). Query i has position lens[b] - Nq + i, or q_pos[b] + i (int32 [B]):
    give q_pos where requests add different numbers of tokens (rows behind them are padding);
    with a window it sees the last ``window`` positions and the first ``sinks``.
    ``max_len``: the longest length, if the host knows it (a hint). Returns
    (O [B, Hq, Nq, d] of o_dtype, LSE fp32 [B, Hq, Nq])."""
    bf16 = _is_bf16(o_dtype)
    if scale is None:
        scale = 1.0 if not isinstance(q, torch.Tensor) or q.dim() != 4 else q.shape[3] ** -0.5
    h = _handle(stream, (q, cache, table, lens, q_pos, o, lse))
    return _native().kv4_fwd(q, cache, table, lens, q_pos, window, sinks, scale, max_len, bf16, o, lse,
                             h)


def attn_window_fwd(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, *, window: int,
                    sinks: int = 0, q_off: int | None = None, kv_off: int = 0,
                    kv_len: int | None = None, scale: float | None = None,
                    o_dtype: torch.dtype = torch.float32, o: torch.Tensor | None = None,
                    lse: torch.Tensor | None = None, stream=None):
    """Attention with a sliding window and sinks. q bf16 [B, Hq, Nq, d]; k, v bf16
    [B, Hkv, L, d], of which the first kv_len rows (default all) hold keys. Row i has
    position q_off + i, key j kv_off + j; q_off defaults to kv_off + kv_len - Nq (the
    queries are the newest rows). A row sees the last ``window`` positions up to its own
    and the first ``sinks``. Key and value rows below kv_len must be finite, also where no
    row sees them (padding included). Returns (O [B, Hq, Nq, d] of o_dtype, LSE fp32 [B, Hq, Nq])."""
    bf16 = _is_bf16(o_dtype)
    if scale is None:
        scale = 1.0 if not isinstance(q, torch.Tensor) or q.dim() != 4 else q.shape[3] ** -0.5
    h = _handle(stream, (q, k, v, o, lse))
    return _native().window_fwd(q, k, v, window, sinks, q_off, kv_off, kv_len, scale, bf16, o, lse, h)
