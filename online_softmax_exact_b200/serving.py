"""Serving operators: pages and slots, normed and rotated heads, the paged 4-bit cache and
attention over it, and attention with a sliding window.

Thin bindings over the entry points of the same names in ``include/attn.h``: they check and
marshal torch tensors, allocate the outputs that are not given, and launch on the tensors'
device and its current stream (or ``stream``). One decoder layer's step over a batch of
requests reads::

    slots, pos, lens, head, served = attn_kv_plan(lens, new_lens, table, free, head,
                                                  page_size=cache.shape[2] * 16, n_new=N)
    q, k, v = attn_qk_norm_rope(qkv, wq, wk, inv_freq, pos, n_heads=Hq, n_kv_heads=Hkv)
    attn_kv4_append(k, v, cache, slots)
    o, lse = attn_kv4_fwd(q, cache, table, lens)            # or, for a whole prompt,
    o, lse = attn_window_fwd(q, k, v, window=W, sinks=S)    # on the bf16 tensors
"""

from __future__ import annotations

import torch

from . import _check, _stream_handle, lib

__all__ = ["kv4_cache", "attn_kv_plan", "attn_qk_norm_rope", "attn_kv4_append", "attn_kv4_read",
           "attn_kv4_fwd", "attn_window_fwd"]

_BF16, _F32, _I32, _U8 = torch.bfloat16, torch.float32, torch.int32, torch.uint8


def _arg(t, dtype, shape, name: str, device: torch.device) -> int:
    """The address of a contiguous tensor of this type, shape and device."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if t.device != device:
        raise ValueError(f"{name} must be on {device}, got {t.device}")
    return t.data_ptr()


def _lead(t, dtype, dims: int, name: str) -> torch.device:
    """The device of the tensor whose shape the others follow."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if t.dim() != dims:
        raise ValueError(f"{name} must have {dims} dimensions, got {list(t.shape)}")
    if t.numel() == 0:
        raise ValueError(f"{name} must not be empty, got {list(t.shape)}")
    return t.device


def _out(t, shape, dtype, device: torch.device, name: str) -> torch.Tensor:
    if t is None:
        return torch.empty(shape, dtype=dtype, device=device)
    _arg(t, dtype, torch.Size(shape), name, device)
    return t


def _raw_stream(device: torch.device, stream, tensors) -> int:
    """The handle of ``stream``, or of the device's current stream. Tensors used on a stream
    other than the current one are recorded there, so that their memory is not reused too
    early."""
    here = torch._C._cuda_getCurrentRawStream(device.index)
    if stream is None:
        return here
    handle = _stream_handle(device, stream)
    if handle != here and isinstance(stream, torch.cuda.Stream):
        for t in tensors:
            if t is not None:
                t.record_stream(stream)
    return handle


def _launch(entry: str, device: torch.device, stream, tensors, *args) -> None:
    """Call the entry point on the stream with ``device`` current."""
    handle = _raw_stream(device, stream, tensors)
    if device.index == torch.cuda.current_device():
        st = getattr(lib(), entry)(*args, handle)
    else:
        with torch.cuda.device(device):
            st = getattr(lib(), entry)(*args, handle)
    if st:
        _check(st, entry)


def kv4_cache(n_pages: int, n_kv_heads: int, d: int, *, page_size: int = 64,
              device=None) -> torch.Tensor:
    """An uninitialised paged 4-bit cache: uint8 [n_pages, n_kv_heads, page_size / 16, 20 d]
    (layout in attn.h)."""
    if n_pages < 1 or n_kv_heads < 1 or d not in (64, 128) or page_size < 16 or page_size % 16:
        raise ValueError("need n_pages, n_kv_heads >= 1, d 64 or 128, page_size a multiple of 16")
    return torch.empty((n_pages, n_kv_heads, page_size // 16, 20 * d), dtype=_U8,
                       device=device if device is not None else "cuda")


def _cache_dims(cache, device: torch.device):
    """(address, n_pages, Hkv, page_size, d) of a cache tensor."""
    if not isinstance(cache, torch.Tensor) or not cache.is_cuda:
        raise ValueError("cache must be a CUDA tensor")
    if cache.dtype != _U8 or cache.dim() != 4 or cache.shape[3] not in (1280, 2560):
        raise ValueError("cache must be uint8 [n_pages, Hkv, page_size / 16, 20 d], d 64 or 128")
    if not cache.is_contiguous() or cache.numel() == 0:
        raise ValueError("cache must be contiguous and not empty")
    if cache.device != device:
        raise ValueError(f"cache must be on {device}, got {cache.device}")
    n_pages, Hkv, blocks, width = cache.shape
    return cache.data_ptr(), n_pages, Hkv, blocks * 16, width // 20


def attn_kv_plan(lens: torch.Tensor, new_lens: torch.Tensor, table: torch.Tensor,
                 free_pages: torch.Tensor, free_head: torch.Tensor, *, page_size: int,
                 n_new: int, stream=None):
    """Pages and slots for new_lens[b] <= n_new tokens of each request that holds lens[b]
    tokens. lens, new_lens int32 [B]; table int32 [B, width], new pages entered in place;
    free_pages int32 [F], taken from free_head (int32 [1]) on. Returns (slots [B, n_new],
    positions [B, n_new], lens [B], free_head [1], served [B]), all int32: slots are -1
    behind a request's tokens and where it was not served (served 0, length unchanged)."""
    dev = _lead(lens, _I32, 1, "lens")
    B = lens.shape[0]
    if _lead(table, _I32, 2, "table") != dev or table.shape[0] != B:
        raise ValueError(f"table must be [{B}, width] on {dev}")
    if not isinstance(free_pages, torch.Tensor) or free_pages.dim() != 1:
        raise ValueError("free_pages must be one-dimensional")
    if n_new < 1 or page_size < 1:
        raise ValueError("need n_new >= 1 and page_size >= 1")
    lens_p = _arg(lens, _I32, lens.shape, "lens", dev)
    new_p = _arg(new_lens, _I32, lens.shape, "new_lens", dev)
    table_p = _arg(table, _I32, table.shape, "table", dev)
    free_p = _arg(free_pages, _I32, free_pages.shape, "free_pages", dev)
    head_p = _arg(free_head, _I32, torch.Size((1,)), "free_head", dev)
    n_free = free_pages.shape[0]
    # one allocation for the five outputs
    buf = torch.empty(2 * B * n_new + 2 * B + 1, dtype=_I32, device=dev)
    slots, pos, lens_out, served, head_out = buf.split((B * n_new, B * n_new, B, B, 1))
    at, n4 = buf.data_ptr(), 4 * B * n_new
    _launch("attn_kv_plan", dev, stream, (lens, new_lens, table, free_pages, free_head, buf),
            lens_p, new_p, table_p, free_p or lens_p, head_p, at, at + n4, at + 2 * n4,
            at + 2 * n4 + 8 * B, at + 2 * n4 + 4 * B, B, n_new, table.shape[1], page_size, n_free)
    return slots.view(B, n_new), pos.view(B, n_new), lens_out, head_out, served


def attn_qk_norm_rope(qkv: torch.Tensor, wq: torch.Tensor, wk: torch.Tensor,
                      inv_freq: torch.Tensor, positions: torch.Tensor, *, n_heads: int,
                      n_kv_heads: int, eps: float = 1e-6, interleaved: bool = False,
                      q: torch.Tensor | None = None, k: torch.Tensor | None = None,
                      v: torch.Tensor | None = None, stream=None):
    """Per-head RMS norms of queries and keys and their rotation, in one pass.
    qkv bf16 [B, N, (n_heads + 2 n_kv_heads) d] (its rows may be strided); wq, wk [d] bf16
    or fp32; inv_freq fp32 [r / 2] for the first r values of a head; positions int32
    [B, N]. Returns bf16 (q [B, n_heads, N, d], k, v [B, n_kv_heads, N, d])."""
    dev = _lead(qkv, _BF16, 3, "qkv")
    B, N, width = qkv.shape
    if n_heads < 1 or n_kv_heads < 1:
        raise ValueError("need n_heads, n_kv_heads >= 1")
    H = n_heads + 2 * n_kv_heads
    d = width // H
    if width != H * d or d not in (64, 128):
        raise ValueError("qkv's last dimension must be (n_heads + 2 n_kv_heads) d, d 64 or 128")
    if qkv.stride(2) != 1:
        raise ValueError("qkv's last dimension must be contiguous")
    if not isinstance(wq, torch.Tensor) or wq.dtype not in (_BF16, _F32):
        raise ValueError("wq and wk must be bf16 or fp32 tensors")
    if not isinstance(inv_freq, torch.Tensor) or inv_freq.dim() != 1 or \
            not 0 < 2 * inv_freq.shape[0] <= d:
        raise ValueError("inv_freq must be fp32 [r / 2] with 0 < r <= d")
    size = torch.Size((d,))
    wq_p, wk_p = _arg(wq, wq.dtype, size, "wq", dev), _arg(wk, wq.dtype, size, "wk", dev)
    f_p = _arg(inv_freq, _F32, inv_freq.shape, "inv_freq", dev)
    p_p = _arg(positions, _I32, torch.Size((B, N)), "positions", dev)
    q = _out(q, (B, n_heads, N, d), _BF16, dev, "q")
    k = _out(k, (B, n_kv_heads, N, d), _BF16, dev, "k")
    v = _out(v, (B, n_kv_heads, N, d), _BF16, dev, "v")
    # the stride of a dimension of one row is never used
    _launch("attn_qk_norm_rope", dev, stream, (qkv, wq, wk, inv_freq, positions, q, k, v),
            qkv.data_ptr(), qkv.stride(0) if B > 1 else 0, qkv.stride(1) if N > 1 else 0,
            wq_p, wk_p, int(wq.dtype == _F32), f_p, inv_freq.shape[0], p_p, q.data_ptr(),
            k.data_ptr(), v.data_ptr(), B, N, n_heads, n_kv_heads, d, float(eps),
            int(bool(interleaved)))
    return q, k, v


def attn_kv4_append(k: torch.Tensor, v: torch.Tensor, cache: torch.Tensor, slots: torch.Tensor, *,
                    stream=None) -> None:
    """Tokens into the 4-bit cache: k, v bf16 [B, Hkv, N, d], slots int32 [B, N] (distinct;
    a negative slot, or one outside the cache, skips its token)."""
    dev = _lead(k, _BF16, 4, "k")
    c_p, n_pages, Hkv, page, d = _cache_dims(cache, dev)
    B, N = k.shape[0], k.shape[2]
    if k.shape[1] != Hkv or k.shape[3] != d:
        raise ValueError(f"k must be [B, {Hkv}, N, {d}] as the cache is, got {list(k.shape)}")
    _launch("attn_kv4_append", dev, stream, (k, v, cache, slots),
            _arg(k, _BF16, k.shape, "k", dev), _arg(v, _BF16, k.shape, "v", dev), c_p,
            _arg(slots, _I32, torch.Size((B, N)), "slots", dev), B, Hkv, N, d, page, n_pages)


def attn_kv4_read(cache: torch.Tensor, table: torch.Tensor, start: torch.Tensor,
                  lens: torch.Tensor, *, n: int, k: torch.Tensor | None = None,
                  v: torch.Tensor | None = None, stream=None):
    """Tokens [start[b], start[b] + n) of each request out of the 4-bit cache, as bf16
    (k, v [B, Hkv, n, d]); zeros at and past lens[b]."""
    dev = _lead(table, _I32, 2, "table")
    c_p, n_pages, Hkv, page, d = _cache_dims(cache, dev)
    B, width = table.shape
    if n < 1:
        raise ValueError("need n >= 1")
    k = _out(k, (B, Hkv, n, d), _BF16, dev, "k")
    v = _out(v, (B, Hkv, n, d), _BF16, dev, "v")
    size = torch.Size((B,))
    _launch("attn_kv4_read", dev, stream, (cache, table, start, lens, k, v), c_p,
            _arg(table, _I32, table.shape, "table", dev), _arg(start, _I32, size, "start", dev),
            _arg(lens, _I32, size, "lens", dev), k.data_ptr(), v.data_ptr(), B, Hkv, n, d, page,
            n_pages, width)
    return k, v


def _o_type(o_dtype) -> int:
    if o_dtype not in (_F32, _BF16):
        raise ValueError("o_dtype must be torch.float32 or torch.bfloat16")
    return int(o_dtype == _BF16)


def attn_kv4_fwd(q: torch.Tensor, cache: torch.Tensor, table: torch.Tensor, lens: torch.Tensor, *,
                 q_pos: torch.Tensor | None = None, window: int = 0, sinks: int = 0,
                 scale: float | None = None, max_len: int = 0, o_dtype: torch.dtype = _F32,
                 o: torch.Tensor | None = None, lse: torch.Tensor | None = None, stream=None):
    """Attention of each request's newest tokens over the 4-bit cache. q bf16
    [B, Hq, Nq, d]; table int32 [B, width]; lens int32 [B], the tokens cached (the queries'
    own among them). Query i has position lens[b] - Nq + i, or q_pos[b] + i (int32 [B]); with a window it sees
    the last ``window`` positions and the first ``sinks``. ``max_len``: the longest length,
    if the host knows it (a hint). Returns (O [B, Hq, Nq, d] of o_dtype, LSE fp32)."""
    dev = _lead(q, _BF16, 4, "q")
    c_p, n_pages, Hkv, page, d = _cache_dims(cache, dev)
    B, Hq, Nq, dq = q.shape
    if dq != d or Hq % Hkv:
        raise ValueError(f"q must be [B, Hq, Nq, {d}] with Hq a multiple of {Hkv}, "
                         f"got {list(q.shape)}")
    if _lead(table, _I32, 2, "table") != dev or table.shape[0] != B:
        raise ValueError(f"table must be [{B}, width] on {dev}")
    bf16 = _o_type(o_dtype if o is None else o.dtype)
    o = _out(o, (B, Hq, Nq, d), _BF16 if bf16 else _F32, dev, "o")
    lse = _out(lse, (B, Hq, Nq), _F32, dev, "lse")
    size = torch.Size((B,))
    n_ws = lib().attn_kv4_fwd_workspace(B, Hq, Hkv, Nq, d)
    ws = torch.empty(n_ws, dtype=_U8, device=dev)
    _launch("attn_kv4_fwd", dev, stream, (q, cache, table, lens, q_pos, o, lse, ws),
            _arg(q, _BF16, q.shape, "q", dev), c_p, _arg(table, _I32, table.shape, "table", dev),
            _arg(lens, _I32, size, "lens", dev),
            None if q_pos is None else _arg(q_pos, _I32, size, "q_pos", dev), o.data_ptr(),
            lse.data_ptr(), bf16, B, Hq, Hkv, Nq, d, page, n_pages, table.shape[1], int(max_len),
            int(window), int(sinks), float(d ** -0.5 if scale is None else scale),
            ws.data_ptr(), n_ws)
    return o, lse


def attn_window_fwd(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, *, window: int,
                    sinks: int = 0, q_off: int | None = None, kv_off: int = 0,
                    kv_len: int | None = None, scale: float | None = None,
                    o_dtype: torch.dtype = _F32, o: torch.Tensor | None = None,
                    lse: torch.Tensor | None = None, stream=None):
    """Attention with a sliding window and sinks. q bf16 [B, Hq, Nq, d]; k, v bf16
    [B, Hkv, L, d], of which the first kv_len rows (default all) hold keys. Row i has
    position q_off + i, key j kv_off + j; q_off defaults to kv_off + kv_len - Nq (the
    queries are the newest rows). A row sees the last ``window`` positions up to its own
    and the first ``sinks``. Returns (O [B, Hq, Nq, d] of o_dtype, LSE fp32)."""
    dev = _lead(q, _BF16, 4, "q")
    B, Hq, Nq, d = q.shape
    if _lead(k, _BF16, 4, "k") != dev or k.shape[0] != B or k.shape[3] != d:
        raise ValueError(f"k and v must be [{B}, Hkv, L, {d}] on {dev}")
    Hkv, L = k.shape[1], k.shape[2]
    n = L if kv_len is None else int(kv_len)
    if not 0 < n <= L:
        raise ValueError(f"kv_len must be in 1..{L}")
    if q_off is None:
        q_off = kv_off + n - Nq
        if q_off < 0:
            raise ValueError("more query rows than key rows: give q_off")
    bf16 = _o_type(o_dtype if o is None else o.dtype)
    o = _out(o, (B, Hq, Nq, d), _BF16 if bf16 else _F32, dev, "o")
    lse = _out(lse, (B, Hq, Nq), _F32, dev, "lse")
    n_ws = lib().attn_window_fwd_workspace(B, Hq, Hkv, Nq, d)
    ws = torch.empty(n_ws, dtype=_U8, device=dev) if n_ws else None
    _launch("attn_window_fwd", dev, stream, (q, k, v, o, lse, ws),
            _arg(q, _BF16, q.shape, "q", dev), _arg(k, _BF16, k.shape, "k", dev),
            _arg(v, _BF16, k.shape, "v", dev), o.data_ptr(), lse.data_ptr(), bf16, B, Hq, Hkv,
            Nq, n, Nq, L, int(q_off), int(kv_off), d, int(window), int(sinks),
            float(d ** -0.5 if scale is None else scale), ws.data_ptr() if n_ws else None, n_ws)
    return o, lse
