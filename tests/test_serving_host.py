"""Host-side checks of the serving operators (no GPU needed): the C entry points reject bad
arguments before touching a device, the Python bindings reject tensors that do not fit, and
the references the GPU tests use agree with each other."""

from __future__ import annotations

import numpy as np
import pytest
import torch

import serving_util as su


@pytest.fixture(scope="module")
def lib():
    from online_softmax_exact_b200 import _abi
    from online_softmax_exact_b200 import build as b

    b.build()
    return _abi.load()


G = 1 << 36  # fake device addresses, 64 GiB apart: never dereferenced by the checks


def statuses():
    from online_softmax_exact_b200 import _abi

    return _abi.ATTN_ERR_INVALID_ARG, _abi.ATTN_ERR_UNSUPPORTED


def call(fn, defaults, **kw):
    args = dict(defaults)
    assert set(kw) <= set(args), kw
    args.update(kw)
    return fn(*args.values())


PLAN = dict(lens=G, new=2 * G, table=3 * G, free=4 * G, head=5 * G, slots=6 * G, pos=7 * G,
            lens_out=8 * G, head_out=9 * G, served=10 * G, B=4, n_new=8, width=16, page=16,
            n_free=100, stream=None)
ROPE = dict(qkv=G, stride_b=8 * 4 * 64, stride_n=4 * 64, wq=2 * G, wk=3 * G, w_fp32=0, inv=4 * G,
            n_freq=32, pos=5 * G, q=6 * G, k=7 * G, v=8 * G, B=2, N=8, Hq=2, Hkv=1, d=64, eps=1e-6,
            inter=0, stream=None)
APPEND = dict(k=G, v=2 * G, cache=3 * G, slots=4 * G, B=2, Hkv=2, N=8, d=64, page=16, n_pages=9,
              stream=None)
READ = dict(cache=G, table=2 * G, start=3 * G, lens=4 * G, k=5 * G, v=6 * G, B=2, Hkv=2, N=8, d=64,
            page=16, n_pages=9, width=4, stream=None)
KV4 = dict(q=G, cache=2 * G, table=3 * G, lens=4 * G, q_pos=None, o=5 * G, lse=6 * G, o_bf16=0, B=2,
           Hq=4, Hkv=2, Nq=1, d=64, page=16, n_pages=9, width=4, max_len=0, window=0, sinks=0,
           scale=0.125, ws=8 * G, ws_bytes=1 << 24, stream=None)
WIN = dict(q=G, k=2 * G, v=3 * G, o=4 * G, lse=5 * G, o_bf16=0, B=2, Hq=4, Hkv=2, Nq=8, Nkv=16,
           q_ld=8, kv_ld=16, q_off=8, kv_off=0, d=64, window=4, sinks=1, scale=0.125,
           ws=6 * G, ws_bytes=1 << 24, stream=None)

INVALID = {
    "attn_kv_plan": (PLAN, [
        *({k: None} for k in list(PLAN)[:10]), dict(lens=G + 2), dict(served=10 * G + 1), dict(B=0),
        dict(n_new=0), dict(width=0), dict(page=0), dict(n_free=-1), dict(slots=G), dict(table=2 * G),
        dict(pos=6 * G + 64), dict(lens_out=G), dict(head_out=5 * G), dict(served=4 * G),
        dict(slots=8 * G - 4)]),
    "attn_qk_norm_rope": (ROPE, [
        *({k: None} for k in ("qkv", "wq", "wk", "inv", "pos", "q", "k", "v")), dict(qkv=G + 8),
        dict(q=6 * G + 2), dict(wq=2 * G + 1), dict(w_fp32=1, wk=3 * G + 2), dict(inv=4 * G + 2),
        dict(B=0), dict(N=0), dict(Hq=0), dict(Hkv=0), dict(w_fp32=2), dict(inter=-1),
        dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf")), dict(n_freq=0),
        dict(n_freq=40), dict(stride_n=4 * 64 + 4), dict(stride_n=3 * 64), dict(stride_n=-256),
        dict(stride_b=-8), dict(stride_b=1 << 61), dict(q=G), dict(k=6 * G + 1024), dict(v=5 * G)]),
    "attn_kv4_append": (APPEND, [
        *({k: None} for k in ("k", "v", "cache", "slots")), dict(k=G + 8), dict(cache=3 * G + 8),
        dict(slots=4 * G + 2), dict(B=0), dict(N=0), dict(Hkv=0), dict(page=0), dict(page=24),
        dict(page=-16), dict(n_pages=0), dict(cache=G), dict(cache=4 * G - 1280)]),
    "attn_kv4_read": (READ, [
        *({k: None} for k in ("cache", "table", "start", "lens", "k", "v")), dict(k=5 * G + 8),
        dict(table=2 * G + 1), dict(B=0), dict(N=0), dict(width=0), dict(page=8), dict(n_pages=0),
        dict(k=6 * G), dict(k=G), dict(v=2 * G)]),
    "attn_kv4_fwd": (KV4, [
        *({k: None} for k in ("q", "cache", "table", "lens", "o", "lse", "ws")), dict(q=G + 8),
        dict(ws=8 * G + 8), dict(ws_bytes=1 << 20), dict(ws=G - 4096), dict(ws=5 * G),
        dict(o=5 * G + 4), dict(q_pos=7 * G + 2), dict(B=0), dict(Hq=3), dict(Hkv=0), dict(Nq=0),
        dict(width=0), dict(max_len=-1), dict(o_bf16=2), dict(window=-1), dict(sinks=-1),
        dict(scale=0.0), dict(scale=-1.0), dict(scale=float("nan")), dict(scale=float("inf")),
        dict(page=20), dict(n_pages=0), dict(o=G), dict(lse=5 * G), dict(lse=2 * G),
        dict(q_pos=6 * G)]),
    "attn_window_fwd": (WIN, [
        *({k: None} for k in ("q", "k", "v", "o", "lse")), dict(q=G + 8), dict(o=4 * G + 8),
        dict(lse=5 * G + 2), dict(B=0), dict(Hq=3), dict(Hkv=0), dict(Nq=0), dict(Nkv=0),
        dict(q_ld=7), dict(kv_ld=15), dict(q_off=-1), dict(kv_off=-1), dict(o_bf16=3),
        dict(window=0), dict(window=-4), dict(sinks=-1), dict(scale=0.0), dict(scale=-0.5),
        dict(scale=float("nan")), dict(o=G), dict(lse=4 * G), dict(o=3 * G - 4096), dict(ws=None),
        dict(ws=6 * G + 4), dict(ws_bytes=1 << 16), dict(ws=G), dict(ws=5 * G - 64)]),
}
UNSUPPORTED = {
    "attn_kv_plan": (PLAN, [dict(B=1 << 20, n_new=1 << 12), dict(B=(1 << 30) + 1, n_new=1), dict(width=1 << 20, page=1 << 12)]),
    "attn_qk_norm_rope": (ROPE, [dict(d=96), dict(d=256), dict(n_freq=12), dict(n_freq=4),
                                 dict(B=1 << 16, N=1 << 16), dict(Hq=1 << 21)]),
    "attn_kv4_append": (APPEND, [dict(d=96), dict(page=1 << 20, n_pages=1 << 12),
                                 dict(B=1 << 16, N=1 << 16), dict(N=1 << 29, Hkv=64, n_pages=1)]),
    "attn_kv4_read": (READ, [dict(d=32), dict(page=1 << 20, n_pages=1 << 12),
                             dict(B=1 << 16, N=1 << 16), dict(width=1 << 28),
                             dict(N=1 << 29, Hkv=64, n_pages=1)]),
    "attn_kv4_fwd": (KV4, [dict(d=256), dict(page=1 << 20, n_pages=1 << 12), dict(width=1 << 28),
                           dict(B=1 << 20, Hq=1 << 12), dict(Nq=1 << 30),
                           dict(B=1 << 16, page=1 << 20, n_pages=1, width=1 << 10)]),
    "attn_window_fwd": (WIN, [dict(d=96), dict(Nq=1 << 31, q_ld=1 << 31), dict(kv_ld=1 << 31),
                              dict(q_off=1 << 61), dict(kv_off=1 << 61), dict(B=1 << 20, Hq=1 << 12)]),
}
DEFAULTS = {k: v[0] for k, v in INVALID.items()}


@pytest.mark.parametrize("entry", sorted(INVALID))
def test_invalid_arguments(lib, entry):
    invalid, _ = statuses()
    defaults, cases = INVALID[entry]
    for kw in cases:
        assert call(getattr(lib, entry), defaults, **kw) == invalid, kw


@pytest.mark.parametrize("entry", sorted(UNSUPPORTED))
def test_unsupported_arguments(lib, entry):
    _, unsupported = statuses()
    defaults, cases = UNSUPPORTED[entry]
    for kw in cases:
        # addresses far enough apart for the larger sizes
        wide = {k: v << 8 for k, v in defaults.items() if isinstance(v, int) and v >= G}
        assert call(getattr(lib, entry), {**defaults, **wide}, **kw) == unsupported, kw


def test_kv4_workspace(lib):
    size = lib.attn_kv4_fwd_workspace
    for bad in ((0, 4, 2, 1, 64), (1, 3, 2, 1, 64), (1, 4, 2, 0, 64), (1, 4, 2, 1, 96)):
        assert size(*bad) == 0
    need = size(2, 4, 2, 1, 64)
    invalid, _ = statuses()
    assert call(lib.attn_kv4_fwd, KV4, ws_bytes=need - 1) == invalid
    assert 0 < need < size(2, 4, 2, 1, 128) < size(200, 32, 8, 1, 128) < 1 << 25


def test_window_workspace(lib):
    """Needed for few query rows only; a call without that need takes a null one."""
    size = lib.attn_window_fwd_workspace
    for bad in ((0, 4, 2, 1, 64), (1, 3, 2, 1, 64), (1, 4, 2, 0, 64), (1, 4, 2, 1, 96)):
        assert size(*bad) == 0
    assert 0 < size(1, 4, 2, 1, 64) < size(1, 4, 2, 1, 128) < 1 << 24
    assert size(1, 4, 2, 4096, 128) == 0
    invalid, _ = statuses()
    need = size(2, 4, 2, 8, 64)
    assert call(lib.attn_window_fwd, WIN, ws_bytes=need - 1) == invalid
    assert call(lib.attn_window_fwd, WIN, Nq=300, q_ld=300, ws=None, ws_bytes=0) not in statuses()


@pytest.mark.parametrize("entry", sorted(DEFAULTS))
def test_valid_arguments_reach_the_device(lib, entry):
    """With no GPU, a valid call passes every check and fails at the first CUDA call; an
    injected failure comes before that, and nothing is counted as launched."""
    from online_softmax_exact_b200._abi import ATTN_ERR_CUDA, ATTN_ERR_INJECTED

    if torch.cuda.is_available():
        pytest.skip("checks the no-device path")
    fn, defaults = getattr(lib, entry), DEFAULTS[entry]
    n0 = lib.attn_launch_count()
    assert lib.attn_debug_inject(ATTN_ERR_INJECTED, 1) == 0
    assert call(fn, defaults) == ATTN_ERR_INJECTED
    assert call(fn, defaults) == ATTN_ERR_CUDA
    assert lib.attn_launch_count() == n0


def test_bindings_refuse_host_tensors():
    import online_softmax_exact_b200 as osx

    i = torch.zeros(2, dtype=torch.int32)
    t2 = torch.zeros((2, 3), dtype=torch.int32)
    x = torch.zeros((1, 2, 3, 64), dtype=torch.bfloat16)
    c = torch.zeros((2, 2, 1, 1280), dtype=torch.uint8)
    for fn in (lambda: osx.attn_kv_plan(i, i, t2, i, i[:1], page_size=16, n_new=1),
               lambda: osx.attn_qk_norm_rope(x[0], x[0, 0, 0], x[0, 0, 0], i.float(), t2, n_heads=1,
                                             n_kv_heads=1),
               lambda: osx.attn_kv4_append(x, x, c, t2),
               lambda: osx.attn_kv4_read(c, t2, i, i, n=3),
               lambda: osx.attn_kv4_fwd(x, c, t2, i),
               lambda: osx.attn_window_fwd(x, x, x, window=4)):
        with pytest.raises(ValueError, match="CUDA tensor"):
            fn()
    for bad in (dict(n_pages=0), dict(d=96), dict(page_size=24), dict(n_kv_heads=0)):
        with pytest.raises(ValueError):
            osx.kv4_cache(**{**dict(n_pages=1, n_kv_heads=1, d=64, page_size=16, device="cpu"), **bad})
    assert osx.kv4_cache(3, 2, 128, page_size=48, device="cpu").shape == (3, 2, 3, 2560)


@pytest.mark.parametrize("d", [64, 128])
def test_word_map_covers_a_block(d):
    """Every nibble of the code words belongs to exactly one (token, value) of each kind."""
    for which, lo in (("k", 0), ("v", 2 * d)):
        seen = {su.word_of(which, t, e, d) for t in range(16) for e in range(d)}
        assert seen == {(w, n) for w in range(lo, lo + 2 * d) for n in range(8)}


@pytest.mark.parametrize("d", [64, 128])
def test_cache_references_agree(d):
    """pack_cache, unpack_token and random_cache describe one format, and the plain form of
    the operators' cases decodes it alike."""
    import perf.operators as cases

    rng = np.random.default_rng(d)
    cache, kp, vp = su.random_cache(rng, 3, 2, 32, d)
    for slot in (0, 17, 40, 95):
        for part, got in zip((kp, vp), su.unpack_token(cache, slot, 1, 32, d)):
            for a, b in zip(part, got):
                assert np.array_equal(a[slot // 32, 1, slot % 32], b)
    table = torch.tensor([[2, 0, 1]])
    for part, got in zip((kp, vp), cases._gather_cache(torch.from_numpy(cache), table, d)):
        want = np.concatenate([su.values(*(x[p] for x in part)) for p in (2, 0, 1)], 1)
        assert np.array_equal(got[0].numpy(), want.astype(np.float32))
    k, v = su.bf16(rng.normal(size=d)), su.bf16(rng.normal(size=d) * 3)
    su.pack_cache(cache, 50, 0, k, v, 32)
    for x, (c, s, z) in zip((k, v), su.unpack_token(cache, 50, 0, 32, d)):
        y = su.values(c, s, z)
        assert np.abs(y - x).max() <= 0.5 * s.max() * (1 + 15 * 2.0 ** -8)
    assert np.array_equal(su.unpack_token(cache, 51, 0, 32, d)[0][0], kp[0][1, 0, 19])


def test_quantise_groups():
    x = np.concatenate([np.full(32, 2.5), np.arange(32.0)])
    c, s, z = su.quantise(x)
    assert (c[:32] == 0).all() and s[0] == 0 and z[0] == 2.5
    assert s[1] == su.bf16(np.array(31 / 15)) and z[1] == 0 and c[32] == 0 and c[63] == 15
