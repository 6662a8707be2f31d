"""attn_window_fwd against the definition in 64 bits."""

from __future__ import annotations

import numpy as np
import pytest
import torch

import serving_util as su
from workloads import randn_bf16

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def osx():
    import online_softmax_exact_b200 as m

    return m


def case(osx, Nq, Nkv, d, window, sinks, B=1, Hq=2, Hkv=1, q_off=None, kv_off=0, kv_len=None,
         scale=None, o_dtype=torch.float32, qsize=1.0, seed=0, **kw):
    q = randn_bf16((B, Hq, Nq, d), seed, 0) * qsize
    k, v = randn_bf16((B, Hkv, Nkv, d), seed, 1), randn_bf16((B, Hkv, Nkv, d), seed, 2)
    n = Nkv if kv_len is None else kv_len
    kg, vg = k.cuda(), v.cuda()
    kg[:, :, n:], vg[:, :, n:] = float("nan"), float("nan")
    o, lse = osx.attn_window_fwd(q.cuda(), kg, vg, window=window, sinks=sinks, q_off=q_off,
                                 kv_off=kv_off, kv_len=kv_len, scale=scale, o_dtype=o_dtype, **kw)
    assert osx.attn_device_status() == osx.ATTN_OK
    off = kv_off + n - Nq if q_off is None else q_off
    see = su.visible(off + np.arange(Nq), kv_off + np.arange(n), window, sinks)
    on, ln = su.to_np(o), su.to_np(lse)
    qn, kn, vn = su.to_np(q), su.to_np(k), su.to_np(v)
    s = np.float64(np.float32(d ** -0.5 if scale is None else scale))
    for b in range(B):
        for h in range(Hq):
            g = h * Hkv // Hq
            ref = su.attention(qn[b, h], kn[b, g, :n], vn[b, g, :n], see, s,
                               o_bf16=o_dtype == torch.bfloat16)
            su.check(on[b, h], ln[b, h], ref, f"batch {b} head {h}")
    return o, lse


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("N", [1, 7, 128, 129, 257, 600])
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (64, 4), (128, 0), (129, 129), (200, 700),
                                          (1000, 3)])
def test_window(osx, d, N, window, sinks):
    case(osx, N, N, d, window, sinks)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("N,H,B", [(17, 90, 2), (128, 12, 1), (129, 13, 1), (257, 6, 1), (600, 3, 1)])
@pytest.mark.parametrize("group", [1, 2])
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (64, 4), (128, 0), (129, 129), (200, 700),
                                          (1000, 3)])
def test_window_tile_form(osx, d, N, H, B, group, window, sinks):
    """Sizes that run on 128-row tiles (no workspace); test_window's run in the token form.
    Groups of two heads run as pairs of heads, single ones as pairs of row tiles."""
    assert osx.lib().attn_window_fwd_workspace(B, group * H, H, N, d) == 0
    case(osx, N, N, d, window, sinks, B=B, Hq=group * H, Hkv=H)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Nq,Nkv,B,Hq,Hkv", [(70, 500, 4, 8, 2), (300, 900, 1, 8, 8), (300, 300, 2, 5, 5)])
@pytest.mark.parametrize("window,sinks", [(200, 4), (33, 0), (5000, 1), (150, 300)])
def test_window_tile_form_newest_rows(osx, d, Nq, Nkv, B, Hq, Hkv, window, sinks):
    assert osx.lib().attn_window_fwd_workspace(B, Hq, Hkv, Nq, d) == 0
    case(osx, Nq, Nkv, d, window, sinks, B=B, Hq=Hq, Hkv=Hkv, o_dtype=torch.bfloat16)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("N,window,sinks", [(2500, 300, 4), (2500, 128, 260), (1537, 1024, 64)])
@pytest.mark.parametrize("Hq,Hkv", [(6, 2), (8, 2), (5, 5)])
def test_window_many_units(osx, d, N, window, sinks, Hq, Hkv):
    case(osx, N, N, d, window, sinks, B=2, Hq=Hq, Hkv=Hkv, o_dtype=torch.bfloat16)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Nq,Nkv", [(1, 1), (1, 17), (1, 900), (2, 900), (5, 1300), (20, 640), (70, 500),
                                    (300, 900)])
@pytest.mark.parametrize("window,sinks", [(200, 4), (33, 0), (5000, 1)])
def test_window_newest_rows(osx, d, Nq, Nkv, window, sinks):
    case(osx, Nq, Nkv, d, window, sinks, B=2, Hq=4, Hkv=2)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (8, 8), (8, 1), (20, 1), (12, 4)])
@pytest.mark.parametrize("Nq", [1, 3, 130])
def test_window_heads(osx, d, Hq, Hkv, Nq):
    case(osx, Nq, 400, d, 150, 4, Hq=Hq, Hkv=Hkv, o_dtype=torch.bfloat16)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Nq,H", [(2, 1), (300, 1), (300, 5)])
@pytest.mark.parametrize("q_off,kv_off", [(0, 0), (0, 100), (350, 0), (1000, 0), (1000, 900),
                                          (10 ** 9, 10 ** 9 - 100), (2 ** 40, 0), (500, 200)])
def test_window_chunk_offsets(osx, d, Nq, H, q_off, kv_off):
    """Chunks before, around and behind the rows' windows, sinks inside and outside the
    chunk: rows without a key are zero with LSE -inf."""
    case(osx, Nq, 333, d, 120, 230, q_off=q_off, kv_off=kv_off, Hq=H, Hkv=H)
    case(osx, Nq, 333, d, 120, 0, q_off=q_off, kv_off=kv_off, Hq=H, Hkv=H)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Nq,Hkv", [(1, 2), (100, 2), (100, 8)])
def test_window_inside_a_longer_buffer(osx, d, Nq, Hkv):
    """Keys behind kv_len are never read (they hold NaN here)."""
    case(osx, Nq, 700, d, 90, 4, B=2, Hq=8, Hkv=Hkv, kv_len=301)
    case(osx, Nq, 700, d, 1000, 4, B=2, Hq=8, Hkv=Hkv, kv_len=512)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Nq,H", [(1, 1), (260, 6)])
@pytest.mark.parametrize("qsize,scale", [(16.0, None), (1.0, 2.0), (1.0, 1e-6)])
def test_window_large_and_flat_scores(osx, d, Nq, H, qsize, scale):
    case(osx, Nq, 500, d, 180, 4, qsize=qsize, scale=scale, Hq=H, Hkv=H)


def test_window_covers_a_causal_call(osx):
    """A window as long as the sequence is causal attention; both are exact."""
    q, k, v = (randn_bf16((1, 4, 900, 128), 3, i).cuda() for i in range(3))
    o, lse = osx.attn_window_fwd(q, k, v, window=900)
    o2, lse2 = osx.attn_fwd(q, k, v, causal=True)
    assert (o - o2).abs().max() <= 2 * 5 * su.HALF_BF16 and (lse - lse2).abs().max() <= 1e-4


@pytest.mark.parametrize("Nq", [1, 3, 200])
def test_window_partials_merge(osx, Nq):
    """Results over two chunks of the keys merge to the result over all of them."""
    q = randn_bf16((1, 4, Nq, 128), 4, 0).cuda()
    k, v = (randn_bf16((1, 2, 600, 128), 4, i).cuda() for i in (1, 2))
    whole = osx.attn_window_fwd(q, k, v, window=300, sinks=4)
    parts = [osx.attn_window_fwd(q, k[:, :, a:b].contiguous(), v[:, :, a:b].contiguous(), window=300,
                                 sinks=4, q_off=600 - Nq, kv_off=a) for a, b in ((0, 450), (450, 600))]
    o, lse = osx.attn_merge([p[0] for p in parts], [p[1] for p in parts])
    assert (o - whole[0]).abs().max() <= 2 * 5 * su.HALF_BF16
    assert (lse - whole[1]).abs().max() <= 1e-4


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Nq,H", [(3, 2), (200, 8)])
def test_window_of_parent_rows(osx, d, Nq, H):
    """The C entry point on rows inside longer parents (q_ld, kv_ld), chunk starts included;
    parent rows outside hold NaN."""
    B, q_ld, kv_ld, q0, k0, Nkv = 2, 300, 500, 31, 77, 380
    q = torch.full((B, H, q_ld, d), float("nan"), dtype=torch.bfloat16)
    k, v = (torch.full((B, H, kv_ld, d), float("nan"), dtype=torch.bfloat16) for _ in range(2))
    q[:, :, q0:q0 + Nq] = randn_bf16((B, H, Nq, d), 6, 0)
    k[:, :, k0:k0 + Nkv], v[:, :, k0:k0 + Nkv] = (randn_bf16((B, H, Nkv, d), 6, i) for i in (1, 2))
    qg, kg, vg = q.cuda(), k.cuda(), v.cuda()
    o = torch.empty((B, H, Nq, d), device="cuda")
    lse = torch.empty((B, H, Nq), device="cuda")
    lib = osx.lib()
    n = lib.attn_window_fwd_workspace(B, H, H, Nq, d)
    ws = torch.empty(max(n, 1), dtype=torch.uint8, device="cuda")
    st = lib.attn_window_fwd(qg.data_ptr() + q0 * d * 2, kg.data_ptr() + k0 * d * 2,
                             vg.data_ptr() + k0 * d * 2, o.data_ptr(), lse.data_ptr(), 0, B, H, H, Nq,
                             Nkv, q_ld, kv_ld, 190, 0, d, 100, 3, d ** -0.5, ws.data_ptr(), n,
                             torch.cuda.current_stream().cuda_stream)
    assert st == osx.ATTN_OK and osx.attn_device_status() == osx.ATTN_OK
    see = su.visible(190 + np.arange(Nq), np.arange(Nkv), 100, 3)
    for b in range(B):
        for h in range(H):
            ref = su.attention(su.to_np(q)[b, h, q0:q0 + Nq], su.to_np(k)[b, h, k0:k0 + Nkv],
                               su.to_np(v)[b, h, k0:k0 + Nkv], see, np.float64(np.float32(d ** -0.5)))
            su.check(su.to_np(o)[b, h], su.to_np(lse)[b, h], ref, f"batch {b} head {h}")
