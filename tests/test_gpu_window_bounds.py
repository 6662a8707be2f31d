"""attn_window_fwd within the bounds of its two forms: the token form's weights are two bf16
numbers, the tile form's one. Partials over two chunks of the keys merge within what each
part's own bound gives."""

from __future__ import annotations

import numpy as np
import pytest
import torch

import serving_util as su
from workloads import randn_bf16

pytestmark = pytest.mark.gpu

# A weight as two bf16 numbers: the upper 8 bits cut off (what is left is below 2^-7 of it),
# the rest rounded by at most 2^-8 of itself. And fp32 sums: a warp's run of at most a few
# blocks and the join of at most 148 parts, in groups, some 64 additions off by 2^-23 each.
TWO_PARTS = 2.0 ** -15 + 64 * 2.0 ** -23


@pytest.fixture(scope="module")
def osx():
    import online_softmax_exact_b200 as m

    return m


def tensors(B, Hq, Hkv, Nq, Nkv, d, seed, qsize=1.0):
    return (randn_bf16((B, Hq, Nq, d), seed, 0) * qsize, randn_bf16((B, Hkv, Nkv, d), seed, 1),
            randn_bf16((B, Hkv, Nkv, d), seed, 2))


def reference(q, k, v, b, h, Hkv, off, kv_off, window, sinks, wround, o_bf16=False):
    g, d = h * Hkv // q.shape[1], q.shape[3]
    see = su.visible(off + np.arange(q.shape[2]), kv_off + np.arange(k.shape[2]), window, sinks)
    return su.attention(su.to_np(q[b, h]), su.to_np(k[b, g]), su.to_np(v[b, g]), see,
                        np.float64(np.float32(d ** -0.5)), wround=wround, o_bf16=o_bf16)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Hq,Hkv", [(2, 2), (4, 1), (8, 2), (9, 1)])
@pytest.mark.parametrize("Nq,Nkv", [(1, 1), (1, 900), (3, 1300), (5, 640), (20, 333)])
@pytest.mark.parametrize("window,sinks,qsize", [(200, 4, 1.0), (5000, 0, 1.0), (5000, 0, 0.0), (600, 40, 4.0)])
def test_token_form(osx, d, Hq, Hkv, Nq, Nkv, window, sinks, qsize):
    assert osx.lib().attn_window_fwd_workspace(2, Hq, Hkv, Nq, d) > 0
    q, k, v = tensors(2, Hq, Hkv, Nq, Nkv, d, Nkv, qsize)
    o, lse = osx.attn_window_fwd(q.cuda(), k.cuda(), v.cuda(), window=window, sinks=sinks)
    assert osx.attn_device_status() == osx.ATTN_OK
    for b in range(2):
        for h in range(Hq):
            ref = reference(q, k, v, b, h, Hkv, Nkv - Nq, 0, window, sinks, TWO_PARTS)
            su.check(su.to_np(o)[b, h], su.to_np(lse)[b, h], ref, f"batch {b} head {h}")


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Nq,Hq,Hkv", [(1, 4, 2), (3, 4, 2), (200, 8, 8)])
@pytest.mark.parametrize("cut", [450, 597])
def test_partials_merge(osx, d, Nq, Hq, Hkv, cut):
    B, n, window, sinks = 2, 600, 300, 4
    q, k, v = tensors(B, Hq, Hkv, Nq, n, d, 4)
    token = osx.lib().attn_window_fwd_workspace(B, Hq, Hkv, Nq, d) > 0
    assert token == (Nq < 200)
    wround = TWO_PARTS if token else su.HALF_BF16
    chunks = [(0, cut), (cut, n)]
    parts = [osx.attn_window_fwd(q.cuda(), k[:, :, a:b].contiguous().cuda(), v[:, :, a:b].contiguous().cuda(),
                                 window=window, sinks=sinks, q_off=n - Nq, kv_off=a) for a, b in chunks]
    o, lse = osx.attn_merge([p[0] for p in parts], [p[1] for p in parts])
    for b in range(B):
        for h in range(Hq):
            refs = [reference(q, k[:, :, x:y], v[:, :, x:y], b, h, Hkv, n - Nq, x, window, sinks, wround)
                    for x, y in chunks]
            ro, rl, _, _ = reference(q, k, v, b, h, Hkv, n - Nq, 0, window, sinks, wround)
            # weights e^(l_i - l) of the parts: off by the parts' own errors of l, by that of l
            # (no more than their largest) and by the merge's exponentials and sums
            bound, lbound = 0, 0
            for po, pl, bo, bl in refs:
                a = np.exp(pl - rl)[:, None]
                err = (bl + max(x[3].max() for x in refs) + 2.0 ** -18)[:, None]
                bound = bound + a * (bo + np.abs(po) * err) * (1 + err)
                lbound = np.maximum(lbound, bl)
            bound = bound + 2.0 ** -22 * np.abs(ro) + 1e-30
            lbound = lbound + 2.0 ** -18 + 2.0 ** -22 * np.abs(rl)
            su.check(su.to_np(o)[b, h], su.to_np(lse)[b, h], (ro, rl, bound, lbound), f"{b} {h}")
