"""attn_qk_norm_rope against its definition in 64 bits."""

from __future__ import annotations

import numpy as np
import pytest
import torch

import serving_util as su

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def osx():
    import online_softmax_exact_b200 as m

    return m


def check(osx, B, N, Hq, Hkv, d, r, interleaved, w_dtype=torch.bfloat16, far=0, pad=0, eps=1e-6,
          size=1.0, stream=None):
    g = torch.Generator().manual_seed(B * 31 + N + Hq + r)
    W = (Hq + 2 * Hkv) * d
    full = torch.randn((B, N, W + pad), generator=g).mul(size).to(torch.bfloat16)
    qkv = full.cuda()[..., pad:]
    wq = (1 + 0.3 * torch.randn(d, generator=g)).to(w_dtype)
    wk = (1 + 0.3 * torch.randn(d, generator=g)).to(w_dtype)
    inv = (10000.0 ** (-torch.arange(0, r, 2).float() / r))
    pos = torch.randint(0, 50, (B, N), generator=g, dtype=torch.int32) + far
    q, k, v = osx.attn_qk_norm_rope(qkv, wq.cuda(), wk.cuda(), inv.cuda(), pos.cuda(), n_heads=Hq,
                                    n_kv_heads=Hkv, eps=eps, interleaved=interleaved,
                                    stream=stream)
    torch.cuda.synchronize()
    x = su.to_np(full[..., pad:]).reshape(B, N, Hq + 2 * Hkv, d).transpose(0, 2, 1, 3)
    for got, rows, w in ((q, x[:, :Hq], wq), (k, x[:, Hq:Hq + Hkv], wk)):
        ref, mag = su.norm_rope(rows, su.to_np(w), su.to_np(inv), pos.numpy()[:, None], eps,
                                interleaved)
        # one rounding to bf16, and fp32 arithmetic: the norm (d terms, each within 2^-24,
        # under a root: (d / 2 + 4) 2^-24 of the value) and the rotation (angle within
        # 2^-22 after its reduction to [-pi, pi], sine and cosine within 2^-21.1: 2^-20)
        err = mag * ((d / 2 + 4) * 2.0 ** -24 + 2.0 ** -20)
        bound = su.HALF_BF16 * (np.abs(ref) + err) + err + 1e-38
        assert (np.abs(su.to_np(got) - ref) <= bound).all()
    assert np.array_equal(su.to_np(v), x[:, Hq + Hkv:])


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("rot", [1.0, 0.5, 0.25])
def test_rope(osx, d, interleaved, rot):
    check(osx, 2, 5, 6, 3, d, int(d * rot), interleaved)


@pytest.mark.parametrize("B,N,Hq,Hkv", [(1, 1, 1, 1), (33, 1, 32, 8), (1, 200, 5, 1), (3, 7, 48, 4),
                                        (1, 3, 1, 60), (2, 2, 64, 64)])
@pytest.mark.parametrize("d", [64, 128])
def test_rope_sizes(osx, B, N, Hq, Hkv, d):
    check(osx, B, N, Hq, Hkv, d, d, False)


@pytest.mark.parametrize("d,r", [(128, 16), (128, 48), (128, 112), (64, 16), (64, 48)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_rope_odd_parts(osx, d, r, interleaved):
    check(osx, 1, 9, 3, 2, d, r, interleaved)


@pytest.mark.parametrize("far", [131072, 10_000_000, 2 ** 31 - 64, -1000])
def test_rope_far_positions(osx, far):
    check(osx, 1, 20, 2, 1, 128, 128, False, far=far)


def test_rope_strided_rows_and_fp32_weights(osx):
    check(osx, 3, 17, 4, 2, 128, 128, False, w_dtype=torch.float32, pad=64)
    check(osx, 3, 17, 4, 2, 64, 64, True, w_dtype=torch.float32, pad=8)


@pytest.mark.parametrize("size,eps", [(1e-12, 1e-6), (0.0, 1e-6), (1e15, 0.0)])
def test_rope_small_and_large_rows(osx, size, eps):
    check(osx, 1, 4, 2, 2, 128, 128, False, size=size, eps=eps)


def test_rope_other_stream_and_one_row_strides(osx):
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    check(osx, 1, 1, 2, 2, 64, 64, False, pad=8, stream=s)
