"""attn_kv4_fwd over many requests (the runs' start is found within a warp up to 32 requests,
by a block-wide scan up to 256, in two passes beyond), and at the limits of its numbers; the
quantiser's codes for every scale."""

from __future__ import annotations

import numpy as np
import pytest
import torch

import serving_util as su
from test_gpu_kv4 import append_case, fwd_case, i32

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def osx():
    import online_softmax_exact_b200 as m

    return m


def ragged(B, longest, empty, seed):
    """Lengths of 1 to longest, 0 where ``empty`` says so."""
    lens = np.random.default_rng(seed).integers(1, longest + 1, B)
    lens[np.array(empty(np.arange(B)))] = 0
    return lens


EMPTY = {
    "none": lambda b: b < 0,
    "first": lambda b: b < len(b) // 3,
    "last": lambda b: b >= len(b) - len(b) // 3,
    "border": lambda b: (b >= len(b) // 2 - 20) & (b < len(b) // 2 + 20),  # across 256 of 512
    "all_but_one": lambda b: b != len(b) - 2,
}


@pytest.mark.parametrize("B", [32, 33, 64, 255, 256, 257, 512, 600])
@pytest.mark.parametrize("empty", sorted(EMPTY))
@pytest.mark.parametrize("d,Nq,Hq,Hkv", [(64, 1, 2, 1), (128, 3, 2, 1)])
def test_fwd_many_requests(osx, B, empty, d, Nq, Hq, Hkv):
    lens = ragged(B, 90, EMPTY[empty], B)
    fwd_case(osx, B, B, Hq, Hkv, Nq, d, 16, lens, width=6)


@pytest.mark.parametrize("d,Nq,Hq,Hkv", [(64, 3, 4, 2), (128, 1, 4, 1), (128, 3, 2, 1)])
def test_fwd_many_requests_of_several_runs(osx, d, Nq, Hq, Hkv):
    """More than 32 requests, a few of them so long that several warps share their units."""
    lens = np.random.default_rng(0).integers(0, 60, 40)
    lens[[0, 17, 33, 39]] = [3000, 2999, 2500, 3000]
    fwd_case(osx, 3, 40, Hq, Hkv, Nq, d, 64, lens, o_dtype=torch.bfloat16)
    fwd_case(osx, 4, 40, Hq, Hkv, Nq, d, 64, lens, window=700, sinks=5)


@pytest.mark.parametrize("B", [48, 300])
def test_fwd_many_requests_merge(osx, B):
    """One call of B requests gives what calls of 20 give, to the rounding of their joins, and
    the same bits again."""
    rng = np.random.default_rng(B)
    page, d, width = 16, 128, 20
    cache, kp, vp = su.random_cache(rng, B * width // 4, 1, page, d)
    cg = torch.from_numpy(cache).cuda()
    table = i32(rng.integers(0, B * width // 4, (B, width)))
    lens = i32(rng.integers(0, width * page + 1, B))
    q = torch.randn((B, 4, 1, d), generator=torch.Generator().manual_seed(B)).bfloat16().cuda()
    o, lse = osx.attn_kv4_fwd(q, cg, table, lens)
    o2, lse2 = osx.attn_kv4_fwd(q, cg, table, lens)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    parts = [osx.attn_kv4_fwd(q[i:i + 20].contiguous(), cg, table[i:i + 20].contiguous(),
                              lens[i:i + 20].contiguous()) for i in range(0, B, 20)]
    po, pl = (torch.cat(x) for x in zip(*parts))
    assert torch.equal(torch.isneginf(lse), torch.isneginf(pl))
    seen = ~torch.isneginf(lse)
    # each within 2^-15 of the values' sizes (at most 0.4 * 15) and some fp32 roundings
    assert (o - po).abs().max() <= 2 * 6.1 * 2.0 ** -15
    assert (lse - pl)[seen].abs().max() <= 1e-4


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("qsize,ksize,scale", [
    (2.0 ** 100, 2.0 ** -110, 2.0 ** 9), (2.0 ** 20, 2.0 ** -100, 2.0 ** 80),
    (2.0 ** -100, 2.0 ** 10, 2.0 ** 88), (2.0 ** 108, 2.0 ** 10, 2.0 ** -118)])
def test_fwd_sizes_with_the_scale(osx, d, qsize, ksize, scale):
    """Query rows, the scale and their product up to 2^112, of both signs of the exponent."""
    for Nq in (1, 2):
        fwd_case(osx, 15, 2, 8, 2, Nq, d, 16, [300, 41], qsize=qsize, ksize=ksize, scale=scale)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("e", [-100, -40, 0, 40, 100])
def test_append_codes_of_every_scale(osx, d, e):
    """Groups whose scale is exactly m 2^e for each of the 128 significands m, holding the
    bf16 values next to every border between two codes."""
    rows = []
    for m in range(128, 256):
        # range 15 m as the difference of two bf16 numbers (8 bits each)
        hi, lo = (15 * m) >> 4 << 4, -((15 * m) & 15)
        border = lo + m * (np.arange(15) + 0.5)
        below = su.bf16(border)
        step = 2.0 ** (np.floor(np.log2(np.maximum(np.abs(below), 2.0 ** -20))) - 7)
        near = np.concatenate([below, np.where(below < border, below + step, below - step)])
        rows.append(np.concatenate([[lo, hi], near.clip(lo, hi)]))
    x = np.array(rows)                                           # 128 groups of 32
    assert np.array_equal(x, su.bf16(x)) and x.shape == (128, 32)
    s = su.quantise(x)[1]
    assert np.array_equal(s[:, 0], np.arange(128, 256))
    t = torch.from_numpy(x * 2.0 ** e).bfloat16().view(1, 1, 128 * 32 // d, d)
    append_case(osx, t, t.flip(2).contiguous(), [list(range(128 * 32 // d))], 16, 128 * 32 // d // 16)
