"""attn_kv_plan over several blocks directly followed by attn_kv4_fwd on the table and lengths
that it writes, with nothing between the launches: the attention's blocks may be resident, and
hold lines of the old table, while the plan still enters pages."""

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


@pytest.mark.parametrize("B,n_new,width", [(32, 100, 7), (48, 64, 5), (600, 5, 3)])
@pytest.mark.parametrize("d", [64, 128])
def test_attention_sees_the_plan_s_pages(osx, B, n_new, width, d):
    """Rows of the table share lines that several blocks of the plan write (rows of 12 to 28
    bytes, 1024 tokens a block). Same buffers every time, other pages and lengths."""
    page, Hkv, Hq = 16, 1, 4
    rng, g = np.random.default_rng(B), torch.Generator().manual_seed(B)
    n_pages = 2 * B * width
    small = torch.from_numpy(su.random_cache(rng, 64, Hkv, page, d)[0]).cuda()
    cache = small[torch.randint(0, 64, (n_pages,), generator=g).cuda()].contiguous()
    q = torch.randn((B, Hq, 1, d), generator=g).bfloat16().cuda()
    states = []
    for _ in range(8):
        perm = torch.randperm(n_pages, generator=g).int()
        lens = torch.randint(0, width * page - n_new + 1, (B,), generator=g).int()
        table = perm[:B * width].view(B, width).clone()
        table[torch.arange(width)[None] >= (lens[:, None] + page - 1) // page] = -1
        new = torch.randint(0, n_new + 1, (B,), generator=g).int()
        states.append([t.cuda() for t in (lens, new, table, perm[B * width:].contiguous())])
    head = torch.zeros(1, dtype=torch.int32).cuda()
    buf = [t.clone() for t in states[0]]

    def attend(settle):
        lens, new, table, free = buf
        out = osx.attn_kv_plan(lens, new, table, free, head, page_size=page, n_new=n_new)
        if settle:
            torch.cuda.synchronize()
        o, lse = osx.attn_kv4_fwd(q, cache, table, out[2], max_len=width * page)
        return o, lse, out[4]

    def load(state):
        for b, t in zip(buf, state):
            b.copy_(t)

    want = []
    for s in states:
        load(s)
        torch.cuda.synchronize()
        want.append(attend(True))
    torch.cuda.synchronize()
    assert all(bool(w[2].all()) for w in want)
    assert not any(torch.equal(a[0], b[0]) for a, b in zip(want, want[1:]))
    got = []
    for _ in range(10):
        for s in states:
            load(s)
            got.append(attend(False))
    torch.cuda.synchronize()
    for i, out in enumerate(got):
        ref = want[i % len(states)]
        assert all(torch.equal(a, b) for a, b in zip(out, ref)), i
    assert osx.attn_device_status() == osx.ATTN_OK
