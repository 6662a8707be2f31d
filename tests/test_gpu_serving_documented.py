"""The decode steps that README.md and the serving module's docstring show, run as written on
a ragged batch: each row that is a token attends from that token's position."""

from __future__ import annotations

import inspect
import pathlib
import re
import textwrap

import numpy as np
import pytest
import torch

import serving_util as su

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def osx():
    import online_softmax_exact_b200 as m

    return m


def readme_step():
    text = (pathlib.Path(__file__).parent.parent / "README.md").read_text()
    blocks = [b for b in re.findall(r"```python\n(.*?)```", text, re.S) if "attn_kv_plan" in b]
    assert len(blocks) == 1
    return blocks[0]


def docstring_step():
    from online_softmax_exact_b200 import serving

    return textwrap.dedent(inspect.getdoc(serving).split("::\n\n", 1)[1])


@pytest.mark.parametrize("source", [readme_step, docstring_step])
def test_documented_step_on_a_ragged_batch(osx, source):
    rng, g = np.random.default_rng(0), torch.Generator().manual_seed(0)
    B, N, Hq, Hkv, d, page, width = 4, 5, 8, 2, 128, 64, 6
    old, new = np.array([130, 0, 63, 200]), np.array([5, 3, 1, 0])
    n_pages = B * width
    cache, kp, vp = su.random_cache(rng, n_pages, Hkv, page, d)
    table = rng.permutation(n_pages).reshape(B, width)
    held = -(-old // page)
    table[np.arange(width)[None] >= held[:, None]] = -1
    free = np.array(sorted(set(range(n_pages)) - set(table[table >= 0])))

    def i32(x):
        return torch.as_tensor(np.ascontiguousarray(x), dtype=torch.int32).cuda()

    seen = {}

    def keep(name):
        def call(*a, **kw):
            seen[name] = getattr(osx, name)(*a, **kw)
            return seen[name]
        return call

    cg = torch.from_numpy(cache).cuda()
    names = {n: keep(n) for n in ("attn_kv_plan", "attn_qk_norm_rope", "attn_kv4_append",
                                  "attn_kv4_fwd", "attn_window_fwd")}
    names["kv4_cache"] = lambda *a, **kw: cg
    W, S = 4096, 4
    space = dict(
        names, osx=type("Osx", (), {k: staticmethod(f) for k, f in names.items()}), cache=cg,
        lens=i32(old), new_lens=i32(new), table=i32(table), free_pages=i32(free), free=i32(free),
        head=i32([0]), N=N, n_pages=n_pages, n_kv_heads=Hkv, n_heads=Hq, Hq=Hq, Hkv=Hkv, d=d, W=W, S=S,
        qkv=torch.randn((B, N, (Hq + 2 * Hkv) * d), generator=g).bfloat16().cuda(),
        wq=torch.ones(d).bfloat16().cuda(), wk=torch.ones(d).bfloat16().cuda(),
        inv_freq=(10000.0 ** (-torch.arange(64) / 64.0)).cuda())
    exec(source(), space)
    torch.cuda.synchronize()
    assert osx.attn_device_status() == osx.ATTN_OK
    # the step leaves the state that the next one starts from
    assert np.array_equal(space["lens"].cpu().numpy(), old + new)
    q, k, v = (su.to_np(t) for t in seen["attn_qk_norm_rope"])
    o, lse = (su.to_np(t) for t in seen["attn_kv4_fwd"])
    for b in range(B):
        pos = np.arange(old[b])
        pg = table[b, pos // page]
        see = su.visible(old[b] + np.arange(new[b]), np.arange(old[b] + new[b]), W, S)
        for h in range(Hkv):
            sides = []
            for part, x in ((kp, k), (vp, v)):
                was = [y[pg, h, pos % page] for y in part]
                now = su.quantise(x[b, h, :new[b]])
                sides.append([np.concatenate([y, z]) for y, z in zip(was, now)])
            vals = [su.values(*x) for x in sides]
            mags = [su.values(c, s, np.abs(z)) for c, s, z in sides]
            for r in range(h * (Hq // Hkv), (h + 1) * (Hq // Hkv)):
                if new[b]:
                    ref = su.attention(q[b, r, :new[b]], *vals, see, np.float64(np.float32(d ** -0.5)),
                                       *mags, mags[1], 2.0 ** -15)
                    su.check(o[b, r, :new[b]], lse[b, r, :new[b]], ref, f"request {b} head {r}")
