"""The serving operators with ``stream=``: what a call allocates belongs to the stream that it
runs on, so that it shares no memory with work that is still pending elsewhere."""

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


def i32(x):
    return torch.as_tensor(np.ascontiguousarray(x), dtype=torch.int32).cuda()


@pytest.fixture(scope="module")
def calls(osx):
    """Each operator that allocates, as a call of the stream alone."""
    g = torch.Generator().manual_seed(0)
    B, Hq, Hkv, d, page, width = 3, 8, 2, 128, 16, 40
    cache = torch.from_numpy(su.random_cache(np.random.default_rng(0), B * width, Hkv, page, d)[0]).cuda()
    table = torch.randperm(B * width, generator=g).int().view(B, width).cuda()
    grown, start = table.clone(), i32([0, 0, 0])
    lens, new = i32([600, 17, 333]), i32([2, 1, 0])
    free, head = (torch.arange(64) + B * width).int().cuda(), i32([0])
    qkv = torch.randn((B, 2, (Hq + 2 * Hkv) * d), generator=g).bfloat16().cuda()
    w = torch.randn(d, generator=g).bfloat16().cuda()
    inv = (10000.0 ** (-torch.arange(d // 2) / (d / 2.0))).cuda()
    pos = i32([[600, 601], [17, 18], [333, 334]])
    q = torch.randn((B, Hq, 2, d), generator=g).bfloat16().cuda()
    k, v = (torch.randn((B, Hkv, 300, d), generator=g).bfloat16().cuda() for _ in range(2))
    out = {
        "plan": lambda **s: osx.attn_kv_plan(lens, new, grown, free, head, page_size=page, n_new=2, **s),
        "rope": lambda **s: osx.attn_qk_norm_rope(qkv, w, w, inv, pos, n_heads=Hq, n_kv_heads=Hkv, **s),
        "read": lambda **s: osx.attn_kv4_read(cache, table, start, lens, n=100, **s),
        "kv4": lambda **s: osx.attn_kv4_fwd(q, cache, table, lens, **s),
        "window": lambda **s: osx.attn_window_fwd(q, k, v, window=90, sinks=4, **s),
    }
    torch.cuda.synchronize()
    return out


def spans(tensors):
    return [(t.data_ptr(), t.data_ptr() + t.numel() * t.element_size()) for t in tensors]


def settled(call, **kw):
    """The call's outputs, with nothing pending before or behind it."""
    torch.cuda.synchronize()
    out = call(**kw)
    torch.cuda.synchronize()
    return out


@pytest.mark.parametrize("raw", [False, True])
@pytest.mark.parametrize("name", ["plan", "rope", "read", "kv4", "window"])
def test_outputs_of_a_given_stream_are_not_the_current_stream_s_freed_memory(calls, name, raw):
    """Blocks just freed on the current stream may still be in use there. (Nothing is in use
    here: the addresses alone are compared.)"""
    first = settled(calls[name])
    freed, want = spans(first), [t.clone() for t in first]
    del first
    side = torch.cuda.Stream()
    got = settled(calls[name], stream=side.cuda_stream if raw else side)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    for lo, hi in spans(got):
        assert not any(lo < h and l < hi for l, h in freed)


@pytest.mark.parametrize("raw", [False, True])
@pytest.mark.parametrize("name", ["kv4", "window"])
def test_workspace_of_a_given_stream_comes_from_its_pool(calls, name, raw):
    """With both outputs given, what a call allocates is its workspace."""
    out = settled(calls[name])
    side = torch.cuda.Stream()
    torch.cuda.empty_cache()

    def held():
        return sum(s["total_size"] for s in torch.cuda.memory_snapshot()
                   if s["stream"] == side.cuda_stream)

    before = held()
    settled(calls[name], stream=side.cuda_stream if raw else side, o=out[0], lse=out[1])
    assert held() > before


@pytest.mark.parametrize("raw", [False, True])
@pytest.mark.parametrize("which", ["kv4", "window"])
def test_unordered_calls_on_two_streams(osx, which, raw):
    """Calls of one size, one on the current stream and one with ``stream=``, nothing ordering
    them: each gives the bits it gives alone."""
    g = torch.Generator().manual_seed(1)
    Hq, Hkv, d, n = 8, 2, 128, 32768
    qs = [torch.randn((1, Hq, 1, d), generator=g).bfloat16().cuda() for _ in range(2)]
    if which == "kv4":
        cache = torch.from_numpy(su.random_cache(np.random.default_rng(1), n // 64, Hkv, 64, d)[0]).cuda()
        table, lens = i32(np.arange(n // 64)[None]), i32([n])

        def call(q, **kw):
            return osx.attn_kv4_fwd(q, cache, table, lens, **kw)
    else:
        k, v = (torch.randn((1, Hkv, n, d), generator=g).bfloat16().cuda() for _ in range(2))

        def call(q, **kw):
            return osx.attn_window_fwd(q, k, v, window=n, **kw)
    want = [[t.clone() for t in settled(lambda: call(q))] for q in qs]
    side = torch.cuda.Stream()
    given = side.cuda_stream if raw else side
    torch.cuda.synchronize()
    for _ in range(50):
        a = call(qs[0])
        b = call(qs[1], stream=given)
        c = call(qs[0])
        torch.cuda.synchronize()
        for got, ref in ((a, want[0]), (b, want[1]), (c, want[0])):
            assert all(torch.equal(x, y) for x, y in zip(got, ref))
    assert osx.attn_device_status() == osx.ATTN_OK


@pytest.mark.parametrize("raw", [False, True])
@pytest.mark.parametrize("name", ["plan", "rope", "read", "kv4", "window"])
def test_outputs_dropped_while_the_current_stream_reads_them(calls, name, raw):
    """Results of another stream, read on the current one and dropped there: the next call on
    that stream does not write over them before they are read."""
    want = [t.clone() for t in settled(calls[name])]
    side = torch.cuda.Stream()
    given = side.cuda_stream if raw else side
    out = settled(calls[name], stream=given)
    torch.cuda._sleep(50_000_000)  # the copies below wait for some 25 ms
    copies = [t.clone() for t in out]
    del out
    with torch.cuda.stream(side):
        keep = [[t.fill_(1) for t in calls[name](stream=given)] for _ in range(4)]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(copies, want))
    assert all(bool((t == 1).all()) for out in keep for t in out)


@pytest.mark.parametrize("handle", [0, 1])
def test_default_stream_by_its_handles(osx, calls, handle):
    for name, call in calls.items():
        want = [t.clone() for t in settled(call)]
        with torch.cuda.stream(torch.cuda.Stream()):
            got = settled(call, stream=handle)
        assert all(torch.equal(a, b) for a, b in zip(got, want)), name


def test_captured_calls_on_a_forked_stream(osx, calls):
    """A captured step whose calls run on a stream forked off the capturing one, by object and
    by handle, replays to the bits of eager calls."""
    want = {n: [t.clone() for t in settled(c)] for n, c in calls.items()}
    side = torch.cuda.Stream()
    got = {}
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        side.wait_stream(torch.cuda.current_stream())
        for i, (n, c) in enumerate(calls.items()):
            got[n] = c(stream=side if i % 2 else side.cuda_stream)
            c()  # and one beside it
        torch.cuda.current_stream().wait_stream(side)
    for _ in range(3):
        for out in got.values():
            for t in out:
                t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for n, out in got.items():
            assert all(torch.equal(a, b) for a, b in zip(out, want[n])), n
