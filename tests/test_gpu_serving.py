"""The serving operators together, as a decoder layer uses them: ragged prompts and decode
steps over the paged 4-bit cache, chunked prompts over a 4-bit history, a captured decode
step, calls on several streams and threads; and what the bindings refuse."""

from __future__ import annotations

import threading

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


class Layer:
    """One attention layer's weights, pages and requests."""

    def __init__(self, osx, B, Hq, Hkv, d, page, width, rot, window, sinks, seed=0):
        self.osx, self.g = osx, torch.Generator().manual_seed(seed)
        self.B, self.Hq, self.Hkv, self.d, self.page, self.rot = B, Hq, Hkv, d, page, rot
        self.window, self.sinks = window, sinks
        self.wq, self.wk = ((1 + 0.2 * torch.randn(d, generator=self.g)).bfloat16().cuda()
                            for _ in range(2))
        self.inv = (10000.0 ** (-torch.arange(0, rot, 2).float() / rot)).cuda()
        self.cache = osx.kv4_cache(B * width + 3, Hkv, d, page_size=page)
        self.cache.fill_(0xFF)  # unwritten parameters are NaN
        self.table = torch.full((B, width), -1, dtype=torch.int32).cuda()
        self.free = torch.randperm(B * width + 3, generator=self.g).int().cuda()
        self.lens = torch.zeros(B, dtype=torch.int32).cuda()
        self.head = torch.zeros(1, dtype=torch.int32).cuda()
        self.keys = [[np.zeros((0, d))] * Hkv for _ in range(B)]    # what the cache stands for
        self.vals = [[np.zeros((0, d))] * Hkv for _ in range(B)]
        self.kz = [[np.zeros((0, d))] * Hkv for _ in range(B)]      # sizes of the stored parts
        self.vz = [[np.zeros((0, d))] * Hkv for _ in range(B)]

    def take(self, new, N):
        """Plans and stores N-padded rows of new[b] tokens; returns the rotated tensors."""
        osx, B = self.osx, self.B
        new = i32(new)
        old = self.lens
        slots, pos, self.lens, self.head, served = osx.attn_kv_plan(
            old, new, self.table, self.free, self.head, page_size=self.page, n_new=N)
        qkv = torch.randn((B, N, (self.Hq + 2 * self.Hkv) * self.d), generator=self.g).bfloat16().cuda()
        q, k, v = osx.attn_qk_norm_rope(qkv, self.wq, self.wk, self.inv, pos, n_heads=self.Hq,
                                        n_kv_heads=self.Hkv)
        osx.attn_kv4_append(k, v, self.cache, slots)
        assert served.all()
        # the norm and rotation
        x = su.to_np(qkv).reshape(B, N, -1, self.d).transpose(0, 2, 1, 3)
        ref, mag = su.norm_rope(x[:, :self.Hq], su.to_np(self.wq), su.to_np(self.inv),
                                pos.cpu().numpy()[:, None], 1e-6, False)
        assert (np.abs(su.to_np(q) - ref) <= su.HALF_BF16 * np.abs(ref) + mag * 2.0 ** -16).all()
        # what the cache now stands for
        kn, vn = su.to_np(k), su.to_np(v)
        for b in range(B):
            n = int(new[b])
            for h in range(self.Hkv):
                for store, size, y in ((self.keys, self.kz, kn), (self.vals, self.vz, vn)):
                    c, s, z = su.quantise(y[b, h, :n])
                    store[b][h] = np.concatenate([store[b][h], su.values(c, s, z)])
                    size[b][h] = np.concatenate([size[b][h], su.values(c, s, np.abs(z))])
        return q, k, v, old

    def check(self, o, lse, q, pos0, rows, what):
        on, ln, qn = su.to_np(o), su.to_np(lse), su.to_np(q)
        for b in range(self.B):
            n = len(self.keys[b][0])
            see = su.visible(int(pos0[b]) + np.arange(rows[b]), np.arange(n), self.window, self.sinks)
            for h in range(self.Hq):
                g = h * self.Hkv // self.Hq
                ref = su.attention(qn[b, h, :rows[b]], self.keys[b][g], self.vals[b][g], see,
                                   np.float64(np.float32(self.d ** -0.5)), self.kz[b][g],
                                   self.vz[b][g], self.vz[b][g], 2.0 ** -15,
                                   o.dtype == torch.bfloat16)
                su.check(on[b, h, :rows[b]], ln[b, h, :rows[b]], ref, f"{what}: request {b} head {h}")


@pytest.mark.parametrize("d,Hq,Hkv,page,rot,window,sinks", [
    (128, 8, 2, 16, 128, 0, 0), (64, 4, 4, 32, 32, 40, 3), (128, 6, 1, 48, 64, 100, 20)])
def test_prompts_then_decode_steps(osx, d, Hq, Hkv, page, rot, window, sinks):
    B, N = 4, 150
    layer = Layer(osx, B, Hq, Hkv, d, page, -(-220 // page), rot, window, sinks)
    prompt = np.array([150, 1, 77, 0])
    q, k, v, _ = layer.take(prompt, N)
    # the prompts' own attention runs on the bf16 tensors, padded rows behind the real ones
    o, lse = osx.attn_window_fwd(q, k, v, window=window or N, sinks=sinks)
    qn, kn, vn = su.to_np(q), su.to_np(k), su.to_np(v)
    for b in range(B):
        see = su.visible(np.arange(prompt[b]), np.arange(prompt[b]), window, sinks)
        for h in range(Hq):
            g = h * Hkv // Hq
            if prompt[b]:
                ref = su.attention(qn[b, h, :prompt[b]], kn[b, g, :prompt[b]], vn[b, g, :prompt[b]],
                                   see, np.float64(np.float32(d ** -0.5)))
                su.check(su.to_np(o)[b, h, :prompt[b]], su.to_np(lse)[b, h, :prompt[b]], ref, "prompt")
    # decode steps: one token each, then up to three drafted ones, then one again
    for new in ([1, 1, 1, 1], [3, 1, 2, 3], [1, 1, 1, 1], [3, 3, 3, 3]):
        n = max(new)
        q, _, _, old = layer.take(np.array(new), n)
        o, lse = osx.attn_kv4_fwd(q, layer.cache, layer.table, layer.lens, q_pos=old,
                                  window=window, sinks=sinks, o_dtype=torch.bfloat16)
        layer.check(o, lse, q, old.cpu().numpy(), new, f"step {new}")
    assert osx.attn_device_status() == osx.ATTN_OK


def test_chunked_prompt_over_a_4_bit_history(osx):
    """A prompt's second chunk: the history read back as bf16, one windowed call over it, one
    over the chunk itself, merged; equal to one call over both."""
    layer = Layer(osx, 2, 8, 2, 128, 16, 12, 128, 70, 4)
    layer.take(np.array([100, 100]), 100)
    q, k, v, old = layer.take(np.array([60, 60]), 60)
    zero = torch.zeros_like(old)
    hk, hv = osx.attn_kv4_read(layer.cache, layer.table, zero, old, n=100)
    a = osx.attn_window_fwd(q, hk, hv, window=70, sinks=4, q_off=100)
    b = osx.attn_window_fwd(q, k, v, window=70, sinks=4, q_off=100, kv_off=100)
    o, lse = osx.attn_merge([a[0], b[0]], [a[1], b[1]])
    whole = osx.attn_window_fwd(q, torch.cat([hk, k], 2), torch.cat([hv, v], 2), window=70, sinks=4)
    assert (o - whole[0]).abs().max() <= 2 * 5 * su.HALF_BF16
    assert (lse - whole[1]).abs().max() <= 1e-4
    # and against the cache itself, which holds the chunk in 4 bits too
    c, lc = osx.attn_kv4_fwd(q, layer.cache, layer.table, layer.lens, window=70, sinks=4)
    layer.check(c, lc, q, [100, 100], [60, 60], "chunk")


def step(osx, s):
    slots, pos, lens, head, served = osx.attn_kv_plan(s["lens"], s["new"], s["table"], s["free"],
                                                      s["head"], page_size=16, n_new=2)
    q, k, v = osx.attn_qk_norm_rope(s["qkv"], s["w"], s["w"], s["inv"], pos, n_heads=8, n_kv_heads=2)
    osx.attn_kv4_append(k, v, s["cache"], slots)
    first = s["lens"].clone()  # (a copy between the launches)
    o, lse = osx.attn_kv4_fwd(q, s["cache"], s["table"], lens, q_pos=first, window=200, sinks=4)
    ck, cv = osx.attn_kv4_read(s["cache"], s["table"], s["lens"], lens, n=3)
    o2, lse2 = osx.attn_window_fwd(q, s["bk"], s["bv"], window=90, sinks=4)
    o3, lse3 = osx.attn_merge([o, o2], [lse, lse2])
    return [slots, pos, lens, head, served, q, k, v, o, lse, ck, cv, o2, lse2, o3, lse3]


def fresh_step(seed):
    g = torch.Generator().manual_seed(seed)
    B, width = 5, 40
    s = dict(lens=torch.randint(0, 600, (B,), generator=g).int().cuda(),
             new=torch.randint(0, 3, (B,), generator=g).int().cuda(),
             free=(torch.randperm(B * width, generator=g).int() + B * width).cuda(),
             head=torch.zeros(1, dtype=torch.int32).cuda(),
             qkv=torch.randn((B, 2, 12 * 128), generator=g).bfloat16().cuda(),
             w=torch.randn(128, generator=g).bfloat16().cuda(),
             inv=(10000.0 ** (-torch.arange(64) / 64.0)).cuda(),
             bk=torch.randn((B, 2, 300, 128), generator=g).bfloat16().cuda(),
             bv=torch.randn((B, 2, 300, 128), generator=g).bfloat16().cuda())
    s["table"] = torch.randperm(B * width, generator=g).int().view(B, width).cuda()
    cache, _, _ = su.random_cache(np.random.default_rng(seed), 2 * B * width, 2, 16, 128)
    s["cache"] = torch.from_numpy(cache).cuda()
    return s


def test_captured_decode_step(osx):
    """A decode step in a CUDA graph, replayed on new contents of the same buffers, gives the
    bits of eager calls; two graphs keep workspaces of their own."""
    static = [fresh_step(1), fresh_step(2)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for s in static:
            step(osx, s)
    torch.cuda.current_stream().wait_stream(side)
    graphs, outs = [], []
    for s in static:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(step(osx, s))
        graphs.append(g)
    for seed in (3, 5):
        new = [fresh_step(seed), fresh_step(seed + 1)]
        want = [[t.clone() for t in step(osx, {k: v.clone() for k, v in s.items()})] for s in new]
        for s, n in zip(static, new):
            for k in s:
                s[k].copy_(n[k])
        torch.cuda.synchronize()
        streams = [torch.cuda.Stream(), torch.cuda.Stream()]
        for g, st in zip(graphs, streams):  # both at once
            with torch.cuda.stream(st):
                g.replay()
        torch.cuda.synchronize()
        for got, ref in zip(outs, want):
            assert all(torch.equal(a, b) for a, b in zip(got, ref))
    assert osx.attn_device_status() == osx.ATTN_OK


def test_streams_and_threads_at_once(osx):
    """The same calls from several threads, each on its own stream, given by name."""
    want = [[t.clone() for t in step(osx, fresh_step(s))] for s in range(3)]
    torch.cuda.synchronize()
    bad = []

    def work(i):
        try:
            st = torch.cuda.Stream()
            with torch.cuda.stream(st):
                for _ in range(20):
                    s = fresh_step(i)
                    got = step(osx, s)
                    st.synchronize()
                    if not all(torch.equal(a, b) for a, b in zip(got, want[i])):
                        bad.append(i)
        except Exception as e:  # noqa: BLE001
            bad.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(3)]
    [t.start() for t in threads]
    [t.join() for t in threads]
    assert not bad


def test_given_stream_and_outputs(osx):
    s = fresh_step(4)
    ref = step(osx, {k: v.clone() for k, v in s.items()})
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    slots, pos, lens, head, served = osx.attn_kv_plan(s["lens"], s["new"], s["table"], s["free"],
                                                      s["head"], page_size=16, n_new=2, stream=st)
    q, k, v = (torch.empty_like(t) for t in ref[5:8])
    got = osx.attn_qk_norm_rope(s["qkv"], s["w"], s["w"], s["inv"], pos, n_heads=8, n_kv_heads=2, q=q,
                                k=k, v=v, stream=st)
    assert all(a.data_ptr() == b.data_ptr() for a, b in zip(got, (q, k, v)))
    osx.attn_kv4_append(k, v, s["cache"], slots, stream=st.cuda_stream)
    o, lse = torch.empty_like(ref[8]), torch.empty_like(ref[9])
    osx.attn_kv4_fwd(q, s["cache"], s["table"], lens, q_pos=s["lens"], window=200, sinks=4, o=o,
                     lse=lse, max_len=602, stream=st)
    kv = osx.attn_kv4_read(s["cache"], s["table"], s["lens"], lens, n=3, stream=st)
    w = osx.attn_window_fwd(q, s["bk"], s["bv"], window=90, sinks=4, stream=st)
    st.synchronize()
    for a, b in zip((slots, pos, lens, head, served, q, k, v, o, lse, *kv, *w), ref):
        assert torch.equal(a, b)


def test_launches_are_counted(osx):
    s = fresh_step(6)
    n = osx.attn_launch_count()
    step(osx, s)
    # plan, norms, append, attention and its join, read, windowed attention and its join, merge
    assert osx.attn_launch_count() - n == 9


def test_offsets_beyond_32_bits(osx):
    """Pages more than 8 GB into a cache, and key rows more than 4 GB into a tensor."""
    d, Hkv, page = 128, 8, 128
    n_pages = 60000
    cache = osx.kv4_cache(n_pages, Hkv, d, page_size=page)
    assert cache.numel() > 9 << 30
    pages = [n_pages - 1, 3, n_pages - 20000]
    g = torch.Generator().manual_seed(1)
    k, v = (torch.randn((1, Hkv, 300, d), generator=g).bfloat16().cuda() for _ in range(2))
    pos = np.arange(300)
    osx.attn_kv4_append(k, v, cache, i32([np.array(pages)[pos // page] * page + pos % page]))
    table, lens = i32([pages]), i32([300])
    rk, rv = osx.attn_kv4_read(cache, table, i32([0]), lens, n=300)
    vals = [su.values(*su.quantise(su.to_np(x)[0])) for x in (k, v)]
    assert np.array_equal(su.to_np(rk)[0], su.bf16(vals[0]))
    assert np.array_equal(su.to_np(rv)[0], su.bf16(vals[1]))
    q = torch.randn((1, Hkv, 1, d), generator=g).bfloat16().cuda()
    o, lse = osx.attn_kv4_fwd(q, cache, table, lens)
    for h in range(Hkv):
        mags = [np.abs(x[h]) + 2 * np.abs(x[h]).max() for x in vals]  # at least scale c + |zero|
        ref = su.attention(su.to_np(q)[0, h], vals[0][h], vals[1][h], np.ones((1, 300), bool),
                           np.float64(np.float32(d ** -0.5)), *mags, mags[1], 2.0 ** -15)
        su.check(su.to_np(o)[0, h], su.to_np(lse)[0, h], ref, f"head {h}")
    del cache

    n = 17_500_000
    for H, Nq in ((1, 1), (1, 2000)):  # token form and tiles
        kk, vv = (torch.zeros((1, H, n, d), dtype=torch.bfloat16).cuda() for _ in range(2))
        tail = [torch.randn((1, H, 2300, d), generator=g).bfloat16() for _ in range(2)]
        kk[:, :, -2300:], vv[:, :, -2300:] = tail[0].cuda(), tail[1].cuda()
        q = torch.randn((1, H, Nq, d), generator=g).bfloat16()
        o, lse = osx.attn_window_fwd(q.cuda(), kk, vv, window=250)
        assert (osx.lib().attn_window_fwd_workspace(1, H, H, Nq, d) > 0) == (Nq == 1)
        see = su.visible(2300 - Nq + np.arange(Nq), np.arange(2300), 250, 0)
        ref = su.attention(su.to_np(q)[0, 0], su.to_np(tail[0])[0, 0], su.to_np(tail[1])[0, 0], see,
                           np.float64(np.float32(d ** -0.5)))
        su.check(su.to_np(o)[0, 0], su.to_np(lse)[0, 0], ref, f"{Nq} rows")
        del kk, vv


# --------------------------------------------------------------------------------- refusals
def test_refusals(osx):
    s = fresh_step(7)
    q = torch.zeros((5, 8, 2, 128), dtype=torch.bfloat16).cuda()
    k = torch.zeros((5, 2, 2, 128), dtype=torch.bfloat16).cuda()
    slots = torch.full((5, 2), -1, dtype=torch.int32).cuda()
    plan = dict(page_size=16, n_new=2)
    rope = dict(n_heads=8, n_kv_heads=2)
    five = [s["lens"], s["new"], s["table"], s["free"], s["head"]]

    def swap(args, i, t):
        return [t if j == i else a for j, a in enumerate(args)]

    value = []
    for i in range(5):
        value += [lambda i=i: osx.attn_kv_plan(*swap(five, i, five[i].long()), **plan),
                  lambda i=i: osx.attn_kv_plan(*swap(five, i, five[i].cpu()), **plan),
                  lambda i=i: osx.attn_kv_plan(*swap(five, i, five[i][None]), **plan)]
    ropes = [s["qkv"], s["w"], s["w"], s["inv"], slots]
    value += [
        lambda: osx.attn_kv_plan(*swap(five, 1, s["new"][:4]), **plan),
        lambda: osx.attn_kv_plan(*swap(five, 2, s["table"][:4]), **plan),
        lambda: osx.attn_kv_plan(*swap(five, 2, s["table"].t()), **plan),
        lambda: osx.attn_kv_plan(*swap(five, 0, s["lens"][:0]), **plan),
        lambda: osx.attn_kv_plan(*five, page_size=0, n_new=2),
        lambda: osx.attn_kv_plan(*five, page_size=16, n_new=0),
        lambda: osx.attn_qk_norm_rope(*swap(ropes, 0, s["qkv"].float()), **rope),
        lambda: osx.attn_qk_norm_rope(*swap(ropes, 0, s["qkv"][0]), **rope),
        lambda: osx.attn_qk_norm_rope(*swap(ropes, 0, s["qkv"].transpose(1, 2)), **rope),
        lambda: osx.attn_qk_norm_rope(*swap(ropes, 1, s["w"].half()), **rope),
        lambda: osx.attn_qk_norm_rope(*swap(ropes, 2, s["w"].float()), **rope),
        lambda: osx.attn_qk_norm_rope(*swap(ropes, 2, s["w"][:64]), **rope),
        lambda: osx.attn_qk_norm_rope(*swap(ropes, 3, s["inv"].double()), **rope),
        lambda: osx.attn_qk_norm_rope(*swap(ropes, 3, torch.cat([s["inv"], s["inv"]])), **rope),
        lambda: osx.attn_qk_norm_rope(*swap(ropes, 3, s["inv"][:0]), **rope),
        lambda: osx.attn_qk_norm_rope(*swap(ropes, 4, slots.long()), **rope),
        lambda: osx.attn_qk_norm_rope(*swap(ropes, 4, slots[:, :1]), **rope),
        lambda: osx.attn_qk_norm_rope(*ropes, n_heads=7, n_kv_heads=2),
        lambda: osx.attn_qk_norm_rope(*ropes, n_heads=0, n_kv_heads=6),
        lambda: osx.attn_qk_norm_rope(*ropes, **rope, q=k),
        lambda: osx.attn_kv4_append(k.float(), k, s["cache"], slots),
        lambda: osx.attn_kv4_append(k, k[:, :, :1], s["cache"], slots),
        lambda: osx.attn_kv4_append(q, q, s["cache"], slots),
        lambda: osx.attn_kv4_append(k, k, s["cache"].int(), slots),
        lambda: osx.attn_kv4_append(k, k, s["cache"][..., :1000], slots),
        lambda: osx.attn_kv4_append(k, k, s["cache"], slots[:4]),
        lambda: osx.attn_kv4_append(k.transpose(2, 3), k, s["cache"], slots),
        lambda: osx.attn_kv4_read(s["cache"], s["table"], s["lens"], s["lens"][:2], n=2),
        lambda: osx.attn_kv4_read(s["cache"], s["table"], s["lens"], s["lens"], n=0),
        lambda: osx.attn_kv4_read(s["cache"], s["table"].long(), s["lens"], s["lens"], n=2),
        lambda: osx.attn_kv4_fwd(q.float(), s["cache"], s["table"], s["lens"]),
        lambda: osx.attn_kv4_fwd(q[..., :64], s["cache"], s["table"], s["lens"]),
        lambda: osx.attn_kv4_fwd(q[:, :7], s["cache"], s["table"], s["lens"]),
        lambda: osx.attn_kv4_fwd(q, s["cache"], s["table"][:3], s["lens"]),
        lambda: osx.attn_kv4_fwd(q, s["cache"], s["table"], s["lens"], q_pos=slots),
        lambda: osx.attn_kv4_fwd(q, s["cache"], s["table"], s["lens"], o_dtype=torch.float16),
        lambda: osx.attn_kv4_fwd(q, s["cache"], s["table"], s["lens"], o=q.half()),
        lambda: osx.attn_kv4_fwd(q, s["cache"], s["table"], s["lens"], window=2 ** 40),
        lambda: osx.attn_window_fwd(q, k.float(), k, window=4),
        lambda: osx.attn_window_fwd(q, k, k[:, :1], window=4),
        lambda: osx.attn_window_fwd(q, k[:4], k[:4], window=4),
        lambda: osx.attn_window_fwd(q, k[:, :, :1].contiguous(), k[:, :, :1].contiguous(), window=4),
        lambda: osx.attn_window_fwd(q, k, k, window=4, kv_len=3),
        lambda: osx.attn_window_fwd(q, k, k, window=4, kv_len=0),
        lambda: osx.attn_window_fwd(q, k, k, window=4, lse=q),
    ]
    n = osx.attn_launch_count()
    for i, fn in enumerate(value):
        with pytest.raises(ValueError):
            fn()
            pytest.fail(f"case {i} was taken")
    status = [
        (osx.ATTN_ERR_UNSUPPORTED, lambda: osx.attn_qk_norm_rope(*swap(ropes, 3, s["inv"][:12]), **rope)),
        (osx.ATTN_ERR_INVALID_ARG, lambda: osx.attn_qk_norm_rope(*ropes, **rope, eps=-1.0)),
        (osx.ATTN_ERR_INVALID_ARG, lambda: osx.attn_kv4_fwd(q, s["cache"], s["table"], s["lens"], scale=0.0)),
        (osx.ATTN_ERR_INVALID_ARG, lambda: osx.attn_kv4_fwd(q, s["cache"], s["table"], s["lens"], window=-1)),
        (osx.ATTN_ERR_INVALID_ARG, lambda: osx.attn_kv4_fwd(q, s["cache"], s["table"], s["lens"], sinks=-1)),
        (osx.ATTN_ERR_INVALID_ARG, lambda: osx.attn_kv4_fwd(q, s["cache"], s["table"], s["lens"], max_len=-1)),
        (osx.ATTN_ERR_INVALID_ARG, lambda: osx.attn_kv4_fwd(q, s["cache"], s["table"], s["lens"],
                                                            o=q)),  # onto the queries
        (osx.ATTN_ERR_INVALID_ARG, lambda: osx.attn_window_fwd(q, k, k, window=0)),
        (osx.ATTN_ERR_INVALID_ARG, lambda: osx.attn_window_fwd(q, k, k, window=4, q_off=-1)),
        (osx.ATTN_ERR_INVALID_ARG, lambda: osx.attn_window_fwd(q, k, k, window=4, scale=float("nan"))),
        (osx.ATTN_ERR_INVALID_ARG, lambda: osx.attn_window_fwd(q, k, k, window=4, o=q)),
        (osx.ATTN_ERR_UNSUPPORTED, lambda: osx.attn_window_fwd(q[..., :32].contiguous(), k[..., :32].contiguous(),
                                                               k[..., :32].contiguous(), window=4)),
    ]
    for i, (want, fn) in enumerate(status):
        with pytest.raises(osx.AttnError) as e:
            fn()
            pytest.fail(f"case {i} was taken")
        assert e.value.status == want, i
    assert osx.attn_launch_count() == n


def test_injected_failure(osx):
    k = torch.zeros((1, 1, 1, 64), dtype=torch.bfloat16).cuda()
    osx.attn_debug_inject(osx.ATTN_ERR_INJECTED, 1)
    with pytest.raises(osx.AttnError) as e:
        osx.attn_window_fwd(k, k.clone(), k.clone(), window=1)
    assert e.value.status == osx.ATTN_ERR_INJECTED
    osx.attn_window_fwd(k, k.clone(), k.clone(), window=1)
    torch.cuda.synchronize()
