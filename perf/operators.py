"""The serving operators' cases: what is timed, on which inputs, and the plain form of each.

The operators are those of a decoder layer that serves long contexts:

  plan    pages and slots for the tokens that a batch of requests is about to add
  rope    norms of queries and keys for each head with the position rotation, from the packed
          projection to the head-major tensors that attention takes
  append  new keys and values into the paged 4-bit cache, and the same tokens read back
  cache   attention of the newest tokens over the paged 4-bit cache
  window  attention with a sliding window and a few first tokens that stay visible

``run`` computes them in elementary torch operations, or with ``own`` set by the calls that a
user makes. ``exact`` computes them from their definitions in 64 bits.
"""

from __future__ import annotations

import math

import torch

own = False

GROUP = 32   # values along d that share one scale and one zero point in the 4-bit cache
BLOCK = 16   # tokens of one block of the 4-bit cache


# ------------------------------------------------------------------------------- the cases
def listed():
    return [
        # a decode step of 32 requests: one token each
        dict(name="plan_token", op="plan", B=32, N=1, page=16, width=512),
        # prompts of many requests arriving together, up to 256 tokens each
        dict(name="plan_prompts", op="plan", B=512, N=256, page=16, width=512),
        # a decode step of 32 requests
        dict(name="rope_token", op="rope", B=32, N=1, Hq=32, Hkv=8, d=128, rot=128, inter=False),
        # a prompt of the length of one ring step's sequence
        dict(name="rope_prompt", op="rope", B=1, N=32768, Hq=32, Hkv=8, d=128, rot=128,
             inter=False),
        # a decode step of 64 requests
        dict(name="append_token", op="append", B=64, N=1, Hkv=8, d=128, page=16, width=64),
        # four ragged prompts of up to 8192 tokens
        dict(name="append_prompt", op="append", B=4, N=8192, Hkv=8, d=128, page=64, width=160),
        # a few short chats at head size 64, three drafted tokens each, windowed
        dict(name="cache_short", op="cache", B=3, Nq=3, Hq=16, Hkv=4, d=64, page=16, width=44,
             longest=700, window=256, sinks=4),
        # a ragged batch of 32 requests, one token each
        dict(name="cache_batch", op="cache", B=32, Nq=1, Hq=32, Hkv=8, d=128, page=16, width=512,
             longest=8192, window=0, sinks=0),
        # one token against the whole 128k-token context
        dict(name="cache_long", op="cache", B=1, Nq=1, Hq=32, Hkv=8, d=128, page=64, width=2048,
             longest=131072, window=0, sinks=0),
        # one token over the last 4096 of 8192 bf16 keys
        dict(name="window_token", op="window", B=4, Nq=1, Nkv=8192, Hq=32, Hkv=8, d=128,
             window=4096, sinks=4),
        # two prompts of an odd length just under 4k
        dict(name="window_4k", op="window", B=2, Nq=4001, Nkv=4001, Hq=16, Hkv=16, d=128,
             window=1024, sinks=4),
        # a 32k prompt with grouped heads
        dict(name="window_32k", op="window", B=1, Nq=32768, Nkv=32768, Hq=32, Hkv=8, d=128,
             window=1024, sinks=64),
    ]


def _log(rng, lo, hi):
    """A whole number whose logarithm is spread evenly over [lo, hi]."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


_HEADS = [(32, 8), (16, 16), (32, 32), (16, 4), (8, 1), (16, 2), (12, 4)]


def draw(rng):
    op = rng.choice(["plan", "rope", "append", "cache", "window"])
    d = rng.choice([64, 128])
    Hq, Hkv = rng.choice(_HEADS)
    page = rng.choice([16, 32, 64, 128])
    if op == "plan":
        B = _log(rng, 1, 512)
        N = _log(rng, 1, min(2048, 131072 // B))
        return dict(op=op, B=B, N=N, page=page, width=8192 // page)
    if op == "rope":
        B = _log(rng, 1, 64)
        N = _log(rng, 1, max(1, 32768 * 48 * 128 // (B * (Hq + 2 * Hkv) * d)))
        return dict(op=op, B=B, N=min(N, 32768), Hq=Hq, Hkv=Hkv, d=d,
                    rot=rng.choice([d, d // 2]), inter=rng.choice([False, True]))
    if op == "append":
        B = _log(rng, 1, 64)
        N = _log(rng, 1, max(1, 32768 * 8 * 128 // (B * Hkv * d)))
        N = min(N, 8192)
        return dict(op=op, B=B, N=N, Hkv=Hkv, d=d, page=page, width=-(-(N + 1500) // page))
    if op == "cache":
        B = _log(rng, 1, 48)
        most = 131072 * 8 * 128 // (B * Hkv * d)
        longest = _log(rng, 40, min(131072, most))
        window = rng.choice([0, 0, _log(rng, 16, 8192)])
        return dict(op=op, B=B, Nq=rng.choice([1, 1, 1, 2, 5]), Hq=Hq, Hkv=Hkv, d=d, page=page,
                    width=-(-longest // page), longest=longest, window=window,
                    sinks=rng.choice([0, 4, 130]) if window else 0)
    window = _log(rng, 32, 4096)
    sinks = rng.choice([0, 1, 4, 64, 200])
    if rng.random() < 0.3:  # newest tokens over a long context
        B = _log(rng, 1, 16)
        Nkv = _log(rng, 64, 32768)
        Nq = min(Nkv, rng.choice([1, 1, 2, 7]))
    else:
        B = rng.choice([1, 1, 2, 3])
        Nq = _log(rng, 64, min(32768, 32768 * 32 * 1024 // (B * Hq * window)))
        Nkv = Nq + rng.choice([0, 0, _log(rng, 1, 2048)])
    return dict(op=op, B=B, Nq=Nq, Nkv=Nkv, Hq=Hq, Hkv=Hkv, d=d, window=window, sinks=sinks)


# ------------------------------------------------------------------------------ the inputs
def _lengths(gen, n, lo, hi):
    """n request lengths in [lo, hi], ragged, the longest among them."""
    x = torch.randint(lo, hi + 1, (n,), generator=gen, device="cuda", dtype=torch.int32)
    x[torch.randint(0, n, (1,), generator=gen, device="cuda")] = hi
    return x


def _codes_words(codes, d, which):
    """Codes [..., 16, d] of one block's tokens to the block's words [..., 2 * d] (int32).

    A word holds eight 4-bit codes, the first in its low bits. Keys: word (r, g, t, i) (at d = 64
    word (g, t, r, i)) holds token 8r + g, values 32i + 8t + e; values: word (h, g, t, b, a) holds
    token 8b + 2t + a, values 64h + 8e + g (e = 0..7).
    """
    lead = codes.shape[:-2]
    n = len(lead)
    if which == "k":
        c = codes.reshape(*lead, 2, 8, d // 32, 4, 8)               # r g i t e
        order = (0, 1, 3, 2, 4) if d == 128 else (1, 3, 0, 2, 4)    # -> words, e last
    else:
        c = codes.reshape(*lead, 2, 4, 2, d // 64, 8, 8)            # b t a h e g
        order = (3, 5, 1, 0, 2, 4)                                  # -> h g t b a, e
    c = c.permute(*range(n), *(n + x for x in order)).reshape(*lead, 2 * d, 8)
    shift = torch.arange(0, 32, 4, device=codes.device)
    w = (c.long() << shift).sum(-1)
    return torch.where(w >= 1 << 31, w - (1 << 32), w).to(torch.int32)


def _words_codes(words, d, which):
    """The inverse: words [..., 2 * d] to codes [..., 16, d] (int32, 0..15)."""
    lead = words.shape[:-1]
    n = len(lead)
    shift = torch.arange(0, 32, 4, device=words.device, dtype=torch.int32)
    c = (words[..., None] >> shift) & 15
    if which == "k":
        if d == 128:
            c = c.reshape(*lead, 2, 8, 4, 4, 8)     # r g t i e
            order = (0, 1, 3, 2, 4)
        else:
            c = c.reshape(*lead, 8, 4, 2, 2, 8)     # g t r i e
            order = (2, 0, 3, 1, 4)
    else:
        c = c.reshape(*lead, d // 64, 8, 4, 2, 2, 8)  # h g t b a e
        order = (3, 2, 4, 0, 5, 1)
    return c.permute(*range(n), *(n + x for x in order)).reshape(*lead, BLOCK, d)


def _quantise(x):
    """bf16 [..., d] to (codes 0..15 int32 [..., d], scale, zero fp32 [..., d / 32])."""
    g = x.float().unflatten(-1, (-1, GROUP))
    lo, hi = g.amin(-1, keepdim=True), g.amax(-1, keepdim=True)
    scale = ((hi - lo) / 15).bfloat16().float()
    c = torch.where(scale > 0, torch.round((g - lo) / torch.where(scale > 0, scale, 1.0)), 0.0)
    return c.clamp(0, 15).int().flatten(-2), scale.squeeze(-1), lo.squeeze(-1)


def _params_words(scale, zero):
    """bf16 scale (low half) and zero point (high half) of each group as one int32."""
    s = scale.bfloat16().view(torch.int16).int() & 0xffff
    z = zero.bfloat16().view(torch.int16).int()
    return s | (z << 16)


def _fill_cache(gen, n_pages, Hkv, page, d):
    """A cache whose pages hold normal keys (with a few large channels) and values."""
    blocks = page // BLOCK
    cache = torch.empty((n_pages, Hkv, blocks, 20 * d), dtype=torch.uint8, device="cuda")
    words = cache.view(torch.int32)
    step = max(1, (1 << 25) // (Hkv * page * d))
    at = 0
    for which in ("k", "v"):
        for p in range(0, n_pages, step):
            n = min(step, n_pages - p)
            x = torch.randn((n, Hkv, blocks, BLOCK, d), generator=gen, device="cuda")
            if which == "k":
                x[..., 3::41] *= 4
            c, s, z = _quantise(x.bfloat16())
            words[p:p + n, ..., at:at + 2 * d] = _codes_words(c, d, which)
            pa = 4 * d + (0 if which == "k" else d // 2)
            words[p:p + n, ..., pa:pa + d // 2] = _params_words(s, z).flatten(-2)
        at += 2 * d
    return cache


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    op, B = case["op"], case["B"]

    def normal(*shape):
        return torch.randn(shape, generator=gen, device="cuda").bfloat16()

    s = dict(case=case)
    if op == "plan":
        N, page, width = case["N"], case["page"], case["width"]
        room = width * page - N
        s["lens"] = _lengths(gen, B, 0, room)
        s["new"] = _lengths(gen, B, 1, N) if N > 1 else torch.ones_like(s["lens"])
        total = B * width
        perm = torch.randperm(2 * total, generator=gen, device="cuda").int()
        held = -(-s["lens"] // page)
        at = torch.arange(width, device="cuda")
        s["table"] = torch.where(at < held[:, None], perm[:total].view(B, width), -1).int()
        s["free"] = perm[total:].contiguous()
        s["head"] = torch.randint(0, 1 + total // 8, (1,), generator=gen, device="cuda",
                                  dtype=torch.int32)
    elif op == "rope":
        N, Hq, Hkv, d = case["N"], case["Hq"], case["Hkv"], case["d"]
        s["qkv"] = normal(B, N, (Hq + 2 * Hkv) * d)
        s["wq"] = (1 + 0.2 * torch.randn(d, generator=gen, device="cuda")).bfloat16()
        s["wk"] = (1 + 0.2 * torch.randn(d, generator=gen, device="cuda")).bfloat16()
        r = case["rot"]
        s["inv"] = 500000.0 ** (-torch.arange(0, r, 2, device="cuda").float() / r)
        start = torch.randint(0, 131072 - N, (B, 1), generator=gen, device="cuda",
                              dtype=torch.int32)
        s["pos"] = start + torch.arange(N, device="cuda", dtype=torch.int32)
    elif op == "append":
        N, Hkv, d, page, width = (case[k] for k in ("N", "Hkv", "d", "page", "width"))
        s["k"], s["v"] = normal(B, Hkv, N, d), normal(B, Hkv, N, d)
        s["k"][..., 3::41] *= 4
        s["start"] = _lengths(gen, B, 0, min(1000, width * page - N))
        new = _lengths(gen, B, (N + 1) // 2, N)
        s["lens"] = s["start"] + new
        n_pages = B * width + 7
        s["table"] = torch.randperm(n_pages, generator=gen, device="cuda")[:B * width].int() \
            .view(B, width)
        pos = s["start"][:, None] + torch.arange(N, device="cuda")
        at = s["table"].gather(1, (pos // page).clamp(max=width - 1)) * page + pos % page
        s["slots"] = torch.where(pos < s["lens"][:, None], at, -1).int()
        s["cache"] = _fill_cache(gen, n_pages, Hkv, page, d)
    elif op == "cache":
        Nq, Hq, Hkv, d, page, width = (case[k] for k in ("Nq", "Hq", "Hkv", "d", "page", "width"))
        s["lens"] = _lengths(gen, B, max(Nq, case["longest"] // 3), case["longest"])
        n_pages = B * width + 3
        s["table"] = torch.randperm(n_pages, generator=gen, device="cuda")[:B * width].int() \
            .view(B, width)
        s["cache"] = _fill_cache(gen, n_pages, Hkv, page, d)
        s["q"] = normal(B, Hq, Nq, d)
    else:
        Nq, Nkv, Hq, Hkv, d = (case[k] for k in ("Nq", "Nkv", "Hq", "Hkv", "d"))
        s["q"], s["k"], s["v"] = normal(B, Hq, Nq, d), normal(B, Hkv, Nkv, d), normal(B, Hkv, Nkv, d)
    return s


# ------------------------------------------------------------------------- the plain forms
def _softmax_parts(s):
    """(p, l, lse) of masked scores s (-inf where masked), rows without a key included."""
    m = s.amax(-1, keepdim=True)
    base = torch.where(m == -math.inf, 0.0, m)
    p = torch.exp(s - base)
    l = p.sum(-1, keepdim=True)
    return p, l, (base + torch.log(l)).squeeze(-1)


def _plain_plan(s):
    c = s["case"]
    page, N = c["page"], c["N"]
    lens, new, table = s["lens"].long(), s["new"].long(), s["table"]
    width = table.shape[1]
    held, want = (lens + page - 1) // page, (lens + new + page - 1) // page
    fits = want <= width
    need = torch.where(fits, want - held, 0)
    ends = need.cumsum(0)
    served = fits & ((need == 0) | (s["head"] + ends <= s["free"].numel()))
    at = torch.arange(width, device=table.device)
    fresh = served[:, None] & (at >= held[:, None]) & (at < want[:, None])
    take = s["head"] + (ends - need)[:, None] + at - held[:, None]
    table = torch.where(fresh, s["free"][take.clamp(0, s["free"].numel() - 1)], table)
    i = torch.arange(N, device=table.device)
    pos = lens[:, None] + i
    put = served[:, None] & (i < new[:, None])
    slot = table.gather(1, (pos // page).clamp(max=width - 1)) * page + pos % page
    out = torch.where(served, lens + new, lens).int()
    head = s["head"] + torch.where(served, need, 0).sum().int()
    return torch.where(put, slot, -1).int(), pos.int(), out, head, served.int(), table


def _plain_rope(s):
    c = s["case"]
    B, N, Hq, Hkv, d, r = (c[k] for k in ("B", "N", "Hq", "Hkv", "d", "rot"))
    x = s["qkv"].view(B, N, Hq + 2 * Hkv, d)
    a = s["pos"].double()[..., None] * s["inv"].double()          # far positions: in 64 bits
    cos, sin = torch.cos(a).float()[:, :, None], torch.sin(a).float()[:, :, None]

    def turned(h, w):
        h = h.float()
        h = h * torch.rsqrt(h.square().mean(-1, keepdim=True) + 1e-6) * w.float()
        t, rest = h[..., :r], h[..., r:]
        if c["inter"]:
            u, v = t[..., 0::2], t[..., 1::2]
            t = torch.stack([u * cos - v * sin, v * cos + u * sin], -1).flatten(-2)
        else:
            u, v = t[..., :r // 2], t[..., r // 2:]
            t = torch.cat([u * cos - v * sin, v * cos + u * sin], -1)
        return torch.cat([t, rest], -1).bfloat16().transpose(1, 2).contiguous()

    return (turned(x[:, :, :Hq], s["wq"]), turned(x[:, :, Hq:Hq + Hkv], s["wk"]),
            x[:, :, Hq + Hkv:].transpose(1, 2).contiguous())


def _gather_cache(cache, table, d):
    """Keys and values fp32 [B, Hkv, tokens, d] that the table's pages stand for."""
    w = cache.view(torch.int32)[table.long()]                     # B P Hkv blocks words
    out = []
    for which, at, pa in (("k", 0, 4 * d), ("v", 2 * d, 4 * d + d // 2)):
        c = _words_codes(w[..., at:at + 2 * d], d, which).float()  # B P Hkv blocks 16 d
        p = w[..., pa:pa + d // 2].unflatten(-1, (BLOCK, d // GROUP)).contiguous()
        p = p.view(torch.bfloat16).unflatten(-1, (-1, 2)).float()  # ... 16 groups (scale, zero)
        x = c.unflatten(-1, (-1, GROUP)) * p[..., 0:1] + p[..., 1:2]
        x = x.flatten(-2).permute(0, 2, 1, 3, 4, 5)
        out.append(x.reshape(x.shape[0], x.shape[1], -1, d))
    return out


def _plain_append(s):
    c = s["case"]
    B, N, Hkv, d, page = (c[k] for k in ("B", "N", "Hkv", "d", "page"))
    words = s["cache"].view(torch.int32)
    blocks, per = page // BLOCK, 5 * d
    slots = s["slots"].long()
    put = slots >= 0
    b, i = put.nonzero(as_tuple=True)
    slot = slots[b, i]
    head = torch.arange(Hkv, device="cuda")
    base = (((slot // page)[:, None] * Hkv + head) * blocks + (slot % page // BLOCK)[:, None]) * per
    row = slot % BLOCK
    flat = words.view(-1)
    t, g8 = torch.arange(4, device="cuda"), torch.arange(8, device="cuda")
    gi, h2 = torch.arange(d // 32, device="cuda"), torch.arange(d // 64, device="cuda")
    shift = torch.arange(0, 32, 4, device="cuda")
    for which, x in (("k", s["k"]), ("v", s["v"])):
        q, scale, zero = _quantise(x[b, :, i])                    # tokens Hkv d
        if which == "k":
            q = q.view(-1, Hkv, d // 32, 4, 8).transpose(2, 3)    # t i e
            r, g = row // 8, row % 8
            if d == 128:
                at = ((r * 8 + g)[:, None, None] * 4 + t[:, None]) * 4 + gi
            else:
                at = ((g[:, None, None] * 4 + t[:, None]) * 2 + r[:, None, None]) * 2 + gi
            pa = 4 * d
        else:
            q = q.view(-1, Hkv, d // 64, 8, 8).transpose(3, 4)    # h g e
            bb, tt, aa = row // 8, row % 8 // 2, row % 2
            at = 2 * d + (h2[:, None] * 32 + g8 * 4)[None] * 4 + \
                (tt * 4 + bb * 2 + aa)[:, None, None]
            pa = 4 * d + d // 2
        w = (q.long() << shift).sum(-1).flatten(2)
        w = torch.where(w >= 1 << 31, w - (1 << 32), w).int()
        flat[base[:, :, None] + at.flatten(1)[:, None]] = w
        flat[base[:, :, None] + pa + row[:, None, None] * (d // 32) + gi] = \
            _params_words(scale, zero)
    return _plain_read(s)


def _plain_read(s):
    """The tokens [start, lens) of each request as bf16 [B, Hkv, N, d], zeros behind them."""
    c = s["case"]
    N, d, page, Hkv = c["N"], c["d"], c["page"], c["Hkv"]
    pos = s["start"].long()[:, None] + torch.arange(N, device="cuda")
    real = pos < s["lens"][:, None]
    pages = N // page + 2                                         # that N tokens can touch
    first = s["start"].long() // page
    some = (first[:, None] + torch.arange(pages, device="cuda")).clamp(max=c["width"] - 1)
    out = []
    for x in _gather_cache(s["cache"], s["table"].gather(1, some), d):
        at = (pos - first[:, None] * page).clamp(max=pages * page - 1)
        x = x.gather(2, at[:, None, :, None].expand(-1, Hkv, -1, d))
        out.append(torch.where(real[:, None, :, None], x, 0.0).bfloat16())
    return tuple(out)


def _plain_cache(s):
    c = s["case"]
    B, Nq, Hq, Hkv, d = (c[k] for k in ("B", "Nq", "Hq", "Hkv", "d"))
    k, v = _gather_cache(s["cache"], s["table"], d)
    L = k.shape[2]
    q = s["q"].float().view(B, Hkv, -1, d)                        # rows: (head of the group, token)
    sc = torch.matmul(q, k.transpose(-1, -2)) * d ** -0.5
    key = torch.arange(L, device="cuda")
    pos = (s["lens"].long()[:, None] - Nq + torch.arange(Nq, device="cuda"))[..., None]
    see = (key <= pos) & (key < s["lens"][:, None, None])
    if c["window"]:
        see &= (key > pos - c["window"]) | (key < c["sinks"])
    sc = sc.view(B, Hkv, -1, Nq, L).masked_fill(~see[:, None, None], -math.inf)
    p, l, lse = _softmax_parts(sc.view(B, Hkv, -1, L))
    o = torch.matmul(p, v) / torch.where(l > 0, l, 1.0)
    return o.view(B, Hq, Nq, d).bfloat16(), lse.view(B, Hq, Nq)


def _plain_window(s):
    c = s["case"]
    B, Nq, Nkv, Hq, Hkv, d, W = (c[k] for k in ("B", "Nq", "Nkv", "Hq", "Hkv", "d", "window"))
    S = min(c["sinks"], Nkv)
    G, off = Hq // Hkv, Nkv - Nq
    # the rows in blocks of C, each against the band of keys that its rows can see
    C = min(max(W, 64), Nq)
    n = -(-Nq // C)
    q = torch.nn.functional.pad(s["q"].float(), (0, 0, 0, n * C - Nq))
    q = q.view(B, Hkv, G, n, C, d).transpose(2, 3).reshape(B, Hkv, n, G * C, d)
    k, v = s["k"].float(), s["v"].float()
    row = off + torch.arange(n * C, device="cuda").view(n, C)     # the rows' positions
    key = row[:, :1] - W + 1 + torch.arange(C + W - 1, device="cuda")  # n, C + W - 1
    at = key.clamp(0, Nkv - 1)
    see = (key[:, None] >= 0) & (key[:, None] <= row[..., None]) & (key[:, None] > row[..., None] - W) \
        & (key[:, None] < Nkv)
    sc = torch.matmul(q, k[:, :, at].transpose(-1, -2)).view(B, Hkv, n, G, C, -1)
    first = torch.arange(S, device="cuda")
    old = first <= row[..., None] - W                             # not in the window already
    ss = torch.matmul(q, k[:, :, None, :S].transpose(-1, -2)).view(B, Hkv, n, G, C, -1)
    sc = torch.cat([ss.masked_fill(~old[:, None], -math.inf),
                    sc.masked_fill(~see[:, None], -math.inf)], -1) * d ** -0.5
    del ss
    p, l, lse = _softmax_parts(sc)
    del sc
    p = p.view(B, Hkv, n, G * C, -1)
    o = torch.matmul(p[..., S:], v[:, :, at]) + torch.matmul(p[..., :S], v[:, :, None, :S])
    o = o.view(B, Hkv, n, G, C, d) / torch.where(l > 0, l, 1.0)
    o = o.transpose(2, 3).reshape(B, Hq, n * C, d)[:, :, :Nq].bfloat16()
    return o.contiguous(), lse.transpose(2, 3).reshape(B, Hq, n * C)[:, :, :Nq].contiguous()


# ------------------------------------------------------------------------------- the passes
def run(state):
    s, c = state, state["case"]
    op = c["op"]
    if own:
        import online_softmax_exact_b200 as osx

        if op == "plan":
            out = osx.attn_kv_plan(s["lens"], s["new"], s["table"], s["free"], s["head"],
                                   page_size=c["page"], n_new=c["N"])
            return (*out, s["table"])
        if op == "rope":
            return osx.attn_qk_norm_rope(s["qkv"], s["wq"], s["wk"], s["inv"], s["pos"],
                                         n_heads=c["Hq"], n_kv_heads=c["Hkv"], eps=1e-6,
                                         interleaved=c["inter"])
        if op == "append":
            osx.attn_kv4_append(s["k"], s["v"], s["cache"], s["slots"])
            return osx.attn_kv4_read(s["cache"], s["table"], s["start"], s["lens"], n=c["N"])
        if op == "cache":
            return osx.attn_kv4_fwd(s["q"], s["cache"], s["table"], s["lens"],
                                    window=c["window"], sinks=c["sinks"],
                                    o_dtype=torch.bfloat16)
        return osx.attn_window_fwd(s["q"], s["k"], s["v"], window=c["window"], sinks=c["sinks"],
                                   o_dtype=torch.bfloat16)
    return {"plan": _plain_plan, "rope": _plain_rope, "append": _plain_append,
            "cache": _plain_cache, "window": _plain_window}[op](s)


# --------------------------------------------------------------------- floors of the passes
def _seen(n_rows, first, n_keys, window, sinks):
    """Pairs (row, key) that n_rows rows at positions first, first + 1, ... see."""
    total = 0
    for i in range(n_rows):
        p = first + i
        hi = min(p, n_keys - 1) + 1
        lo = max(0, p - window + 1) if window else 0
        total += max(0, hi - lo) + min(sinks if window else 0, lo, hi)
    return total


def work(case):
    c = case
    op, B = c["op"], c["B"]
    if op == "plan":
        # lengths, the table entries that the new tokens need, slots and positions
        return dict(bytes=B * (4 * 5 + c["N"] * 8 + 8 * (c["N"] / c["page"] + 1)), flops=0)
    if op == "rope":
        x = B * c["N"] * (c["Hq"] + 2 * c["Hkv"]) * c["d"]
        return dict(bytes=4 * x + 4 * B * c["N"],
                    flops=9 * B * c["N"] * (c["Hq"] + c["Hkv"]) * c["d"])
    if op == "append":
        # three quarters of the rows hold tokens; read bf16, write 5 bits a value, then back
        x = 2 * B * c["N"] * c["Hkv"] * c["d"]
        return dict(bytes=0.75 * x * (2 + 0.625 + 0.625) + 2 * x, flops=4 * x)
    if op == "cache":
        mean = 2 * c["longest"] // 3
        w = min(mean, c["window"] + c["sinks"]) if c["window"] else mean
        if B == 1:
            w = min(c["longest"], c["window"] + c["sinks"]) if c["window"] else c["longest"]
        return dict(bytes=B * (w + c["Nq"] - 1) * c["Hkv"] * c["d"] * 1.25
                    + 4 * B * c["Hq"] * c["Nq"] * (c["d"] + 1),
                    flops=4 * B * c["Hq"] * c["Nq"] * c["d"] * w)
    off = c["Nkv"] - c["Nq"]
    pairs = _seen(c["Nq"], off, c["Nkv"], c["window"], c["sinks"])
    keys = min(c["Nkv"], c["Nq"] + c["window"] - 1 + c["sinks"])
    return dict(bytes=4 * B * c["Hq"] * c["Nq"] * (c["d"] + 1) + 4 * B * c["Hkv"] * keys * c["d"],
                flops=4 * B * c["Hq"] * c["d"] * pairs)


# ----------------------------------------------------------------- the definitions in 64 bits
def _exact_rows(q, k, v, see, scale):
    """One head's rows against its keys by the definition: q [n, d], k, v [m, d], see [n, m]."""
    s = (q @ k.T * scale).masked_fill(~see, -math.inf)
    lse = torch.logsumexp(s, -1)
    p = torch.exp(s - torch.where(lse == -math.inf, 0.0, lse)[:, None])
    return p @ v, lse


def _exact_value(block, d, which, token):
    """The d values of one token of a block (bytes, numpy) by the layout's definition."""
    import numpy as np

    words = block.view(np.uint32)
    at = 0 if which == "k" else 2 * d
    e = np.arange(d)
    if which == "k":
        i, t, n = e // 32, e % 32 // 8, e % 8
        r, g = token // 8, token % 8
        w = (r * 32 + g * 4 + t) * 4 + i if d == 128 else ((g * 4 + t) * 2 + r) * 2 + i
    else:
        h, n, g = e // 64, e % 64 // 8, e % 8
        w = (h * 32 + g * 4 + token % 8 // 2) * 4 + token // 8 * 2 + token % 2
    code = (words[..., at + w] >> (4 * n).astype(np.uint32)) & 15
    pa = 4 * d + (0 if which == "k" else d // 2) + token * (d // 32) + e // 32
    p = words[..., pa]
    scale = (p << np.uint32(16)).view(np.float32).astype(np.float64)
    zero = (p & np.uint32(0xffff0000)).view(np.float32).astype(np.float64)
    return code * scale + zero


def _exact_keys(cache, table, n, page, d):
    """Keys and values fp64 [Hkv, n, d] of one request's first n tokens."""
    import numpy as np

    pages = -(-n // page)
    c = cache[table[:pages].long()].cpu().numpy()                 # pages Hkv blocks bytes
    out = []
    for which in ("k", "v"):
        x = np.stack([_exact_value(c, d, which, t) for t in range(BLOCK)], 3)
        x = x.transpose(1, 0, 2, 3, 4).reshape(c.shape[1], -1, d)[:, :n]
        out.append(torch.from_numpy(np.ascontiguousarray(x)).cuda())
    return out


def exact(case, seed):
    c, op = case, case["op"]
    if op == "plan":
        return None                                               # whole numbers
    s = prepare(case, seed)
    B, d = c["B"], c["d"]
    if op == "rope":
        N, Hq, Hkv, r = c["N"], c["Hq"], c["Hkv"], c["rot"]
        x = s["qkv"].view(B, N, Hq + 2 * Hkv, d).permute(0, 2, 1, 3)
        a = s["pos"].double()[:, None, :, None] * s["inv"].double()
        turn = torch.polar(torch.ones_like(a), a)                 # a rotation is a product

        def one(h, w):
            h = h.double()
            h = h / (h.pow(2).sum(-1, keepdim=True) / d + 1e-6).sqrt() * w.double()
            if c["inter"]:
                z = torch.view_as_complex(h[..., :r].unflatten(-1, (-1, 2)).contiguous()) * turn
                y = torch.view_as_real(z).flatten(-2)
            else:
                z = torch.complex(h[..., :r // 2], h[..., r // 2:r]) * turn
                y = torch.cat([z.real, z.imag], -1)
            return torch.cat([y, h[..., r:]], -1)

        return one(x[:, :Hq], s["wq"]), one(x[:, Hq:Hq + Hkv], s["wk"]), x[:, Hq + Hkv:].double()
    if op == "append":
        out = []
        for x in (s["k"], s["v"]):
            g = x.double().unflatten(-1, (-1, GROUP))
            lo, hi = g.amin(-1, keepdim=True), g.amax(-1, keepdim=True)
            scale = ((hi - lo) / 15).bfloat16().double()
            code = ((g - lo) / scale).round().clamp(0, 15)
            y = torch.where(scale > 0, code * scale + lo, lo).flatten(-2)
            put = (s["slots"] >= 0)[:, None, :, None]
            out.append(torch.where(put, y, 0.0))
        return tuple(out)
    if op == "cache":
        Nq, Hq, Hkv = c["Nq"], c["Hq"], c["Hkv"]
        o = torch.empty((B, Hq, Nq, d), dtype=torch.float64, device="cuda")
        lse = torch.empty((B, Hq, Nq), dtype=torch.float64, device="cuda")
        for b in range(B):
            n = int(s["lens"][b])
            k, v = _exact_keys(s["cache"], s["table"][b], n, c["page"], d)
            pos = n - Nq + torch.arange(Nq, device="cuda")[:, None]
            key = torch.arange(n, device="cuda")
            see = key <= pos
            if c["window"]:
                see &= (pos - key < c["window"]) | (key < c["sinks"])
            for h in range(Hq):
                g = h * Hkv // Hq
                o[b, h], lse[b, h] = _exact_rows(s["q"][b, h].double(), k[g], v[g], see, d ** -0.5)
        return o, lse
    Nq, Nkv, Hq, Hkv, W = (c[k] for k in ("Nq", "Nkv", "Hq", "Hkv", "window"))
    o = torch.empty((B, Hq, Nq, d), dtype=torch.float64, device="cuda")
    lse = torch.empty((B, Hq, Nq), dtype=torch.float64, device="cuda")
    step = 2048
    for r in range(0, Nq, step):
        n = min(step, Nq - r)
        pos = Nkv - Nq + r + torch.arange(n, device="cuda")[:, None]
        key = torch.arange(Nkv, device="cuda")
        key = torch.cat([key[:c["sinks"]], key[max(0, Nkv - Nq + r - W + 1):Nkv - Nq + r + n]])
        key = key.unique()
        see = (key <= pos) & ((pos - key < W) | (key < c["sinks"]))
        for b in range(B):
            for h in range(Hq):
                g = h * Hkv // Hq
                k, v = s["k"][b, g, key].double(), s["v"][b, g, key].double()
                o[b, h, r:r + n], lse[b, h, r:r + n] = _exact_rows(
                    s["q"][b, h, r:r + n].double(), k, v, see, d ** -0.5)
    return o, lse
