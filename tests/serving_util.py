"""References of the serving operators in 64 bits (numpy), written from the definitions in
include/attn.h, and the error bounds the GPU tests hold the kernels to."""

from __future__ import annotations

import numpy as np
import torch

HALF_BF16 = 2.0 ** -8   # largest relative error of a rounding to bf16 (half a step)


def to_np(t: torch.Tensor) -> np.ndarray:
    return t.detach().to("cpu", torch.float64).numpy()


def bf16(x: np.ndarray) -> np.ndarray:
    """fp64 values rounded to the nearest bf16 (through fp32, ties to even)."""
    t = torch.from_numpy(np.ascontiguousarray(x, np.float32)).to(torch.bfloat16)
    return t.to(torch.float64).numpy()


# ------------------------------------------------------------------------------------ plan
def plan(lens, new, table, free, head, page, n_new):
    """(slots, positions, lens, head, served, table) of attn_kv_plan."""
    lens, new, table = [int(x) for x in lens], [int(x) for x in new], np.array(table)
    B, width = table.shape
    held_table = table.copy()
    slots = np.full((B, n_new), -1, np.int64)
    pos = np.zeros((B, n_new), np.int64)
    out, served = list(lens), [0] * B
    want_total = taken = 0
    for b in range(B):
        pos[b] = lens[b] + np.arange(n_new)
        if lens[b] < 0 or new[b] < 0 or new[b] > n_new:
            continue
        held, want = -(-lens[b] // page), -(-(lens[b] + new[b]) // page)
        if want > width:
            continue
        need, start = want - held, head + want_total
        want_total += need
        if need and (head < 0 or start + need > len(free)):
            continue
        served[b], out[b] = 1, lens[b] + new[b]
        taken += need
        for p in range(held, want):
            table[b, p] = free[start + p - held]
        for i in range(new[b]):
            p = pos[b, i] // page
            pg = table[b, p] if p >= held else held_table[b, p]
            if pg >= 0 and pg * page + page - 1 < 2 ** 31:
                slots[b, i] = pg * page + pos[b, i] % page
    pos = (pos + 2 ** 31) % 2 ** 32 - 2 ** 31  # stored as int32
    return slots, pos, np.array(out), head + taken, np.array(served), table


# -------------------------------------------------------------------------- norms, rotation
def norm_rope(x, w, inv_freq, pos, eps, interleaved):
    """x [..., N, d] fp64 (bf16 values), pos [N]-broadcastable -> rows in fp64, and the size
    of the terms each value is a sum of."""
    d, f = x.shape[-1], len(inv_freq)
    y = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * w
    a = pos[..., None].astype(np.float64) * inv_freq
    c, s = np.cos(a), np.sin(a)
    out, mag = y.copy(), np.abs(y)
    i, j = (np.arange(0, 2 * f, 2), np.arange(1, 2 * f, 2)) if interleaved else \
        (np.arange(f), np.arange(f, 2 * f))
    u, v = y[..., i], y[..., j]
    out[..., i], out[..., j] = u * c - v * s, v * c + u * s
    mag[..., i] = mag[..., j] = np.abs(u) + np.abs(v)
    assert out.shape[-1] == d
    return out, mag


# ------------------------------------------------------------------------------ 4-bit cache
def quantise(x):
    """bf16 values [..., d] (fp64) -> codes [..., d], scale, zero [..., d / 32] (fp64)."""
    g = x.reshape(*x.shape[:-1], x.shape[-1] // 32, 32)
    lo, hi = g.min(-1) + 0.0, g.max(-1)  # a zero point of -0 is +0
    scale = bf16((hi - lo) / 15)
    with np.errstate(divide="ignore", invalid="ignore"):
        c = np.rint((g - lo[..., None]) / scale[..., None])
    c = np.where(scale[..., None] > 0, c, 0).clip(0, 15)
    return c.reshape(x.shape).astype(np.int64), scale, lo


def values(codes, scale, zero):
    return codes * np.repeat(scale, 32, -1) + np.repeat(zero, 32, -1)


def word_of(which, token, e, d):
    """(word in the block, nibble) of value e of a token."""
    if which == "k":
        r, g, i, t, n = token // 8, token % 8, e // 32, e % 32 // 8, e % 8
        w = ((r * 8 + g) * 4 + t) * 4 + i if d == 128 else ((g * 4 + t) * 2 + r) * 2 + i
        return w, n
    b, t, a, h, n, g = token // 8, token % 8 // 2, token % 2, e // 64, e % 64 // 8, e % 8
    return 2 * d + (((h * 8 + g) * 4 + t) * 2 + b) * 2 + a, n


def pack_cache(cache, slot, h, k, v, page):
    """Writes one token's keys and values (fp64 [d]) of head h into the cache (uint8 numpy)."""
    d = len(k)
    words = cache.view(np.uint32)[slot // page, h, slot % page // 16]
    row = slot % 16
    for which, x in (("k", k), ("v", v)):
        c, s, z = quantise(x)
        for e in range(d):
            w, n = word_of(which, row, e, d)
            words[w] = (int(words[w]) & ~(15 << (4 * n)) & 0xffffffff) | (int(c[e]) << (4 * n))
        p0 = 4 * d + (0 if which == "k" else d // 2) + row * (d // 32)
        su = torch.from_numpy(s).to(torch.bfloat16).view(torch.int16).numpy().astype(np.int64)
        zu = torch.from_numpy(z).to(torch.bfloat16).view(torch.int16).numpy().astype(np.int64)
        for i in range(d // 32):
            words[p0 + i] = (int(su[i]) & 0xffff) | ((int(zu[i]) & 0xffff) << 16)


def unpack_token(cache, slot, h, page, d):
    """(codes [d], scale, zero [d / 32]) of the keys and of the values in a slot."""
    words = cache.view(np.uint32)[slot // page, h, slot % page // 16].astype(np.int64)
    row, out = slot % 16, []
    for which in ("k", "v"):
        c = np.empty(d, np.int64)
        for e in range(d):
            w, n = word_of(which, row, e, d)
            c[e] = (int(words[w]) >> (4 * n)) & 15
        p0 = 4 * d + (0 if which == "k" else d // 2) + row * (d // 32)
        p = words[p0:p0 + d // 32]
        f = [np.array([(int(x) >> sh & 0xffff) << 16 for x in p], np.uint32).view(np.float32)
             .astype(np.float64) for sh in (0, 16)]
        out.append((c, f[0], f[1]))
    return out


def token_words(d):
    """Word map of a block: for each token the words that hold its codes, and the rest."""
    return {t: sorted({word_of(w, t, e, d)[0] for w in "kv" for e in range(d)})
            for t in range(16)}


def random_cache(rng, n_pages, Hkv, page, d, ksize=1.0, vsize=1.0):
    """A cache of random codes and sensible parameters (times a power of two), and what it
    stands for: cache uint8, and per (k, v) codes [n_pages, Hkv, page, d], scale, zero [.., d / 32]."""
    blocks = page // 16
    cache = np.zeros((n_pages, Hkv, blocks, 20 * d), np.uint8)
    words = cache.view(np.uint32)
    parts = []
    for which in ("k", "v"):
        c = rng.integers(0, 16, (n_pages, Hkv, blocks, 16, d))
        size = ksize if which == "k" else vsize
        s = bf16(rng.uniform(0.05, 0.4, (n_pages, Hkv, blocks, 16, d // 32))) * size
        z = bf16(rng.uniform(-3, 0.2, s.shape)) * size
        e = np.arange(d)
        for t in range(16):
            w, n = zip(*(word_of(which, t, x, d) for x in e))
            np.bitwise_or.at(words, (slice(None), slice(None), slice(None), np.array(w)),
                             (c[..., t, :] << (4 * np.array(n))).astype(np.uint32))
        su = torch.from_numpy(s).to(torch.bfloat16).view(torch.int16).numpy().astype(np.int64) & 0xffff
        zu = torch.from_numpy(z).to(torch.bfloat16).view(torch.int16).numpy().astype(np.int64) & 0xffff
        p0 = 4 * d + (0 if which == "k" else d // 2)
        words[..., p0:p0 + d // 2] = (su | zu << 16).reshape(*s.shape[:3], -1).astype(np.uint32)
        parts.append((c.reshape(n_pages, Hkv, page, d), s.reshape(n_pages, Hkv, page, -1),
                      z.reshape(n_pages, Hkv, page, -1)))
    return cache, parts[0], parts[1]


# -------------------------------------------------------------------------------- attention
def visible(pos, key, window, sinks):
    see = key[None, :] <= pos[:, None]
    if window:
        see &= (key[None, :] > pos[:, None] - window) | (key[None, :] < sinks)
    return see


def attention(q, k, v, see, scale, kmag=None, vmag=None, vfull=None, wround=HALF_BF16,
              o_bf16=False):
    """One head by the definition: q [n, d], k, v [m, d], see [n, m] ->
    (o, lse, bound on |dO|, bound on |dLSE|).

    kmag [m, d]: the size of the terms whose sum a key value is in the kernel (default |k|);
    vmag [m, d]: the part of a value whose weight is rounded for the matrix unit (default
    |v|), by wround (bf16: 2^-8); vfull [m, d]: the size of all its terms (default |v|).
    Scores: fp32 sums of d products (each addition off by at most 2^-23 of the terms, since a
    matrix unit may cut rather than round), so a score is off by at most
    es = (d + 4) 2^-23 scale sum |q| kmag, a weight by a factor e^(2 es) (its own score and
    the denominator) plus the exponential's 2^-21; O's own rounding is 2^-8 of |O| (bf16) or
    2^-22 (fp32, with the sums)."""
    n, d = q.shape
    kmag = np.abs(k) if kmag is None else kmag
    vmag = np.abs(v) if vmag is None else vmag
    vfull = np.abs(v) if vfull is None else vfull
    s = np.where(see, q @ k.T * scale, -np.inf)
    es = np.where(see, (np.abs(q) @ kmag.T) * scale * (d + 4) * 2.0 ** -23, 0).max(-1, initial=0)
    m = s.max(-1, initial=-np.inf)
    base = np.where(np.isneginf(m), 0, m)
    p = np.exp(s - base[:, None])
    l = p.sum(-1)
    with np.errstate(divide="ignore"):
        lse = np.where(l > 0, base + np.log(l), -np.inf)
    p = p / np.where(l > 0, l, 1)[:, None]
    o = p @ v
    rel = np.expm1(2 * es) + 2.0 ** -20
    bo = rel[:, None] * (p @ vfull) + wround * (p @ vmag) * (1 + rel[:, None])
    bo += (HALF_BF16 if o_bf16 else 2.0 ** -22) * (np.abs(o) + bo) + 1e-30
    bl = es + 2.0 ** -20 + 2.0 ** -22 * np.abs(np.where(np.isfinite(lse), lse, 0))
    return o, lse, bo, bl


def check(o, lse, ref, what=""):
    """o [n, d], lse [n] (fp64) against attention()'s answer."""
    ro, rl, bo, bl = ref
    assert np.array_equal(np.isneginf(lse), np.isneginf(rl)), f"{what}: rows without a key"
    assert np.isfinite(o).all(), f"{what}: non-finite O"
    off = np.abs(o - ro) - bo
    assert off.max() <= 0, (f"{what}: |dO| {np.abs(o - ro).flat[off.argmax()]:.3e} over its bound "
                            f"{bo.flat[off.argmax()]:.3e}")
    fin = np.isfinite(rl)
    if fin.any():
        off = np.abs(lse[fin] - rl[fin]) - bl[fin]
        assert off.max() <= 0, (f"{what}: |dLSE| {np.abs(lse[fin] - rl[fin])[off.argmax()]:.3e} "
                                f"over its bound {bl[fin][off.argmax()]:.3e}")
