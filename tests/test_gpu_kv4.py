"""The paged 4-bit cache: attn_kv4_append and attn_kv4_read against the format's definition
(codes and parameters bit for bit), attn_kv4_fwd against attention in 64 bits over the
values that the cache stands for."""

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


# ---------------------------------------------------------------------------------- append
def append_case(osx, k, v, slots, page, n_pages):
    """Appends into a cache of 0xA5 bytes and compares every byte."""
    B, Hkv, N, d = k.shape
    cache = torch.full((n_pages, Hkv, page // 16, 20 * d), 0xA5, dtype=torch.uint8).cuda()
    osx.attn_kv4_append(k.cuda(), v.cuda(), cache, i32(slots))
    got = cache.cpu().numpy()
    want = np.full(got.shape, 0xA5, np.uint8)
    kn, vn = su.to_np(k), su.to_np(v)
    for b in range(B):
        for i in range(N):
            s = int(slots[b][i])
            if 0 <= s < n_pages * page:
                for h in range(Hkv):
                    su.pack_cache(want, s, h, kn[b, h, i], vn[b, h, i], page)
    assert np.array_equal(got, want), [
        (b, h, i) for b in range(B) for i in range(N) for h in range(Hkv)
        if 0 <= slots[b][i] < n_pages * page
        and any((x != y).any() for a, c in zip(su.unpack_token(got, slots[b][i], h, page, d),
                                               su.unpack_token(want, slots[b][i], h, page, d))
                for x, y in zip(a, c))]
    return cache


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("B,N,Hkv,page,first", [
    (3, 1, 2, 16, 5), (1, 16, 1, 16, 0), (1, 40, 2, 16, 0), (2, 50, 1, 32, 7), (1, 33, 3, 64, 15),
    (1, 100, 1, 48, 1),
])
def test_append_runs_of_slots(osx, d, B, N, Hkv, page, first):
    g = torch.Generator().manual_seed(d + N)
    k, v = (torch.randn((B, Hkv, N, d), generator=g).to(torch.bfloat16) for _ in range(2))
    per = -(-(first + N) // page)
    n_pages = B * per + 1
    pages = np.random.default_rng(N).permutation(n_pages)[:B * per].reshape(B, per)
    pos = first + np.arange(N)
    slots = pages[:, pos // page] * page + pos % page
    append_case(osx, k, v, slots, page, n_pages)


@pytest.mark.parametrize("d", [64, 128])
def test_append_scattered_and_skipped_slots(osx, d):
    """Slots in any order, -1 and slots outside the cache skip their rows; every other byte
    of the cache stays."""
    rng = np.random.default_rng(d)
    g = torch.Generator().manual_seed(d)
    k, v = (torch.randn((3, 2, 21, d), generator=g).to(torch.bfloat16) for _ in range(2))
    slots = rng.permutation(6 * 32)[:63].reshape(3, 21)
    slots[0, 3] = slots[1, 0] = -1
    slots[2, 20], slots[2, 19], slots[2, 1] = 6 * 32, 2 ** 31 - 1, -2 ** 31
    append_case(osx, k, v, slots, 32, 6)
    append_case(osx, k, v, np.full((3, 21), -1), 32, 6)


@pytest.mark.parametrize("d", [64, 128])
def test_append_values_at_the_format_s_edges(osx, d):
    """Equal values (scale 0), ties between codes, subnormals, ranges from 2^-120 to 2^126."""
    rows = [torch.full((d,), 0.75), torch.zeros(d), torch.arange(d) % 32 / 2.0,
            (torch.arange(d) % 31).float(), torch.randn(d) * 2.0 ** -120,
            torch.randn(d) * 2.0 ** 120, torch.randn(d) * 1e-40, torch.linspace(-1, 1, d) * 2.0 ** 126,
            torch.cat([torch.full((d - 1,), -0.0), torch.tensor([0.0])]),
            torch.where(torch.arange(d) % 32 == 5, 1000.0, 0.001), torch.randn(d) + 100]
    x = torch.stack(rows).to(torch.bfloat16).view(1, 1, len(rows), d)
    append_case(osx, x, x.flip(2).contiguous(), [list(range(16, 16 + len(rows)))], 16, 4)


def test_append_many_ties(osx):
    """Multiples of a half step against a scale that is exact in bf16: half the quotients
    are ties and go to the even code."""
    g = torch.Generator().manual_seed(0)
    x = torch.randint(0, 61, (1, 2, 64, 128), generator=g).float() / 2
    x[..., ::32], x[..., 1::32] = 0.0, 30.0
    k = (x * 2.0 ** torch.randint(-8, 8, (1, 2, 64, 1), generator=g)).to(torch.bfloat16)
    append_case(osx, k, (-k).contiguous(), [list(range(64))], 64, 1)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("page", [16, 48, 64])
def test_read(osx, d, page):
    rng = np.random.default_rng(d + page)
    B, Hkv, width, n_pages = 5, 2, 4, 23
    cache, kp, vp = su.random_cache(rng, n_pages, Hkv, page, d)
    table = rng.permutation(n_pages)[:B * width].reshape(B, width)
    table[3, 1], table[4, 0] = -1, n_pages
    lens = np.array([width * page, 37, 0, 2 * page + 3, 3 * page])
    start = np.array([0, 5, 0, 7, -3])
    n = 3 * page + 10
    k, v = osx.attn_kv4_read(torch.from_numpy(cache).cuda(), i32(table), i32(start), i32(lens), n=n)
    for got, (c, s, z) in ((k, kp), (v, vp)):
        want = np.zeros((B, Hkv, n, d))
        for b in range(B):
            for i in range(n):
                p = start[b] + i
                if start[b] < 0 or p >= lens[b] or p // page >= width:
                    continue
                pg = table[b, p // page]
                if 0 <= pg < n_pages:
                    o = p % page
                    want[b, :, i] = su.bf16(su.values(c[pg, :, o], s[pg, :, o], z[pg, :, o]))
        assert np.array_equal(su.to_np(got), want)


def test_read_past_the_table(osx):
    cache, kp, _ = su.random_cache(np.random.default_rng(1), 2, 1, 16, 64)
    k, v = osx.attn_kv4_read(torch.from_numpy(cache).cuda(), i32([[1]]), i32([10]), i32([100]), n=20)
    c, s, z = kp
    assert np.array_equal(su.to_np(k)[0, 0, :6], su.bf16(su.values(c[1, 0, 10:], s[1, 0, 10:], z[1, 0, 10:])))
    assert not k[0, 0, 6:].any() and not v[0, 0, 6:].any()


# --------------------------------------------------------------------------------- forward
def fwd_case(osx, seed, B, Hq, Hkv, Nq, d, page, lens, window=0, sinks=0, q_pos=None, scale=None,
             o_dtype=torch.float32, qsize=1.0, max_len=0, bad_pages=(), width=None, table=None,
             ksize=1.0, vsize=1.0, poison_unseen=None):
    rng = np.random.default_rng(seed)
    lens = np.asarray(lens)
    if width is None:
        width = max(1, int(-(-max(int(lens.max()), 1) // page)))
    n_pages = B * width + 2
    cache, kp, vp = su.random_cache(rng, n_pages, Hkv, page, d, ksize, vsize)
    if table is None:
        table = rng.permutation(n_pages)[:B * width].reshape(B, width)
    for b, p, x in bad_pages:
        table[b, p] = x
    # rows of a request's last page past its length that no other request holds there, and
    # pages nobody holds: any bits
    words = cache.view(np.uint32)
    spots = [{(int(table[b, p // page]), p % page) for p in span}
             for b in range(B) for n in [int(min(max(lens[b], 0), width * page))]
             for span in (range(n), range(n, -(-n // page) * page))]
    for pg, p in set().union(*spots[1::2]) - set().union(*spots[::2]):
        if 0 <= pg < n_pages:
            row = p % 16
            for p0 in (4 * d, 4 * d + d // 2):
                words[pg, :, p // 16, p0 + row * (d // 32):p0 + (row + 1) * (d // 32)] = 0x7fc07f80
    if poison_unseen is not None:
        # parameters of every token that no row of its request sees
        for b in range(B):
            n = int(min(max(lens[b], 0), width * page))
            pos = (n - Nq if q_pos is None else q_pos[b]) + np.arange(Nq)
            for p in np.flatnonzero(~su.visible(pos, np.arange(n), window, sinks).any(0)):
                row = p % 16
                for p0 in (4 * d, 4 * d + d // 2):
                    words[table[b, p // page], :, p % page // 16,
                          p0 + row * (d // 32):p0 + (row + 1) * (d // 32)] = poison_unseen
    words[sorted(set(range(n_pages)) - set(table.flat))] = 0xffffffff
    g = torch.Generator().manual_seed(seed)
    q = (torch.randn((B, Hq, Nq, d), generator=g) * qsize).to(torch.bfloat16)
    scale = d ** -0.5 if scale is None else scale
    o, lse = osx.attn_kv4_fwd(q.cuda(), torch.from_numpy(cache).cuda(), i32(table), i32(lens),
                              q_pos=None if q_pos is None else i32(q_pos), window=window,
                              sinks=sinks, scale=scale, o_dtype=o_dtype, max_len=max_len)
    assert osx.attn_device_status() == osx.ATTN_OK
    assert o.dtype == o_dtype
    on, ln, qn = su.to_np(o), su.to_np(lse), su.to_np(q)
    for b in range(B):
        n = int(min(max(lens[b], 0), width * page))
        key = np.arange(n)
        pg = table[b, key // page] if n else np.zeros(0, int)
        real = (pg >= 0) & (pg < n_pages)
        safe = np.where(real, pg, 0)
        pos = (n - Nq if q_pos is None else q_pos[b]) + np.arange(Nq)
        see = su.visible(pos, key, window, sinks) & real[None]
        for h in range(Hkv):
            def take(part):
                return [x[safe, h, key % page] for x in part]

            kc, ks, kz = take(kp)
            vc, vs, vz = take(vp)
            kf, vf = su.values(kc, ks, kz), su.values(vc, vs, vz)
            # the kernel sums scale * c and zero apart; the weight of scale * c enters as
            # two bf16 numbers: the upper 8 bits cut off, the rest (below 2^-7 of it)
            # rounded by at most 2^-8 of itself
            kmag, vmag = su.values(kc, ks, np.abs(kz)), su.values(vc, vs, 0 * vz)
            vfull = su.values(vc, vs, np.abs(vz))
            for x in range(Hq // Hkv):
                r = h * (Hq // Hkv) + x
                ref = su.attention(qn[b, r], kf, vf, see, np.float64(np.float32(scale)), kmag,
                                   vmag, vfull, 2.0 ** -15, o_dtype == torch.bfloat16)
                su.check(on[b, r], ln[b, r], ref, f"request {b} head {r}")
    return o, lse


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("page", [16, 32, 48, 128])
@pytest.mark.parametrize("Hq,Hkv", [(4, 4), (8, 2), (8, 1)])
def test_fwd(osx, d, page, Hq, Hkv):
    fwd_case(osx, d + page, 4, Hq, Hkv, 1, d, page, [1, 17, 200, 333])


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Nq,Hq,Hkv", [(2, 4, 2), (3, 12, 4), (5, 16, 2), (17, 3, 1), (40, 2, 2),
                                       (1, 32, 1), (1, 9, 1)])
def test_fwd_several_rows(osx, d, Nq, Hq, Hkv):
    """Row counts of 1 to 40 per key/value head: one and two tiles of eight, and several."""
    fwd_case(osx, Nq + Hq, 3, Hq, Hkv, Nq, d, 16, [Nq, 50, 260], o_dtype=torch.bfloat16)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("lens", [[0, 1, 2], [15, 16, 17], [0, 0, 0], [31, 32, 33], [63, 64, 65]])
def test_fwd_short_lengths(osx, d, lens):
    """Lengths around blocks and stages, empty requests, more rows than tokens."""
    fwd_case(osx, sum(lens), 3, 4, 2, 1, d, 16, lens, width=8)
    fwd_case(osx, sum(lens), 3, 4, 2, 4, d, 16, lens, width=8)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (16, 4), (33, 0), (64, 20), (100, 130),
                                          (5000, 4), (257, 1000)])
def test_fwd_window(osx, d, window, sinks):
    fwd_case(osx, window + sinks, 3, 4, 2, 1, d, 16, [600, 37, 303], window=window, sinks=sinks)
    fwd_case(osx, window + sinks, 2, 4, 2, 5, d, 32, [600, 301], window=window, sinks=sinks)


@pytest.mark.parametrize("d", [64, 128])
def test_fwd_positions_of_the_callers_choice(osx, d):
    """Rows before, among and far behind the cached tokens; rows whose window holds none."""
    lens = [100, 100, 100, 100, 100, 100]
    pos = [0, -2, 50, 99, 120, 2 ** 31 - 10]
    fwd_case(osx, 1, 6, 4, 2, 4, d, 16, lens, q_pos=pos)
    fwd_case(osx, 2, 6, 4, 2, 4, d, 16, lens, q_pos=pos, window=30, sinks=0)
    fwd_case(osx, 3, 6, 4, 2, 4, d, 16, lens, q_pos=pos, window=30, sinks=5)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("bits", [0x7fc07fc0, 0x7f803f80, 0x3f807f80, 0xff80ff80])
def test_fwd_unseen_tokens_hold_any_bits(osx, d, bits):
    """Tokens before the window, between sinks and window, and behind the rows' positions
    (never written, or another request's by now) share blocks with tokens that are seen:
    NaN and infinities in their parameters do not reach the result."""
    kw = dict(poison_unseen=bits)
    fwd_case(osx, 21, 3, 4, 2, 1, d, 16, [600, 37, 303], window=70, **kw)
    fwd_case(osx, 22, 3, 4, 2, 1, d, 16, [600, 37, 303], window=33, sinks=5, **kw)
    fwd_case(osx, 23, 2, 8, 2, 5, d, 32, [600, 301], window=40, sinks=17, **kw)
    fwd_case(osx, 24, 3, 4, 2, 3, d, 16, [200, 200, 200], q_pos=[0, 50, 120], **kw)
    fwd_case(osx, 25, 2, 4, 4, 1, d, 64, [5000, 4000], window=2001, q_pos=[3000, 3999], **kw)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Nq,Hq,n", [(3, 2, 100), (5, 4, 700), (8, 2, 33)])
def test_fwd_token_seen_by_the_last_row_only(osx, d, Nq, Hq, n):
    """NaN parameters of the newest token change no bit of the rows before it."""
    rng = np.random.default_rng(n)
    cache, _, _ = su.random_cache(rng, n // 16 + 1, 1, 16, d)
    g = torch.Generator().manual_seed(n)
    q = torch.randn((1, Hq, Nq, d), generator=g).to(torch.bfloat16).cuda()
    table = i32(rng.permutation(n // 16 + 1)[None])

    def run():
        return osx.attn_kv4_fwd(q, torch.from_numpy(cache).cuda(), table, i32([n]))

    o, lse = run()
    words, row = cache.view(np.uint32), (n - 1) % 16
    for p0 in (4 * d, 4 * d + d // 2):
        words[int(table[0, (n - 1) // 16]), :, 0,
              p0 + row * (d // 32):p0 + (row + 1) * (d // 32)] = 0x7fc07fc0
    o2, lse2 = run()
    assert torch.equal(o[:, :, :-1], o2[:, :, :-1]) and torch.equal(lse[:, :, :-1], lse2[:, :, :-1])


@pytest.mark.parametrize("d", [64, 128])
def test_fwd_long(osx, d):
    """Clusters of blocks on one unit, many stages per warp, a ragged batch; the hint does
    not change the definition."""
    fwd_case(osx, 5, 1, 8, 1, 1, d, 64, [20000], o_dtype=torch.bfloat16)
    fwd_case(osx, 6, 2, 8, 2, 1, d, 128, [9000, 100])
    fwd_case(osx, 7, 2, 4, 2, 3, d, 16, [5000, 100], max_len=64)
    fwd_case(osx, 7, 2, 4, 2, 3, d, 16, [5000, 100], max_len=10 ** 9)


@pytest.mark.parametrize("d", [64, 128])
def test_fwd_bad_pages_and_lengths(osx, d):
    """Pages outside the cache hide their tokens; lengths outside the table are cut."""
    fwd_case(osx, 8, 3, 4, 2, 2, d, 16, [100, 90, 80],
             bad_pages=[(0, 0, -1), (0, 3, 10 ** 6), (1, 5, -2 ** 31), (2, 2, 2 ** 31 - 1)])
    fwd_case(osx, 9, 3, 4, 2, 1, d, 16, [64, 64, 64], bad_pages=[(0, p, -1) for p in range(4)])
    fwd_case(osx, 10, 3, 4, 2, 1, d, 16, [-5, 1000, 2 ** 31 - 1], width=5)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("qsize,scale", [(8.0, None), (1.0, 3.0), (0.0, None), (1.0, 1e-6)])
def test_fwd_large_and_flat_scores(osx, d, qsize, scale):
    """Running maxima that move by hundreds of octaves, and uniform weights."""
    fwd_case(osx, 11, 2, 8, 2, 1, d, 32, [700, 45], qsize=qsize, scale=scale)


def test_fwd_weights_err_to_neither_side(osx):
    """Flat weights over many tokens, codes of one size against the zero point that cancels
    them: what is left is as exact as unbiased roundings leave it. (Each weight's error is at
    most 2^-15 of it; a bias of half that would move the result by 2^-16 * 15 scale.)"""
    rng = np.random.default_rng(0)
    n, page, d = 20480, 64, 128
    cache, kp, vp = su.random_cache(rng, n // page, 1, page, d)
    q = torch.randn((1, 4, 1, d), generator=torch.Generator().manual_seed(0)).to(torch.bfloat16)
    table = np.arange(n // page)[None]
    o, _ = osx.attn_kv4_fwd(q.cuda(), torch.from_numpy(cache).cuda(), i32(table), i32([n]), scale=0.1)
    k, v = (su.values(*[x.reshape(n, -1) for x in p]) for p in (kp, vp))
    full = su.values(vp[0].reshape(n, d), vp[1].reshape(n, -1), np.abs(vp[2].reshape(n, -1)))
    for h in range(4):
        s = su.to_np(q)[0, h] @ k.T * np.float64(np.float32(0.1))
        p = np.exp(s - s.max())
        p /= p.sum()
        # independent errors of up to 2^-15 add as their squares do: six of their deviations,
        # and fp32 sums (256 runs of 80 tokens each: 2^-24 of a run's sum, 2^-24 in the join)
        bound = 6 * 2.0 ** -15 * np.sqrt(p[0] ** 2 @ full ** 2)
        bound = bound + 2.0 ** -18 * (p[0] @ full)
        assert (np.abs(su.to_np(o)[0, h, 0] - p[0] @ v) <= bound).all()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("qsize,ksize,vsize", [
    (1.0, 1.0, 2.0 ** -35), (1.0, 1.0, 2.0 ** 21), (2.0 ** 90, 2.0 ** -90, 1.0),
    (2.0 ** -60, 2.0 ** 60, 1.0), (2.0 ** 20, 2.0 ** -18, 2.0 ** 10), (2.0 ** -110, 1.0, 1.0)])
def test_fwd_sizes_of_values(osx, d, qsize, ksize, vsize):
    """Queries, keys and values of any size: their operands carry powers of two."""
    fwd_case(osx, 14, 2, 8, 2, 1, d, 16, [300, 41], qsize=qsize, ksize=ksize, vsize=vsize)
    fwd_case(osx, 14, 2, 8, 2, 2, d, 16, [300, 41], qsize=qsize, ksize=ksize, vsize=vsize)


def test_fwd_shared_pages(osx):
    """Requests may share pages (a common prefix): the same page in several rows, and twice
    in one."""
    table = np.array([[0, 1, 2, 0], [0, 1, 3, 4]])
    fwd_case(osx, 12, 2, 4, 2, 1, 128, 16, [60, 64], table=table)


def test_fwd_is_deterministic_and_merges(osx):
    """Two calls give the same bits; the partials of two requests over halves of a table
    merge to the whole."""
    rng = np.random.default_rng(3)
    cache, _, _ = su.random_cache(rng, 40, 2, 16, 128)
    cg = torch.from_numpy(cache).cuda()
    q = torch.randn((1, 8, 1, 128), generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).cuda()
    table = i32(rng.permutation(40)[None])
    o, lse = osx.attn_kv4_fwd(q, cg, table, i32([640]))
    o2, lse2 = osx.attn_kv4_fwd(q, cg, table, i32([640]))
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    a = osx.attn_kv4_fwd(q, cg, table[:, :17].contiguous(), i32([272]))
    b = osx.attn_kv4_fwd(q, cg, table[:, 17:].contiguous(), i32([368]))
    om, lm = osx.attn_merge([a[0], b[0]], [a[1], b[1]])
    # weights rounded against other bases: 2^-15 each way of scale * c, up to 0.4 * 15
    assert (om - o).abs().max() <= 2 * 6 * 2.0 ** -15 and (lm - lse).abs().max() <= 1e-4
