"""attn_kv_plan against its definition, value for value."""

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


def dev(x):
    return torch.as_tensor(np.ascontiguousarray(x), dtype=torch.int32).cuda()


def run(osx, lens, new, table, free, head, page, n_new):
    tab = dev(table)
    ten = [dev(lens), dev(new), tab, dev(free), dev([head])]
    out = osx.attn_kv_plan(*ten, page_size=page, n_new=n_new)
    ref = su.plan(lens, new, table, free, head, page, n_new)
    for name, got, want in zip(("slots", "positions", "lens", "head", "served", "table"),
                               (*out, tab), ref):
        want = np.asarray(want).reshape(got.shape)
        assert np.array_equal(got.cpu().numpy(), want), name
    # the same inputs again: the same answers, the table as it is
    again = osx.attn_kv_plan(*ten, page_size=page, n_new=n_new)
    assert all(torch.equal(a, b) for a, b in zip(out, again))
    assert np.array_equal(tab.cpu().numpy(), ref[-1])
    return ref


def case(rng, B, n_new, page, width, n_free, lens_hi=None, new_lo=0):
    lens = rng.integers(0, (width * page if lens_hi is None else lens_hi) + 1, B)
    new = rng.integers(new_lo, n_new + 1, B)
    perm = rng.permutation(B * width + n_free)
    table = np.where(np.arange(width) < -(-lens[:, None] // page),
                     perm[:B * width].reshape(B, width), -7)
    return lens, new, table, perm[B * width:]


@pytest.mark.parametrize("B,n_new,page,width", [
    (1, 1, 16, 1), (1, 1, 1, 5), (3, 1, 16, 9), (32, 1, 64, 40), (5, 7, 16, 12), (2, 1500, 16, 130),
    (700, 1, 32, 8), (513, 3, 16, 6), (512, 128, 16, 40), (1, 5000, 128, 50), (1100, 40, 48, 5),
])
def test_plan(osx, B, n_new, page, width):
    rng = np.random.default_rng(B * 1009 + n_new)
    lens, new, table, free = case(rng, B, n_new, page, width, B * (n_new // page + 2) + 5)
    run(osx, lens, new, table, free, 3, page, n_new)


@pytest.mark.parametrize("short", [0, 1, 5, 11, 1000])
@pytest.mark.parametrize("B,n_new,page", [(9, 40, 16), (600, 33, 16), (40, 1, 16)])
def test_plan_when_the_free_list_ends(osx, B, n_new, page, short):
    """Requests are served up to the one whose pages the list no longer holds; those behind
    it that need no page still are."""
    rng = np.random.default_rng(short + B)
    width = 12
    lens, new, table, _ = case(rng, B, n_new, page, width, 10, lens_hi=100)
    need = int((-(-(lens + new) // page) - -(-lens // page)).sum())
    free = rng.permutation(5000)[:max(0, need - short) + 4] + 10000
    ref = run(osx, lens, new, table, free, 4, page, n_new)
    if short and need:
        assert (ref[4] == 0).any()


def test_plan_without_a_free_page(osx):
    lens, new = [16, 15, 32], [1, 1, 0]
    table = [[3, -1, -1], [4, -1, -1], [5, 6, -1]]
    ref = run(osx, lens, new, table, np.empty(0, np.int64), 0, 16, 1)
    assert list(ref[4]) == [0, 1, 1]


@pytest.mark.parametrize("head", [-1, -2 ** 31, 2, 50, 2 ** 31 - 1])
def test_plan_with_a_head_outside_the_list(osx, head):
    run(osx, [16, 3, 0], [4, 4, 4], [[1, -1], [2, -1], [-1, -1]], [7, 8], head, 16, 4)


def test_plan_values_without_sense(osx):
    """Negative or too large lengths are not served and take nothing; a held page that is
    negative, and a slot beyond 31 bits, give no slot."""
    big = 2 ** 31 - 1
    lens = [-1, 5, 5, 5, big, 30, 17, 16, 0]
    new = [2, -1, 9, 4, 4, 4, 4, 4, 0]
    table = np.full((9, 2), -1)
    table[1:4, 0] = [1, 2, 3]
    table[5] = [4, -3]          # held page without sense
    table[6] = [5, big // 8]    # its slots pass 31 bits
    table[7, 0] = 6
    lens_out = run(osx, lens, new, table, [20, 21, 22, 23], 0, 16, 8)[2]
    assert list(lens_out) == [-1, 5, 5, 9, big, 30, 21, 20, 0]


def test_plan_on_another_stream(osx):
    rng = np.random.default_rng(2)
    lens, new, table, free = case(rng, 50, 9, 16, 10, 200)
    ref = su.plan(lens, new, table, free, 0, 16, 9)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    out = osx.attn_kv_plan(dev(lens), dev(new), dev(table), dev(free), dev([0]), page_size=16,
                           n_new=9, stream=s)
    torch.cuda.synchronize()
    assert np.array_equal(out[0].cpu().numpy(), ref[0])
