"""attn_qk_norm_rope at the sizes of values that its header allows."""

from __future__ import annotations

import pytest

from test_gpu_qk_norm_rope import check

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def osx():
    import online_softmax_exact_b200 as m

    return m


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("size,eps", [(2.0 ** 57, 1e-6), (2.0 ** 57, 0.0), (2.0 ** -60, 0.0),
                                      (2.0 ** -60, 1e-6)])
def test_rope_sizes_of_values(osx, d, size, eps):
    """Normal values times 2^57 stay below 2^60."""
    check(osx, 2, 9, 4, 2, d, d, False, size=size, eps=eps)
