"""The serving binding is compiled against one torch and one Python: another version has it
built again, and is refused until it is (no GPU needed)."""

from __future__ import annotations

import pytest
import torch


@pytest.fixture()
def built():
    from online_softmax_exact_b200 import build as b

    b.build()
    return b


def test_binding_of_another_torch_is_built_again(built, monkeypatch, tmp_path):
    made = []
    monkeypatch.setattr(built, "_build_binding", made.append)
    monkeypatch.setattr(built, "BINDING_STAMP", tmp_path / "stamp")
    (tmp_path / "stamp").write_text(built.binding_target())
    built.build()
    assert not made
    monkeypatch.setattr(torch, "__version__", "0.0.0")
    built.build()
    assert len(made) == 1 and made[0].startswith("torch 0.0.0, python ")
    built.build()
    assert len(made) == 1  # and once only


def test_binding_of_another_torch_is_refused(built, monkeypatch):
    from online_softmax_exact_b200 import _abi

    monkeypatch.setattr(_abi, "_serving", None)
    assert _abi.load_serving().built_for == _abi.binding_target()
    monkeypatch.setattr(_abi, "_serving", None)
    monkeypatch.setattr(torch, "__version__", "0.0.0")
    with pytest.raises(ImportError, match="built for torch .*build it again"):
        _abi.load_serving()
    assert _abi._serving is None
