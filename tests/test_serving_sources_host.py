"""What the serving kernels' sources may not contain (no GPU needed).

Their launches are programmatic dependents: a kernel's blocks may be resident while the launch
before it still writes. Loads through the read-only path (ld.global.nc: __ldg, or a const
__restrict__ pointer) need data that nobody writes during the kernel's lifetime, and neither
the compiler nor the cache orders them behind the dependency wait."""

from __future__ import annotations

import re
from pathlib import Path

CSRC = Path(__file__).resolve().parent.parent / "online_softmax_exact_b200" / "csrc"


def sources(name, seen=None):
    """A source and everything of this directory that it includes."""
    seen = {} if seen is None else seen
    if name not in seen and (CSRC / name).exists():
        seen[name] = (CSRC / name).read_text()
        for inc in re.findall(r'^#include "([^"]+)"', seen[name], re.M):
            sources(inc, seen)
    return seen


def code(text):
    return re.sub(r"//[^\n]*|/\*.*?\*/", "", text, flags=re.S)


def test_the_walk_finds_the_kernels():
    assert {"kv4_fwd_kernel.cuh", "kv_plan_kernel.cuh", "kv4_copy_kernels.cuh", "decode_common.cuh",
            "qk_norm_rope_kernel.cuh", "window_token_kernel.cuh",
            "attn_window_kernel.cuh"} <= set(sources("serve_kernels.cu"))


def test_dependent_launches_read_through_the_coherent_path():
    bad = [(name, m.group(0)) for name, text in sources("serve_kernels.cu").items()
           for m in re.finditer(r"__ldg\b|__ldlu\b|\.global\.nc\b|\.nc\.|__restrict__", code(text))]
    assert not bad


def test_every_kernel_waits_for_the_launch_before():
    for name, text in sources("serve_kernels.cu").items():
        for body in re.split(r"__global__", code(text))[1:]:
            if name == "attn_fwd_kernel.cuh":
                continue  # launched by attn_kernels.cu, never as a dependent
            assert "grid_dependency_wait();" in body, name
