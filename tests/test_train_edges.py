"""Operators of a training step at the ends of their ranges, as far as that needs no GPU."""

import os
import re

import numpy as np

import clebsch_gordan_tensor_racah_gb300 as cg
from oracle import train as otr


def test_oracle_gradient_of_a_norm_without_z_matches_differences():
    irreps, kw = "3x0e+2x1o+2x2e", dict(alpha=0.6, eps=1e-3)
    rng = np.random.default_rng(7)
    dim, chan = otr.sizes(irreps)
    h, gout, gy = (rng.standard_normal((3, dim)) for _ in range(3))
    pre = 1 + 0.3 * rng.standard_normal(chan)

    def loss(h):
        out, y = otr.resnorm_forward(irreps, h=h, pre=pre, **kw)
        return (out * gout).sum() + (y * gy).sum()

    gh = otr.resnorm_backward(irreps, gout, gy, h, pre=pre, **kw)[0]
    num = np.zeros_like(h)
    for i in np.ndindex(h.shape):
        d = np.zeros_like(h)
        d[i] = 1e-6
        num[i] = (loss(h + d) - loss(h - d)) / 2e-6
    # truncation 1e-12 x third derivative, rounding 1e-16 / 1e-6
    assert np.abs(num - gh).max() < 1e-7 * max(1.0, np.abs(gh).max())


def _with_headers(path, seen):
    """Names of a source and of the quoted headers beside it, transitively."""
    if path in seen or not os.path.exists(path):
        return seen
    seen.add(path)
    for name in re.findall(r'^\s*#\s*include\s+"([^"]+)"', open(path).read(), re.M):
        _with_headers(os.path.join(os.path.dirname(path), name), seen)
    return seen


def test_kernels_that_start_early_read_nothing_through_the_read_only_path():
    # a kernel that chain.cuh launches is resident while the one before it writes: its operands change during its life
    csrc = os.path.join(os.path.dirname(cg.__file__), "csrc")
    early = [s for s in map(lambda f: os.path.join(csrc, f), sorted(os.listdir(csrc)))
             if s.endswith(".cu") and "chain_enter()" in "".join(open(p).read() for p in _with_headers(s, set()) if not p.endswith("chain.cuh"))]
    assert any(s.endswith("adamw.cu") for s in early) and any(s.endswith("resnorm_f32_bwd.cu") for s in early)
    for path in set().union(*(_with_headers(s, set()) for s in early)):
        code = re.sub(r"//[^\n]*|/\*.*?\*/", "", open(path).read(), flags=re.S)
        assert not re.search(r"__ldg\s*\(|ld\.global(\.\w+)*\.nc|__restrict__", code), path


def test_tables_are_complete_when_a_plan_is_returned():
    # a synchronous copy from pageable memory may return before it has arrived, and orders only the default stream behind it:
    # every table goes through upload(), which waits
    csrc = os.path.join(os.path.dirname(cg.__file__), "csrc")
    calls = [(f, m) for f in sorted(os.listdir(csrc)) if f.endswith((".cu", ".cuh", ".h"))
             for m in re.findall(r"[^\n]*\b(?:cudaMemcpy|cudaMemset)\s*\([^\n]*", re.sub(r"//[^\n]*", "", open(os.path.join(csrc, f)).read()))]
    assert [f for f, _ in calls] == ["api.cu"] and "cudaStreamSynchronize(cudaStreamLegacy)" in calls[0][1]
