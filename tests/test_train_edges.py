"""Operators of a training step at the ends of their ranges, as far as that needs no GPU."""

import os
import re
import subprocess
import sys

import numpy as np
import pytest

import clebsch_gordan_tensor_racah_gb300 as cg
from clebsch_gordan_tensor_racah_gb300 import _build
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


def test_the_library_builds_and_loads_without_torch():
    # None in sys.modules: importing torch raises ImportError, as on a machine that has none
    code = ("import sys; sys.modules['torch'] = None\n"
            "from clebsch_gordan_tensor_racah_gb300 import _build\n"
            "assert _build.build() == _build.LIB\n"
            "import clebsch_gordan_tensor_racah_gb300 as cg\n"
            "assert cg.cgtp_real_cg_block(1, 1, 1) is not None\n")
    root = os.path.dirname(os.path.dirname(cg.__file__))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr


def test_an_interrupted_link_of_the_binding_is_not_up_to_date(tmp_path, monkeypatch):
    torch = pytest.importorskip("torch")
    _build.build()
    monkeypatch.setattr(_build, "BINDING", str(tmp_path / "_binding.so"))
    monkeypatch.setattr(_build, "BINDING_STAMP", str(tmp_path / "stamp"))
    (tmp_path / "stamp").write_text(torch.__version__)      # of an earlier build with the same torch

    def interrupted(cmd):
        with open(cmd[cmd.index("-o") + 1], "wb") as f:
            f.write(b"half")
        raise RuntimeError("interrupted")

    monkeypatch.setattr(_build, "_run", interrupted)
    with pytest.raises(RuntimeError, match="interrupted"):
        _build.build()
    assert _build._binding_command() is not None
