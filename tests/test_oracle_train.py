"""The oracle of the training-step operators against independent facts (CPU).

* the norm's gradients against central differences of its forward, and its equivariance;
* AdamW against the closed form of its first step and against accumulation by hand;
* the 8-bit code tables: monotone, continuous where the linear range meets the exponents.
"""

import numpy as np
import pytest

from oracle import cg as ocg
from oracle import train as otr

IRREPS = "3x0e+2x1o+2x2e"


def _case(rng, n=3, irreps=IRREPS):
    dim, chan = otr.sizes(irreps)
    f = lambda *s: rng.standard_normal(s)  # noqa: E731
    return dict(h=f(n, dim), z=f(n, dim), q=f(n, chan), post=1 + 0.3 * f(chan), scale=f(chan), pre=1 + 0.3 * f(chan))


@pytest.mark.parametrize("act", ["none", "identity", "sigmoid", "silu"])
@pytest.mark.parametrize("pre_norm,post_norm", [(True, True), (True, False), (False, True)])
def test_backward_matches_differences(act, pre_norm, post_norm):
    rng = np.random.default_rng(5)
    c = _case(rng)
    kw = dict(act=act, pre_norm=pre_norm, post_norm=post_norm, alpha=0.7, eps=1e-3)
    dim, _ = otr.sizes(IRREPS)
    gout, gy = rng.standard_normal((3, dim)), rng.standard_normal((3, dim))

    def loss(c):
        out, y = otr.resnorm_forward(IRREPS, **c, **kw)
        return (out * gout).sum() + (0.0 if y is None else (y * gy).sum())

    x, _ = otr.resnorm_forward(IRREPS, **c, **kw)
    got = otr.resnorm_backward(IRREPS, gout, gy, x, c["z"], c["q"], c["post"], c["scale"], c["pre"], **kw)
    for name, g in zip(("h", "z", "q", "post", "scale", "pre"), got):
        if name == "pre" and not pre_norm:
            continue
        num = np.zeros_like(c[name])
        for i in np.ndindex(num.shape):
            d = {s: {k: v.copy() for k, v in c.items()} for s in (1, -1)}
            for s in d:
                d[s][name][i] += s * 1e-6
            num[i] = (loss(d[1]) - loss(d[-1])) / 2e-6
        # central differences: truncation 1e-12 x third derivative, rounding 1e-16 / 1e-6
        assert np.abs(num - g).max() < 1e-7 * max(1.0, np.abs(g).max()), name


def test_norm_is_equivariant():
    rng = np.random.default_rng(6)
    c = _case(rng, n=2, irreps="4x1o")
    axis = rng.standard_normal(3)
    R = ocg.wigner_d_real(1, axis / np.linalg.norm(axis), 1.1)
    turn = lambda x: (x.reshape(2, 4, 3) @ R.T).reshape(2, -1)  # noqa: E731
    out, y = otr.resnorm_forward("4x1o", **c, act="silu")
    out2, y2 = otr.resnorm_forward("4x1o", **dict(c, h=turn(c["h"]), z=turn(c["z"])), act="silu")
    assert np.abs(turn(out) - out2).max() < 1e-13 and np.abs(turn(y) - y2).max() < 1e-13


def test_adamw_first_step_moves_by_the_rate():
    # from zero states the corrected averages are g and g^2: the step is lr sign(g) for eps = 0
    g = np.array([3.0, -0.01, 1e-5])
    p, m, v = otr.adamw(np.ones(3), g, np.zeros(3), np.zeros(3), 0.1, (0.9, 0.999), 0.0, 0.5, 1)
    assert np.allclose(p, (1 - 0.05) - 0.1 * np.sign(g), rtol=1e-12)
    assert np.allclose(m, 0.1 * g) and np.allclose(v, 0.001 * g * g)


@pytest.mark.parametrize("top", [15, 31])
def test_code_tables(top):
    t = otr.code_table(top)
    assert t[0] == 0 and np.all(np.diff(t) > 0) and len(t) == 8 * (top + 1)
    assert t[8] - t[7] == t[1]           # no jump above the linear range
    assert t[-1] == 1.875 and t[-8] == 1.0
