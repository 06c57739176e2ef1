"""Operators of a training step at the ends of their ranges, as far as that needs no GPU."""

import numpy as np

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
