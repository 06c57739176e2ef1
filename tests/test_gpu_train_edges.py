"""Operators of a training step at the ends of their ranges: norms without z, norms of tiny blocks, far
gates, small eps and small decays."""

import numpy as np
import pytest

from oracle import train as otr

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

KINDS = ["f32", "f64", "bf16", "bf16s"]


def cg():
    import clebsch_gordan_tensor_racah_gb300 as m
    return m


def _plan(irreps, kind, **kw):
    dtype = {"f32": torch.float32, "f64": torch.float64}.get(kind, torch.bfloat16)
    return cg().ResNormPlan(irreps, dtype=dtype, storage=kind == "bf16s", **kw)


def _num(t):
    return t.double().cpu().numpy()


def _rowmax(a):
    return np.abs(a).max(axis=1, keepdims=True)


# staged rows (several rows a warp, a warp a row, several warps a row) and rows read in place
@pytest.mark.parametrize("irreps", ["4x0e+3x1o", "64x0e+64x1o", "128x0e+128x1o+128x2e", "300x0e", "5000x0e"])
@pytest.mark.parametrize("kind", KINDS)
def test_without_z_the_residual_factor_has_no_gradient(irreps, kind):
    # the stream is h itself, so gh = gout where y has no gradient: exactly, as p (pre 0 - 0 x) = 0
    for pre_norm in (True, False):
        plan = _plan(irreps, kind, alpha=0.6, pre_norm=pre_norm)
        gen = torch.Generator(device="cuda").manual_seed(1)
        h, gout = (torch.randn(9, plan.dim, device="cuda", generator=gen).to(plan.stream_dtype) for _ in range(2))
        gy = torch.zeros(9, plan.dim, device="cuda", dtype=plan.in_dtype) if pre_norm else None
        gh = cg().cgtp_resnorm_backward(plan, gout, gy, h)[0]
        assert torch.equal(gh, gout)


@pytest.mark.parametrize("irreps", ["3x0e+2x1o+2x2e", "4500x0e"])
def test_gradients_without_z_against_differences_of_the_kernel(irreps):
    plan = _plan(irreps, "f64", alpha=0.6, eps=1e-3)
    rng = np.random.default_rng(4)
    dev = lambda a: torch.from_numpy(a).cuda()  # noqa: E731
    h, gout, gy = (dev(rng.standard_normal((3, plan.dim))) for _ in range(3))
    pre = dev(1 + 0.3 * rng.standard_normal(plan.channels))

    def loss(h):
        out, y = cg().cgtp_resnorm_forward(plan, h, pre=pre)
        return float((out * gout).sum() + (y * gy).sum())

    gh = cg().cgtp_resnorm_backward(plan, gout, gy, h, pre=pre)[0].view(-1)
    for i in range(0, h.numel(), max(1, h.numel() // 40)):
        at = []
        for s in (1e-5, -1e-5):
            moved = h.clone()
            moved.view(-1)[i] += s
            at.append(loss(moved))
        # the loss is a sum of up to 13,500 terms of size 1: 1e-13 of it over 2e-5, and the third derivative x 1e-10
        assert abs((at[0] - at[1]) / 2e-5 - float(gh[i])) < 1e-6, i
