"""Gated residual norm on the GPU against the FP64 oracle.

Tolerances.  u = 2^-24 (FP32) or 2^-53 (FP64).  A block sum over n_b elements is a tree over at
most 256 threads of sequential sums: for the sizes here its relative error stays below 24 u, and an
element passes through fewer than 20 further roundings and one exponential (2 u), each relative to the
largest term that enters it.  K = 64 u times that term bounds all of it.  Outputs stored in
bfloat16 add one rounding, 2^-8 of the value.  Sums over rows: the same K u times the sum of the
terms' magnitudes (the longest sequential sum here has 32 rows).
"""

import numpy as np
import pytest

from oracle import train as otr

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

K = 64
MANY = "+".join(["4x0e", "3x1o", "2x2e"] * 14)
MORE = "+".join(["4x0e", "3x1o", "2x2e", "40x0e", "33x1o", "1x7o"] * 13)
IRREPS = ["128x0e+128x1o+128x2e", "64x0e+64x1o+64x2e", "128x0e+128x3o", "8x0e+8x1o", "1x0e", "1x3o", "33x0e+17x1o+5x2e", "32x0e+32x1o+32x2e+32x3o", "3x7o+2x4e+1x0e+5x6e+2x5o",
          "300x0e", "16x0e+16x1o+16x2e+16x3o+16x4e+16x5o+16x6e+16x7o"]
KINDS = ["f32", "f64", "bf16", "bf16s"]


def cg():
    import clebsch_gordan_tensor_racah_gb300 as m
    return m


def _plan(irreps, kind, **kw):
    dtype = {"f32": torch.float32, "f64": torch.float64}.get(kind, torch.bfloat16)
    return cg().ResNormPlan(irreps, dtype=dtype, storage=kind == "bf16s", **kw)


def _unit(kind):
    return 2.0 ** -53 if kind == "f64" else 2.0 ** -24


def _dev(a, dtype, layout):
    """Rows on the GPU: contiguous, a column range of wider rows, or one that starts off 16 bytes."""
    t = torch.from_numpy(np.ascontiguousarray(a)).to("cuda").to(dtype)
    if layout == "plain" or t.dim() == 1:
        return t
    left, right = (8, 24) if layout == "range" else (3, 2)
    wide = torch.full((t.shape[0], t.shape[1] + left + right), 7.0, dtype=dtype, device="cuda")
    wide[:, left:left + t.shape[1]] = t
    return wide[:, left:left + t.shape[1]]


def _num(t):
    return None if t is None else t.double().cpu().numpy()


def _inputs(plan, irreps, n, rng, layout, act, has_h=True, has_z=True, factors=True):
    dim, chan = otr.sizes(irreps)
    f = rng.standard_normal
    rows = {}
    rows["h"] = f((n, dim)) * 2 if has_h else None
    rows["z"] = f((n, dim)) * np.exp(f((n, 1))) if has_z else None
    if has_z and n:
        rows["z"][::5] = 0.0           # receivers without edges
    rows["q"] = 3 * f((n, chan)) if has_z and act != "none" else None
    rows["gout"], rows["gy"] = f((n, dim)), f((n, dim))
    t = {k: None if v is None else _dev(v, plan.stream_dtype if k in ("h", "gout") else plan.in_dtype, layout)
         for k, v in rows.items()}
    for k in ("post", "scale", "pre"):
        t[k] = _dev(1 + 0.4 * f(chan), plan.param_dtype, "plain") if factors else None
    if not plan.pre_norm:
        t["gy"] = None
    return t


def _oracle_args(t):
    return dict(z=_num(t["z"]), q=_num(t["q"]), post=_num(t["post"]), scale=_num(t["scale"]), pre=_num(t["pre"]))


def _close(got, want, bound, kind_dtype, what):
    """|got - want| <= bound (+ the rounding of a bfloat16 result), bound broadcast over the row."""
    got = _num(got)
    tol = bound + (2.0 ** -8 * np.abs(want) if kind_dtype == torch.bfloat16 else 0.0) + 1e-300
    worst = np.abs(got - want) / tol
    assert got.shape == want.shape and np.all(worst <= 1), f"{what}: {np.nanmax(worst):.3g} x the bound"


def _rowmax(a):
    return np.abs(a).max(axis=1, keepdims=True) if a.size else np.zeros((a.shape[0], 1))


def check(irreps, kind, n, layout="plain", act="sigmoid", pre_norm=True, post_norm=True, has_h=True, has_z=True,
          factors=True, alpha=1.0, eps=1e-5, seed=0, row_units=K):
    rng = np.random.default_rng(seed + n)
    opt = dict(act=act, pre_norm=pre_norm, post_norm=post_norm, alpha=alpha, eps=eps)
    plan = _plan(irreps, kind, **opt)
    t = _inputs(plan, irreps, n, rng, layout, act, has_h, has_z, factors)
    u = K * _unit(kind)
    fac = dict(post=t["post"], scale=t["scale"], pre=t["pre"])
    out, y = cg().cgtp_resnorm_forward(plan, t["h"], t["z"], t["q"], **fac)
    o = _oracle_args(t)
    dim, chan = otr.sizes(irreps)
    want, _ = otr.resnorm_forward(irreps, h=_num(t["h"]), **o, **opt)
    if has_z:
        _close(out, want, u * (_rowmax(want) + (abs(alpha) * _rowmax(_num(t["h"])) if has_h else 0)), plan.stream_dtype, "out")
    else:
        assert out is t["h"]
    if pre_norm:
        x = _num(out)                  # the norm is of the stream as it is stored
        _, want = otr.resnorm_forward(irreps, h=x, pre=o["pre"], pre_norm=True, eps=eps)
        _close(y, want, u * np.abs(want).max(initial=0.0), plan.out_dtype, "y")
    # backward
    grads = cg().cgtp_resnorm_backward(plan, t["gout"], t["gy"], out, t["z"], t["q"], **fac)
    args = (_num(t["gout"]), _num(t["gy"]), _num(out), o["z"], o["q"], o["post"], o["scale"], o["pre"])
    want = otr.resnorm_backward(irreps, *args, **opt)
    # the largest terms that enter a row of d, of gz and of gq
    pre = np.ones(chan) if o["pre"] is None else o["pre"]
    base = (np.ones(chan) if o["post"] is None else o["post"]) * (1.0 if o["scale"] is None else o["scale"])
    d = _rowmax(args[0])
    if pre_norm:
        least = np.full((n, 1), np.inf)
        for e, _, _, _ in otr._blocks(irreps):
            least = np.minimum(least, np.sqrt((args[2][:, e] ** 2).mean(axis=1, keepdims=True) + eps))
        d = d + 2 * np.abs(pre).max() * _rowmax(args[1]) / least * np.maximum(1, _rowmax(args[2]) / least)
    _close(grads[0], want[0], u * abs(alpha) * d, plan.stream_dtype, "gh")
    if has_z:
        a, da = otr.gate(act, o["q"]) if act != "none" else (np.ones((n, chan)), np.zeros((n, chan)))
        r, zr = np.zeros((n, 1)), np.zeros((n, 1))
        for e, _, _, _ in otr._blocks(irreps):
            s = 1 / np.sqrt((o["z"][:, e] ** 2).mean(axis=1, keepdims=True) + eps) if post_norm else np.ones((n, 1))
            r, zr = np.maximum(r, s), np.maximum(zr, s * _rowmax(o["z"][:, e]))
        w = _rowmax(base * a)
        _close(grads[1], want[1], u * 2 * r * w * d * np.maximum(1, zr ** 2), plan.out_dtype, "gz")
        if act != "none":
            # a'(q) of silu and sigmoid is a difference of numbers of size 1
            _close(grads[2], want[2], u * 15 * d * zr * np.abs(base).max() * np.maximum(1, _rowmax(da)), plan.out_dtype, "gq")
    if n == 0 or not factors:
        assert all(g is None for g in grads[3:]) if not factors else all(not g.any() for g in grads[3:])
        return
    amax = d * (zr * _rowmax(a) if has_z else 0)
    terms = 15 * amax.sum()            # at most 15 components a channel
    u = row_units * _unit(kind)
    for i, (name, other) in enumerate((("gpost", o["scale"]), ("gscale", o["post"]))):
        if has_z:
            _close(grads[3 + i], want[3 + i], u * terms * np.abs(other).max(), None, name)
    if pre_norm:
        mag = np.zeros(chan)
        for e, c, mul, dd in otr._blocks(irreps):
            b, k = args[2][:, e].reshape(n, mul, dd), args[1][:, e].reshape(n, mul, dd)
            p = 1 / np.sqrt((b ** 2).mean(axis=(1, 2), keepdims=True) + eps)
            mag[c] = np.abs(p * b * k).sum(axis=(0, 2))
        _close(grads[5], want[5], u * mag.max(), None, "gpre")


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("irreps", IRREPS)
def test_matches_oracle(irreps, kind):
    for n in (1, 7, 130):
        check(irreps, kind, n)


@pytest.mark.parametrize("irreps", ["700x0e+700x1o+701x2e", "5000x0e", MANY, MORE, "64x0e+64x1o+64x2e+64x3o+64x4e+64x5o+64x6e+64x7o"])
def test_wide_rows_and_many_blocks(irreps):
    check(irreps, "f32", 9)
    check(irreps, "bf16", 9, layout="range")
    check(irreps, "f64", 3)


@pytest.mark.parametrize("layout", ["plain", "range", "odd"])
@pytest.mark.parametrize("kind", KINDS)
def test_layouts_and_row_counts(kind, layout):
    for n in (0, 1, 2, 33, 64, 65):
        check("33x0e+17x1o+5x2e", kind, n, layout=layout, act="silu")
        check("16x0e+16x1o", kind, n, layout=layout, act="identity")


@pytest.mark.parametrize("act", ["none", "identity", "sigmoid", "silu"])
@pytest.mark.parametrize("has_h,has_z,pre_norm,post_norm", [
    (True, True, True, True), (True, True, True, False), (True, True, False, True), (True, True, False, False),
    (False, True, True, True), (False, True, False, True), (True, False, True, True)])
def test_parts(act, has_h, has_z, pre_norm, post_norm):
    for kind in ("f32", "bf16"):
        check("12x0e+7x1o+9x2e", kind, 21, act=act, has_h=has_h, has_z=has_z, pre_norm=pre_norm, post_norm=post_norm,
              alpha=0.6, eps=1e-3)
        check("12x0e+7x1o+9x2e", kind, 21, act=act, has_h=has_h, has_z=has_z, pre_norm=pre_norm, post_norm=post_norm,
              factors=False)


@pytest.mark.parametrize("irreps,n", [
    ("64x0e+64x1o+64x2e", 5001), ("128x0e+128x1o+128x2e", 3001), ("128x0e+128x3o", 3003), ("16x0e+16x1o+16x7o", 5003),
    ("8x0e+8x1o", 40001), ("33x0e+17x1o+5x2e", 20001), ("1024x0e", 1001), ("3x1o", 30001), ("4x0e", 1003), ("2x0e+2x1o", 777), (MORE, 301), (MANY, 5001)])
@pytest.mark.parametrize("kind,layout", [("f32", "plain"), ("bf16", "range"), ("bf16s", "plain"), ("f32", "odd")])
def test_more_rows_than_one_turn_of_the_grid(irreps, n, kind, layout):
    # every group takes several tiles, with a last one that is not full.  Sums over rows have up to 250
    # additions in a row (a group's rows, 128 rows side by side or groups of a CTA, CTAs): 256 u of the terms.
    check(irreps, kind, n, layout=layout, act="silu", seed=11, row_units=256)


def test_many_rows_sum_in_a_fixed_order():
    irreps, n = "32x0e+32x1o+32x2e", 40000
    plan = _plan(irreps, "f32", act="sigmoid")
    t = _inputs(plan, irreps, n, np.random.default_rng(3), "plain", "sigmoid")
    fac = dict(post=t["post"], scale=t["scale"], pre=t["pre"])
    runs = []
    for _ in range(2):
        out, y = cg().cgtp_resnorm_forward(plan, t["h"], t["z"], t["q"], **fac)
        runs.append((out, y) + cg().cgtp_resnorm_backward(plan, t["gout"], t["gy"], out, t["z"], t["q"], **fac))
    for a, b in zip(*runs):
        assert torch.equal(a, b)
    o = _oracle_args(t)
    want = otr.resnorm_backward(irreps, _num(t["gout"]), _num(t["gy"]), _num(runs[0][0]), o["z"], o["q"], o["post"],
                                o["scale"], o["pre"], act="sigmoid")
    for got, ref in zip(runs[0][5:], want[3:]):
        # 40,000 terms of random sign: sequential parts of at most 300 rows, each sum below 300 x its
        # largest term; 5 standard deviations of their rounding stay below 1e-5 of the largest sum
        assert np.abs(_num(got) - ref).max() <= 1e-5 * np.abs(ref).max()


def test_gradients_against_differences_of_the_kernel():
    irreps, n = "3x0e+2x1o+2x2e", 3
    plan = _plan(irreps, "f64", act="silu", alpha=0.8, eps=1e-3)
    t = _inputs(plan, irreps, n, np.random.default_rng(4), "plain", "silu")
    t["z"] = t["z"] + 0.5

    def loss(t):
        out, y = cg().cgtp_resnorm_forward(plan, t["h"], t["z"], t["q"], post=t["post"], scale=t["scale"], pre=t["pre"])
        return out, float((out * t["gout"]).sum() + (y * t["gy"]).sum())

    out, _ = loss(t)
    grads = cg().cgtp_resnorm_backward(plan, t["gout"], t["gy"], out, t["z"], t["q"], post=t["post"], scale=t["scale"], pre=t["pre"])
    for name, g in zip(("h", "z", "q", "post", "scale", "pre"), grads):
        for i in range(t[name].numel()):
            at = []
            for s in (1e-6, -1e-6):
                moved = dict(t, **{name: t[name].clone()})
                moved[name].view(-1)[i] += s
                at.append(loss(moved)[1])
            assert abs((at[0] - at[1]) / 2e-6 - float(g.view(-1)[i])) < 1e-7 * max(1.0, float(g.abs().max())), (name, i)


def test_a_bad_row_stays_alone():
    irreps = "20x0e+9x1o"
    for kind in ("f32", "bf16s"):
        plan = _plan(irreps, kind, act="silu")
        t = _inputs(plan, irreps, 50, np.random.default_rng(5), "plain", "silu")
        fac = dict(post=t["post"], scale=t["scale"], pre=t["pre"])
        good = cg().cgtp_resnorm_forward(plan, t["h"], t["z"], t["q"], **fac)
        gg = cg().cgtp_resnorm_backward(plan, t["gout"], t["gy"], good[0], t["z"], t["q"], **fac)
        z = t["z"].clone()
        z[11, 3], z[12, 20], z[13, 0] = float("nan"), float("inf"), torch.finfo(z.dtype).min
        bad = cg().cgtp_resnorm_forward(plan, t["h"], z, t["q"], **fac)
        bg = cg().cgtp_resnorm_backward(plan, t["gout"], t["gy"], good[0], z, t["q"], **fac)
        keep = torch.ones(50, dtype=torch.bool, device="cuda")
        keep[11:14] = False
        for a, b in list(zip(good, bad)) + list(zip(gg[:3], bg[:3])):
            assert torch.equal(a[keep], b[keep])
        assert bool(torch.isnan(bad[0][11, :20]).any()) and bool(torch.isfinite(bad[0][11, 20:]).all())


def test_gates_far_out_stay_finite():
    irreps = "4x0e"
    plan = _plan(irreps, "f32", act="silu")
    q = torch.tensor([[200.0, -200.0, 88.8, -104.0]], device="cuda")
    h, z = torch.zeros(1, 4, device="cuda"), torch.ones(1, 4, device="cuda")
    out, y = cg().cgtp_resnorm_forward(plan, h, z, q)
    g = cg().cgtp_resnorm_backward(plan, z, z, out, z, q)
    assert all(bool(torch.isfinite(v).all()) for v in (out, y) + g[:3])
    assert abs(float(out[0, 0]) - 200.0) < 1e-2 and float(out[0, 1]) == 0.0


def test_offsets_beyond_32_bits():
    irreps, n, ld = "8x0e+8x1o", 3, (1 << 30) + 4096
    plan = _plan(irreps, "bf16s", act="sigmoid")
    wide = torch.empty(n, ld, dtype=torch.bfloat16, device="cuda")
    t = _inputs(plan, irreps, n, np.random.default_rng(6), "plain", "sigmoid")
    h, z, q = wide[:, :32], wide[:, 64:96], wide[:, 128:144]
    h.copy_(t["h"]), z.copy_(t["z"]), q.copy_(t["q"])
    out, y = wide[:, 192:224], wide[:, 256:288]
    cg().cgtp_resnorm_forward(plan, h, z, q, out=out, y=y)
    a, b = cg().cgtp_resnorm_forward(plan, t["h"], t["z"], t["q"])
    assert torch.equal(out, a) and torch.equal(y, b)
    gz = wide[:, 320:352]
    gh, _, gq, _, _, _ = cg().cgtp_resnorm_backward(plan, h, z, out, z, q, outs=(torch.empty_like(a), gz, torch.empty_like(t["q"]), None, None, None))
    want = cg().cgtp_resnorm_backward(plan, t["h"], t["z"], a, t["z"], t["q"])
    assert torch.equal(gh, want[0]) and torch.equal(gz, want[1]) and torch.equal(gq, want[2])


def test_another_stream():
    irreps = "64x0e+64x1o"
    plan = _plan(irreps, "f32", act="none")
    t = _inputs(plan, irreps, 3000, np.random.default_rng(7), "plain", "none")
    want = cg().cgtp_resnorm_forward(plan, t["h"], t["z"], post=t["post"], scale=t["scale"], pre=t["pre"])
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        z = t["z"] * 1.0
        got = cg().cgtp_resnorm_forward(plan, t["h"], z, post=t["post"], scale=t["scale"], pre=t["pre"])
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    # a stream given by name, while another is current
    with torch.cuda.stream(s):
        z = t["z"] * 1.0
    got = cg().cgtp_resnorm_forward(plan, t["h"], z, post=t["post"], scale=t["scale"], pre=t["pre"], stream=s)
    grads = cg().cgtp_resnorm_backward(plan, t["gout"], t["gy"], got[0], z, post=t["post"], scale=t["scale"], pre=t["pre"], stream=s)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    ref = cg().cgtp_resnorm_backward(plan, t["gout"], t["gy"], want[0], t["z"], post=t["post"], scale=t["scale"], pre=t["pre"])
    assert all(a is None or torch.equal(a, b) for a, b in zip(grads, ref))


def test_nothing_outside_the_rows_is_written():
    irreps, n = "33x0e+17x1o+5x2e", 37
    dim, chan = otr.sizes(irreps)
    for kind in KINDS:
        plan = _plan(irreps, kind, act="silu")
        for layout in ("range", "odd"):
            t = _inputs(plan, irreps, n, np.random.default_rng(8), layout, "silu")
            blank = lambda w, dt: _dev(np.zeros((n, w)), dt, layout)  # noqa: E731, B023
            out, y = blank(dim, plan.stream_dtype), blank(dim, plan.out_dtype)
            cg().cgtp_resnorm_forward(plan, t["h"], t["z"], t["q"], out=out, y=y)
            gh, gz, gq = blank(dim, plan.stream_dtype), blank(dim, plan.out_dtype), blank(chan, plan.out_dtype)
            cg().cgtp_resnorm_backward(plan, t["gout"], t["gy"], out, t["z"], t["q"], outs=(gh, gz, gq, None, None, None))
            for v in (out, y, gh, gz, gq):
                base = v._base
                left = 8 if layout == "range" else 3
                assert bool((base[:, :left] == 7).all()) and bool((base[:, left + v.shape[1]:] == 7).all())


def test_refusals():
    m = cg()
    plan = _plan("4x0e+4x1o", "f32", act="sigmoid")
    h = torch.zeros(5, 16, device="cuda")
    q = torch.zeros(5, 8, device="cuda")
    bad = [
        (ValueError, lambda: m.cgtp_resnorm_forward(plan, None)),
        (ValueError, lambda: m.cgtp_resnorm_forward(plan, h[:, :12], h, q)),
        (TypeError, lambda: m.cgtp_resnorm_forward(plan, h.double(), h, q)),
        (TypeError, lambda: m.cgtp_resnorm_forward(plan, h.cpu(), h, q)),
        (ValueError, lambda: m.cgtp_resnorm_forward(plan, h[:1].expand(5, 16), h, q)),       # rows overlap
        (ValueError, lambda: m.cgtp_resnorm_forward(plan, h, torch.zeros(16, 5, device="cuda").t(), q)),
        (ValueError, lambda: m.cgtp_resnorm_forward(plan, h, h, q, pre=torch.ones(7, device="cuda"))),
        (m.CgtpError, lambda: m.cgtp_resnorm_forward(plan, h, h)),                            # no gates
        (m.CgtpError, lambda: m.cgtp_resnorm_backward(plan, h, None, h, h, q)),               # gy is needed
        (m.CgtpError, lambda: m.cgtp_resnorm_backward(plan, h, h, None, h, q)),               # x is needed
        (ValueError, lambda: m.cgtp_resnorm_backward(plan, None, None, h, h, q)),
    ]
    for kind, call in bad:
        with pytest.raises(kind):
            call()
