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


@pytest.mark.parametrize("irreps", ["8x0e+4x1o", "64x0e+64x1o", "128x0e+128x1o+128x2e", "5000x0e"])
@pytest.mark.parametrize("eps,size", [(1e-26, 0.0), (1e-30, 0.0), (1e-37, 0.0), (0.0, 1e-13), (0.0, 1e-15), (1e-30, 1e-14)])
@pytest.mark.parametrize("has_z", [False, True])
def test_tiny_blocks_and_small_eps(irreps, eps, size, has_z):
    # The inverse rms p is up to 3e18 here, and every gradient is a number that FP32 holds: where z is given, z is of
    # size 1 and alpha = 0, so that x = out = w z stays normal or, with w = size, as small as without z.
    # 64 u of the largest term of a row of d (the terms of d are of size |gout| + 2 p |pre gy|): see the derivation
    # with the other norm tests.
    rng = np.random.default_rng(3)
    plan = _plan(irreps, "f32", alpha=0.0, eps=eps, post_norm=has_z)
    dim, chan = plan.dim, plan.channels
    dev = lambda a: torch.from_numpy(a.astype(np.float32)).cuda()  # noqa: E731
    f = rng.standard_normal
    x, gout, gy, pre = dev(f((5, dim)) * size), dev(f((5, dim))), dev(f((5, dim))), dev(1 + 0.3 * f(chan))
    z = dev(f((5, dim))) if has_z else None
    scale = dev(np.full(chan, size)) if has_z else None
    if has_z:
        x = cg().cgtp_resnorm_forward(plan, None, z, scale=scale, pre=pre)[0]
    got = cg().cgtp_resnorm_backward(plan, gout, gy, x, z, scale=scale, pre=pre, need_gh=True)
    o = [_num(t) for t in (gout, gy, x)]
    want = otr.resnorm_backward(irreps, *o, z=None if z is None else _num(z), scale=None if z is None else _num(scale), pre=_num(pre),
                                alpha=0.0, eps=eps, post_norm=has_z)
    u = 64 * 2.0 ** -24
    at = 0
    for mul, d in otr.parse(irreps):
        cut = slice(at, at + mul * d)
        at += mul * d
        rms = np.sqrt((o[2][:, cut] ** 2).mean(axis=1, keepdims=True) + eps)
        bound = _rowmax(o[0][:, cut]) + 2 * np.abs(_num(pre)).max() * _rowmax(o[1][:, cut]) / rms * np.maximum(1, _rowmax(o[2][:, cut]) / rms)
        if not has_z:
            assert np.all(np.abs(_num(got[0])[:, cut] - want[0][:, cut]) <= u * bound)
        else:
            zb = _num(z)[:, cut]
            r = 1 / np.sqrt((zb ** 2).mean(axis=1, keepdims=True) + eps)
            assert np.all(np.abs(_num(got[1])[:, cut] - want[1][:, cut]) <= u * 2 * r * size * bound * np.maximum(1, (r * _rowmax(zb)) ** 2) + 1e-37)
    assert all(g is None or bool(torch.isfinite(g).all()) for g in got)


@pytest.mark.parametrize("irreps", ["8x0e+4x1o", "128x0e+128x1o+128x2e", "5000x0e"])
def test_zero_z_and_small_eps(irreps):
    # a block of zeros under the rms of z: out = alpha h, gz = r w d with r = 3e19, d = gout: finite
    plan = _plan(irreps, "f32", pre_norm=False, eps=1e-39)
    gen = torch.Generator(device="cuda").manual_seed(5)
    h, gout = (torch.randn(4, plan.dim, device="cuda", generator=gen) for _ in range(2))
    z = torch.zeros_like(h)
    out, _ = cg().cgtp_resnorm_forward(plan, h, z)
    assert torch.equal(out, h)
    gh, gz, _, _, _, _ = cg().cgtp_resnorm_backward(plan, gout, None, out, z)
    assert torch.equal(gh, gout)
    want = _num(gout) / np.sqrt(float(np.float32(1e-39)))
    assert np.all(np.abs(_num(gz) - want) <= 8 * 2.0 ** -24 * np.abs(want))


def test_first_calls_on_another_stream():
    # a plan's and an optimizer's tables are there when they are made, whatever stream the first call is on
    side = torch.cuda.Stream()
    rng = np.random.default_rng(2)
    irreps = "+".join(["4x0e", "3x1o", "2x2e"] * 40)       # more blocks than travel in the kernel's parameters
    numel = [int(v) for v in rng.integers(1, 40000, size=1500)]
    g = [torch.from_numpy(rng.standard_normal(k)).float().cuda() for k in numel]
    h, pre = torch.randn(500, otr.sizes(irreps)[0], device="cuda"), torch.ones(otr.sizes(irreps)[1], device="cuda")
    torch.cuda.synchronize()
    runs = []
    for stream in (None, side, side, side):
        plan = _plan(irreps, "f32")
        opt = cg().AdamW(numel)
        clip = cg().cgtp_grad_norm(opt, g, 1.0, stream=stream)
        y = cg().cgtp_resnorm_forward(plan, h, stream=stream)[1]
        gpre = cg().cgtp_resnorm_backward(plan, h, h, h, pre=pre, stream=stream)[5]
        torch.cuda.synchronize()
        runs.append((clip, y, gpre))
    for got in runs[1:]:
        assert all(torch.equal(a, b) for a, b in zip(got, runs[0]))


@pytest.mark.parametrize("act", ["sigmoid", "silu"])
def test_far_gates_keep_their_relative_accuracy(act):
    # An exponential and a reciprocal (a unit in the last place, 2 u, each), a sum and two products (u each): 8 u; the gradient
    # s (1 - s) or s (1 + q (1 - s)) has another four roundings.  Both without cancellation for q <= -2 (silu: 1 + q (1 - s)
    # is below -0.76 there, and the error of q (1 - s) at most 4 times its size).
    q = torch.linspace(-86.0, 40.0, 4096, device="cuda")[None, :].contiguous()
    plan = cg().ResNormPlan("4096x0e", act=act, pre_norm=False, post_norm=False)
    one = torch.ones_like(q)
    out, _ = cg().cgtp_resnorm_forward(plan, None, one, q)
    u, x = 2.0 ** -24, _num(q)
    s = 1 / (1 + np.exp(-x))
    want = s if act == "sigmoid" else x * s
    assert (np.abs(_num(out) - want) / np.abs(want)).max() <= 8 * u
    gq = _num(cg().cgtp_resnorm_backward(plan, one, None, None, one, q, need_gh=False)[2])
    want = s * (1 - s) if act == "sigmoid" else s * (1 + x * (1 - s))
    low = x <= -2
    assert (np.abs(gq - want)[low] / np.abs(want[low])).max() <= (8 + 4 * (1 if act == "sigmoid" else 4)) * u


@pytest.mark.parametrize("state_kind", ["f32", "8bit"])
@pytest.mark.parametrize("beta2", [0.999, 0.99999])
def test_small_averages_under_a_small_eps(state_kind, beta2):
    # From zero states the step is lr |g| / (|g| + eps).  v = (1 - beta2) g^2 just below the smallest normal float keeps
    # 22 bits, of which the root halves the error; 16 u for the step's other roundings: 2^-20 in all.
    size = (0.9 * 2.0 ** -126 / (1 - beta2)) ** 0.5
    for eps in (1e-12, 1e-11, 1e-10, 1e-9):
        g, p = [torch.full((200,), size, device="cuda")], [torch.zeros(200, device="cuda")]
        opt = cg().AdamW([200], state=state_kind)
        cg().cgtp_adamw_step(opt, p, g, opt.new_state(), lr=1e-2, betas=(0.9, beta2), eps=eps, step=1)
        g64 = float(g[0][0])
        want = 1e-2 * g64 / (g64 + eps)
        assert float((p[0].double() + want).abs().max()) <= 2.0 ** -20 * want, (eps, float(p[0][0]), want)


@pytest.mark.parametrize("state_kind,dtype", [("f32", "float32"), ("f32", "float64"), ("8bit", "float32")])
@pytest.mark.parametrize("lr,wd", [(1e-3, 1e-4), (1e-4, 1e-4), (1e-5, 1e-2), (1e-3, 1e-2)])
def test_small_decays_act_in_the_mean(state_kind, dtype, lr, wd):
    # lr wd down to 1e-8, far below the rounding of 1 - lr wd.  The parameters lie in [1, 2) and a moving step of random
    # size makes the rounding of each new value independent: its standard deviation is 2^-23 / sqrt(12), and the mean over 2^20
    # elements stays within 5 x 2^-23 / sqrt(12) / 2^10 = 1.7e-10.  The step itself has errors of at most 16 u of its size
    # that are odd in m: 16 u lr / 2^10 in the mean.
    k = 1 << 20
    dtype = getattr(torch, dtype)
    gen = torch.Generator(device="cuda").manual_seed(7)
    p = [1 + torch.rand(k, device="cuda", generator=gen, dtype=dtype)]
    opt = cg().AdamW([k], param_dtype=dtype, state=state_kind)
    state = opt.new_state()
    if state_kind == "8bit":
        state["m"].copy_(torch.randint(0, 256, (k,), device="cuda", generator=gen))
        state["m_exp"].fill_(126)
        state["v"].fill_(8 * 31)
        state["v_exp"].fill_(127)
    else:
        state["m"].copy_(2 * torch.rand(k, device="cuda", generator=gen, dtype=dtype) - 1)
        state["v"].fill_(1.0)
    g = 2 * torch.rand(k, device="cuda", generator=gen, dtype=dtype) - 1
    m, v = cg().cgtp_adamw_state_values(opt, state)
    want, _, _ = otr.adamw(_num(p[0]), _num(g), _num(m), _num(v), lr, (0.9, 0.999), 1e-8, wd, 1000000)
    cg().cgtp_adamw_step(opt, p, [g], state, lr=lr, eps=1e-8, weight_decay=wd, step=1000000)
    assert abs((_num(p[0]) - want).mean()) <= 1.7e-10 + 16 * 2.0 ** -24 * lr / 2 ** 10


def test_infinite_parameters_stay():
    inf = float("inf")
    for state_kind in ("f32", "8bit"):
        for wd in (0.0, 0.1):
            p = [torch.tensor([inf, -inf, 1.0, float("nan")] * 40, device="cuda")]
            opt = cg().AdamW([160], state=state_kind)
            cg().cgtp_adamw_step(opt, p, [torch.ones(160, device="cuda")], opt.new_state(), lr=1e-2, weight_decay=wd, step=1)
            q = p[0].view(-1, 4)
            assert bool((q[:, 0] == inf).all()) and bool((q[:, 1] == -inf).all()) and bool(torch.isfinite(q[:, 2]).all()) and bool(torch.isnan(q[:, 3]).all())


def test_calls_on_another_device_than_the_plans_are_refused():
    # a plan that says that it lives on a second device: its tables would not be where the current device launches
    def moved(o):
        o.device, o._native = torch.device("cuda", 1), o._native[:-1] + (1,)
        return o

    m = cg()
    plan, opt, full = m.ResNormPlan("4x0e+4x1o"), m.AdamW([7], state="8bit"), m.AdamW([7])
    h, g, state = torch.ones(5, 16, device="cuda"), [torch.ones(7, device="cuda")], opt.new_state()
    assert plan.device == opt.device == h.device
    m.cgtp_resnorm_forward(plan, h)
    plan, opt, full = moved(plan), moved(opt), moved(full)
    for call in (lambda: m.cgtp_resnorm_forward(plan, h), lambda: m.cgtp_resnorm_backward(plan, h, h, h),
                 lambda: m.cgtp_grad_norm(opt, g, 1.0), lambda: m.cgtp_adamw_step(opt, g, g, state, lr=1.0),
                 lambda: m.cgtp_adamw_step(full, g, g, full.new_state(), lr=1.0), lambda: m.cgtp_adamw_state_values(opt, state)):
        with pytest.raises(ValueError, match="cuda:1.*cuda:0"):
            call()
    assert bool((g[0] == 1).all()) and not state["m"].any()


def test_out_of_memory_is_torchs_own_error():
    # an allocation that the caching allocator refuses under a limit on this process: nothing is asked of the device
    plan = cg().ResNormPlan("64x0e+64x1o")
    h = torch.zeros(100000, plan.dim, device="cuda")
    torch.cuda.empty_cache()
    total = torch.cuda.get_device_properties(0).total_memory
    torch.cuda.set_per_process_memory_fraction((torch.cuda.memory_reserved() + (1 << 20)) / total)
    try:
        with pytest.raises(torch.OutOfMemoryError):
            cg().cgtp_resnorm_forward(plan, h)
    finally:
        torch.cuda.set_per_process_memory_fraction(1.0)
    assert bool((cg().cgtp_resnorm_forward(plan, h)[1] == 0).all())


def test_gradients_of_extreme_size():
    # 3e38 squared is infinite: v of its block is stored as NaNs, as a block that holds an infinity is.  Its own step is zero
    # (a finite m over an infinite root); the others of the block move by lr |g| / (|g| + eps) with their unrounded v.
    list_ = [3e38, 1e-38, 1e-45, 0.0, -3e38, 1e19, 1e-20, -0.0]
    g = torch.tensor(list_ * 16, device="cuda")
    for state_kind in ("8bit", "f32"):
        opt = cg().AdamW([128], state=state_kind)
        state, p = opt.new_state(), [torch.zeros(128, device="cuda")]
        cg().cgtp_adamw_step(opt, p, [g], state, lr=1e-3, step=1)
        q = p[0].view(16, 8)
        assert bool(torch.isfinite(q).all()) and not q[:, [0, 3, 4, 7]].any()
        assert float((q[:, 5] + 1e-3).abs().max()) <= 16 * 2.0 ** -24 * 1e-3
        m, v = cg().cgtp_adamw_state_values(opt, state)
        assert bool(torch.isfinite(m).all())
        assert bool(torch.isnan(v).all()) if state_kind == "8bit" else bool(torch.isinf(v.view(16, 8)[:, [0, 4]]).all())
        if state_kind == "8bit":      # codes of 8 steps a binade: next to 0.1 g
            assert float((m.view(16, 8)[:, 0] / 3e37 - 1).abs().max()) <= 0.125
    # large numbers whose squares are finite
    g = torch.tensor([1e19, -1e19, 1e18, 3e17] * 32, device="cuda")
    opt = cg().AdamW([128], state="8bit")
    state, p = opt.new_state(), [torch.zeros(128, device="cuda")]
    cg().cgtp_adamw_step(opt, p, [g], state, lr=1e-3, step=1)
    m, v = cg().cgtp_adamw_state_values(opt, state)
    assert float((p[0] + 1e-3 * torch.sign(g)).abs().max()) <= 16 * 2.0 ** -24 * 1e-3
    assert float((m / (0.1 * g) - 1).abs().max()) <= 0.125 and float((v / (1e-3 * g * g) - 1).abs().max()) <= 0.125


@pytest.mark.parametrize("state_kind", ["f32", "8bit"])
def test_passes_in_a_cuda_graph_with_the_step_outside(state_kind):
    # step count, rate and seed are values of the call: a loop that captures its passes and calls the step outside the
    # graph is the eager loop, bit for bit
    torch.manual_seed(6)
    plan = cg().ResNormPlan("64x0e+64x1o", act="silu")
    n, dim, chan = 1000, plan.dim, plan.channels
    h, z, gout, gy = (torch.randn(n, dim, device="cuda") for _ in range(4))
    q, gains = torch.randn(n, chan, device="cuda"), [1 + 0.1 * torch.randn(chan, device="cuda") for _ in range(3)]
    opt = cg().AdamW([chan] * 3, state=state_kind)

    def passes(p):
        out, _ = cg().cgtp_resnorm_forward(plan, h, z, q, post=p[0], scale=p[1], pre=p[2])
        grads = list(cg().cgtp_resnorm_backward(plan, gout, gy, out, z, q, post=p[0], scale=p[1], pre=p[2])[3:])
        return grads, cg().cgtp_grad_norm(opt, grads, 1.0)

    def step(p, state, grads, clip, t):
        cg().cgtp_adamw_step(opt, p, grads, state, lr=1e-2 / t, weight_decay=0.1, step=t, clip=clip, seed=t)

    eager, captured = [g.clone() for g in gains], [g.clone() for g in gains]
    s_eager, s_captured = opt.new_state(), opt.new_state()
    passes(eager)                      # before the capture: the first launch of a kernel sets its attributes
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        grads, clip = passes(captured)
    for t in range(1, 5):
        step(eager, s_eager, *passes(eager), t)
        graph.replay()
        step(captured, s_captured, grads, clip, t)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(eager, captured))
    assert all(a is None or torch.equal(a, s_captured[k]) for k, a in s_eager.items())


@pytest.mark.parametrize("kind", ["f32", "bf16s"])
def test_gates_at_the_ends_of_the_type(kind):
    inf, nan = float("inf"), float("nan")
    dtype = torch.bfloat16 if kind == "bf16s" else torch.float32
    top = float(torch.finfo(dtype).max)
    far = [-(2.0 ** k) * f for k in range(7, 128, 3) for f in (1.0, 1.2578125, 1.734375)]    # exact in both types
    q = torch.tensor([[-inf, inf, nan, -top, top, 0.0, -0.0] + far + [-v for v in far]], device="cuda").to(dtype)
    width = q.shape[1]
    one = torch.ones_like(q)
    n = len(far)
    for act in ("sigmoid", "silu"):
        plan = _plan("%dx0e" % width, kind, act=act, pre_norm=False, post_norm=False)
        out = cg().cgtp_resnorm_forward(plan, None, one, q)[0][0]
        gq = cg().cgtp_resnorm_backward(plan, one, None, None, one, q, need_gh=False)[2][0]
        up = torch.ones(n, device="cuda", dtype=dtype) if act == "sigmoid" else q[0, 7 + n:]
        assert torch.equal(out[7:7 + n], torch.zeros_like(up)) and torch.equal(out[7 + n:], up)
        assert not gq[7:7 + n].any() and torch.equal(gq[7 + n:], torch.full_like(up, 0.0 if act == "sigmoid" else 1.0))
        first = out[:7].tolist()
        assert first[3:] == ([0.0, 1.0, 0.5, 0.5] if act == "sigmoid" else [0.0, top, 0.0, 0.0]) and first[2] != first[2]
        assert first[1] == (1.0 if act == "sigmoid" else inf) and (first[0] == 0.0 if act == "sigmoid" else first[0] != first[0])
        assert gq[3:5].tolist() == [0.0, 0.0 if act == "sigmoid" else 1.0] and bool(torch.isnan(gq[2]))
