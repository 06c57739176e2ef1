"""AdamW, its 8-bit states and the gradient norm on the GPU against the FP64 oracle.

Tolerances.  u = 2^-24 (FP32) or 2^-53.  m and v are sums of two products: 4 u of the larger term.
The parameter: 4 u of p, plus 16 u of the step (a quotient with a square root, the factors rounded
to FP32).  The norm: 64 u (sums of at most 32 squares a thread, then FP64).  A stored 8-bit value lies
at a code next to the exact one: within one step of the grid, 2^-3 of the value or the smallest code.
"""

import numpy as np
import pytest

from oracle import train as otr

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

SHAPES = [(8, 64), (64, 64), (1,), (33,), (127,), (128,), (129,), (0,), (3, 5, 7), (1000,), (70, 1153)]
NUMEL = [int(np.prod(s)) for s in SHAPES]


def cg():
    import clebsch_gordan_tensor_racah_gb300 as m
    return m


def _place(a, dtype, offset):
    """A contiguous tensor that starts `offset` elements after a 16-byte boundary."""
    k = a.size
    flat = torch.full((k + offset + 8,), 7.0, dtype=dtype, device="cuda")
    t = flat[offset:offset + k]
    t.copy_(torch.from_numpy(a.reshape(-1)).to(dtype))
    return t.view(a.shape)


def _sets(rng, dtype, grad_dtype, offset, shapes=SHAPES):
    spread = lambda s: np.exp(rng.standard_normal(s) * 2)  # noqa: E731
    p = [_place(rng.standard_normal(s), dtype, offset) for s in shapes]
    g = [_place(rng.standard_normal(s) * spread(s) * 1e-2, grad_dtype, offset) for s in shapes]
    return p, g


def _num(t):
    return t.double().cpu().numpy()


def _starts(numel):
    return np.concatenate([[0], np.cumsum([-(-k // 128) * 128 for k in numel])]).astype(int)


@pytest.mark.parametrize("offset", [0, 1, 3])
@pytest.mark.parametrize("dtype,grad_dtype,copies", [("float32", "float32", False), ("float32", "bfloat16", True),
                                                     ("float64", "float64", False)])
def test_full_states_match_oracle(dtype, grad_dtype, copies, offset):
    dtype, grad_dtype = getattr(torch, dtype), getattr(torch, grad_dtype)
    rng = np.random.default_rng(offset)
    u = 2.0 ** -53 if dtype == torch.float64 else 2.0 ** -24
    p, g = _sets(rng, dtype, grad_dtype, offset)
    decay = [float(i % 3) for i in range(len(p))]
    opt = cg().AdamW(NUMEL, param_dtype=dtype, grad_dtype=grad_dtype, decay_scale=decay)
    state = opt.new_state()
    co = [_place(np.zeros(s), torch.bfloat16, offset) for s in SHAPES] if copies else None
    starts = _starts(NUMEL)
    assert opt.state_numel == starts[-1]
    kw = dict(lr=1e-2, betas=(0.9, 0.99), eps=1e-6, weight_decay=0.1)
    for step in (1, 2, 3):
        before = [_num(t) for t in p]
        m0, v0 = _num(state["m"]), _num(state["v"])
        clip = cg().cgtp_grad_norm(opt, g, 0.5) if step == 2 else None
        cg().cgtp_adamw_step(opt, p, g, state, step=step, copies=co, clip=clip, **kw)
        coef = 1.0
        if clip is not None:
            n, want = otr.grad_norm([_num(t) for t in g], 0.5)
            assert abs(float(clip[0]) - n) <= 64 * u * n and abs(float(clip[1]) - want) <= 66 * u * want
            coef = float(clip[1])
        m1, v1 = _num(state["m"]), _num(state["v"])
        for i, k in enumerate(NUMEL):
            cut = slice(starts[i], starts[i] + k)
            # with the coefficient the GPU used, the gradient has one more rounding
            q, m, v = otr.adamw(before[i].reshape(-1), _num(g[i]).reshape(-1), m0[cut], v0[cut], 1e-2, (0.9, 0.99), 1e-6,
                                0.1 * decay[i], step, coef)
            gi = coef * np.abs(_num(g[i]).reshape(-1))
            assert np.all(np.abs(m1[cut] - m) <= 4 * u * (np.abs(m0[cut]) + gi))
            assert np.all(np.abs(v1[cut] - v) <= 6 * u * (v0[cut] + gi * gi) + 1e-44)
            move = np.abs(q - before[i].reshape(-1) * (1 - 1e-2 * 0.1 * decay[i]))
            # where m is a difference, its error enters the step as 4 u (|m0| + |g|) / |m| of it
            lost = 4 * u * (np.abs(m0[cut]) + gi) / np.maximum(np.abs(m), 1e-300)
            tol = 4 * u * np.abs(before[i].reshape(-1)) + (16 * u + lost) * move
            assert np.all(np.abs(_num(p[i]).reshape(-1) - q) <= tol)
            if co:
                assert torch.equal(co[i], p[i].to(torch.bfloat16))
            pad = slice(starts[i] + k, starts[i + 1])
            assert not m1[pad].any() and not v1[pad].any()
    for t in p + g + (co or []):      # the elements around the tensors
        if t.numel():
            base = t._base if t._base.dim() == 1 else t._base._base
            k = t.numel()
            assert bool((base[:offset] == 7).all()) and bool((base[offset + k:] == 7).all())


def _exact_codes(x, exp, top):
    """Neighbouring code values around x >= 0 in blocks with exponents exp."""
    table = otr.code_table(top)
    scale = np.exp2(np.repeat(exp.astype(float), 128) - 127)
    at = np.searchsorted(table, x / scale, side="right") - 1
    hi = np.minimum(at + 1, len(table) - 1)
    return table[at] * scale, np.where(x / scale == table[at], table[at], table[hi]) * scale


@pytest.mark.parametrize("offset,grad", [(0, "float32"), (1, "float32"), (0, "bfloat16")])
def test_eight_bit_states(offset, grad):
    rng = np.random.default_rng(10 + offset)
    p, g = _sets(rng, torch.float32, getattr(torch, grad), offset)
    opt = cg().AdamW(NUMEL, grad_dtype=getattr(torch, grad), state="8bit")
    state = opt.new_state()
    starts = _starts(NUMEL)
    real = np.zeros(starts[-1], dtype=bool)
    for i, k in enumerate(NUMEL):
        real[starts[i]:starts[i] + k] = True
    for step in (1, 2, 3):
        m0, v0 = (_num(t) for t in cg().cgtp_adamw_state_values(opt, state))
        codes = {k: t.cpu().numpy() for k, t in state.items()}
        assert np.array_equal(m0, otr.state_values(codes["m"], codes["m_exp"], 15, True))
        assert np.array_equal(v0, otr.state_values(codes["v"], codes["v_exp"], 31, False))
        before = [_num(t).reshape(-1) for t in p]
        cg().cgtp_adamw_step(opt, p, g, state, lr=1e-2, betas=(0.9, 0.99), eps=1e-6, weight_decay=0.1, step=step, seed=3)
        flat_g = np.zeros(starts[-1])
        flat_p = np.zeros(starts[-1])
        for i, k in enumerate(NUMEL):
            flat_g[starts[i]:starts[i] + k] = _num(g[i]).reshape(-1)
            flat_p[starts[i]:starts[i] + k] = before[i]
        q, m, v = otr.adamw(flat_p, flat_g, m0, v0, 1e-2, (0.9, 0.99), 1e-6, 0.1, step)
        u = 2.0 ** -24
        for i, k in enumerate(NUMEL):
            cut = slice(starts[i], starts[i] + k)
            lost = 4 * u * (np.abs(m0[cut]) + np.abs(flat_g[cut])) / np.maximum(np.abs(m[cut]), 1e-300)
            tol = 4 * u * np.abs(flat_p[cut]) + (16 * u + lost) * np.abs(q[cut] - flat_p[cut] * (1 - 1e-3))
            assert np.all(np.abs(_num(p[i]).reshape(-1) - q[cut]) <= tol)
        m1, v1 = (_num(t) for t in cg().cgtp_adamw_state_values(opt, state))
        exp = {k: state[k].cpu().numpy() for k in ("m_exp", "v_exp")}
        slack = 4 * u * (np.abs(m0) + np.abs(flat_g))      # m may be a difference of larger numbers
        for got, want, off, e, top in ((np.abs(m1), np.abs(m), slack, exp["m_exp"], 15), (v1, v, 6 * u * v, exp["v_exp"], 31)):
            lo, hi = _exact_codes(np.maximum(want - off, 0), e, top)[0], _exact_codes(want + off, e, top)[1]
            if top == 31:
                least = otr.code_table(top)[1] * np.exp2(np.repeat(e.astype(float), 128) - 127)
                hi = np.where(want > 0, np.maximum(hi, least), hi)
                assert np.all(v1[real & (v > 0)] > 0)
            # 1e-12: values of the grid itself
            assert np.all(got >= lo * (1 - 1e-12)) and np.all(got <= hi * (1 + 1e-12))
            assert not got[~real].any()
        sure = (m1 != 0) & (np.abs(m) > slack)
        assert np.all(m1[sure] * m[sure] > 0)


def _encode(x, top, noise, sign):
    """Codes and block exponents of FP32 values x >= 0, rounded up where 20 random bits reach the next code."""
    bits = x.view(np.uint32).astype(np.int64).reshape(-1, 128)
    exp = np.maximum((bits.max(axis=1, keepdims=True) + 0xFFFFF) >> 23, otr.E_MIN)
    base, noise = exp - top, noise.reshape(-1, 128)
    normal = ((bits + noise) >> 20) - (base << 3)
    fine = x.reshape(-1, 128) * ((256 - base) << 23).astype(np.uint32).view(np.float32)
    low = np.floor(fine + noise.astype(np.float32) * np.float32(2.0 ** -20)).astype(np.int64)
    code = np.where(bits >= (base + 1) << 23, normal, low)
    if top == 31:
        code = np.where(bits > 0, np.maximum(code, 1), code)
    return (code.reshape(-1) | sign.astype(np.int64) << 7).astype(np.uint8), exp.reshape(-1).astype(np.uint8)


def _noise(total, seed, step):
    mask, low = (1 << 64) - 1, 0xFFFFFFFF
    z = (seed + step * 0x9E3779B97F4A7C15) & mask
    z = ((z ^ (z >> 29)) * 0xBB67AE8584CAA73B) & mask
    z = ((z ^ (z >> 32)) * 0x9E3779B97F4A7C15) & mask
    z ^= z >> 29
    x = (np.arange(total, dtype=np.uint64) * np.uint64(0x9E3779B1) + np.uint64(z & low)) & np.uint64(low)
    x = ((x ^ (x >> np.uint64(15))) * np.uint64(0xBB67AE85)) & np.uint64(low)
    x = ((x ^ (x >> np.uint64(13))) * np.uint64(0x3C6EF373) + np.uint64(z >> 32)) & np.uint64(low)
    return (x ^ (x >> np.uint64(16))).astype(np.int64)


@pytest.mark.parametrize("offset,grad", [(0, "float32"), (1, "float32"), (0, "bfloat16")])
def test_eight_bit_codes_are_a_function_of_the_fp32_arithmetic(offset, grad):
    # every product and sum of m and v is rounded once, so the codes can be had from FP32 arithmetic on the CPU, bit for bit
    rng = np.random.default_rng(20)
    shapes = SHAPES + [(300, 1024)]
    numel = [int(np.prod(s)) for s in shapes]
    p, g = _sets(rng, torch.float32, getattr(torch, grad), offset, shapes)
    starts, f = _starts(numel), np.float32
    flat = np.zeros(starts[-1], dtype=f)
    for i, k in enumerate(numel):
        flat[starts[i]:starts[i] + k] = g[i].float().cpu().numpy().reshape(-1)
    opt = cg().AdamW(numel, grad_dtype=getattr(torch, grad), state="8bit")
    state = opt.new_state()
    for step in (1, 2, 3):
        m, v = (t.cpu().numpy() for t in cg().cgtp_adamw_state_values(opt, state))
        cg().cgtp_adamw_step(opt, p, g, state, lr=1e-2, step=step, seed=77)
        m = m * f(0.9) + flat * f(1 - 0.9)
        v = v * f(0.999) + (flat * flat) * f(1 - 0.999)
        r = _noise(starts[-1], 77, step)
        got = {k: t.cpu().numpy() for k, t in state.items()}
        for name, x, top, noise, sign in (("m", np.abs(m), 15, (r >> 16) << 4, np.signbit(m)), ("v", v, 31, (r & 0xFFFF) << 4, np.zeros(m.shape, bool))):
            code, exp = _encode(x, top, noise, sign)
            assert np.array_equal(got[name], code) and np.array_equal(got[name + "_exp"], exp), (name, step)


def test_eight_bit_rounding_is_unbiased_and_a_function_of_seed_and_step():
    # v = 1 with beta2 = 0.999 and a zero gradient: 0.1% a step, far below the grid's 12.5%
    k = 1 << 16
    opt = cg().AdamW([k], state="8bit")
    p, g = [torch.zeros(k, device="cuda")], [torch.zeros(k, device="cuda")]

    def run(seed, steps=100):
        state = opt.new_state()
        state["v"].fill_(8 * 31)
        state["v_exp"].fill_(127)
        for t in range(steps):
            cg().cgtp_adamw_step(opt, p, g, state, lr=0.0, step=t + 1, seed=seed)
        return state

    a, b, c = run(1), run(1), run(2)
    assert torch.equal(a["v"], b["v"]) and not torch.equal(a["v"], c["v"])
    v = _num(cg().cgtp_adamw_state_values(opt, a)[1])
    # mean 0.999^100 = 0.9048; the spread of one element is below sqrt(100 x 0.001 x 0.125) = 0.11
    assert abs(v.mean() - 0.999 ** 100) < 5 * 0.11 / np.sqrt(k)
    # neighbours are independent: correlation of 65,536 pairs within 5 standard deviations
    d = v - v.mean()
    for lag in (1, 2, 4, 32, 128):
        assert abs((d[lag:] * d[:-lag]).mean() / (d * d).mean()) < 5 / np.sqrt(k)


def test_values_on_the_grid_stay():
    # beta1 = 0 and beta2 = 0 store g and g^2: powers of two are codes, whatever the noise
    g = torch.exp2(torch.arange(128, device="cuda").remainder(7).float() - 3)
    opt = cg().AdamW([128], state="8bit")
    state = opt.new_state()
    cg().cgtp_adamw_step(opt, [torch.zeros(128, device="cuda")], [g], state, lr=1e-3, betas=(0.0, 0.0), step=1, seed=9)
    m, v = cg().cgtp_adamw_state_values(opt, state)
    assert torch.equal(m, g) and torch.equal(v, g * g)


@pytest.mark.parametrize("state_kind", ["f32", "8bit"])
def test_missing_gradients_and_non_finite_norms_change_nothing(state_kind):
    rng = np.random.default_rng(2)
    p, g = _sets(rng, torch.float32, torch.float32, 0)
    opt = cg().AdamW(NUMEL, state=state_kind)
    state = opt.new_state()
    cg().cgtp_adamw_step(opt, p, g, state, lr=1e-2, step=1)
    keep = [t.clone() for t in p], {k: None if t is None else t.clone() for k, t in state.items()}
    some = [None if i % 2 else t for i, t in enumerate(g)]
    clip = cg().cgtp_grad_norm(opt, some)
    want, _ = otr.grad_norm([_num(t) for t in g[::2]], 1.0)
    assert abs(float(clip[0]) - want) <= 64 * 2.0 ** -24 * want and float(clip[1]) == 1.0
    cg().cgtp_adamw_step(opt, p, some, state, lr=1e-2, step=2, clip=clip)
    starts = _starts(NUMEL)
    for i, k in enumerate(NUMEL):
        same = torch.equal(p[i], keep[0][i]) and torch.equal(state["m"][starts[i]:starts[i + 1]], keep[1]["m"][starts[i]:starts[i + 1]])
        assert same == (i % 2 == 1 or k == 0)
    for bad in (float("nan"), float("inf")):
        keep = [t.clone() for t in p], {k: None if t is None else t.clone() for k, t in state.items()}
        broken = [t.clone() for t in g]
        broken[1].view(-1)[5] = bad
        clip = cg().cgtp_grad_norm(opt, broken, 1.0)
        assert not np.isfinite(float(clip[0])) and np.isnan(float(clip[1]))
        cg().cgtp_adamw_step(opt, p, broken, state, lr=1e-2, step=3, clip=clip)
        assert all(torch.equal(a, b) for a, b in zip(p, keep[0]))
        assert all(a is None or torch.equal(a, keep[1][k]) for k, a in state.items())


def test_a_nan_gradient_without_clipping_stays_in_its_place():
    opt8, opt = cg().AdamW([300], state="8bit"), cg().AdamW([300])
    g = torch.ones(300, device="cuda")
    g[130] = float("nan")
    for o, last in ((opt, 131), (opt8, 256)):
        state, p = o.new_state(), [torch.zeros(300, device="cuda")]
        cg().cgtp_adamw_step(o, p, [g], state, lr=1e-2, step=1)
        m, v = cg().cgtp_adamw_state_values(o, state)
        assert int(torch.isnan(p[0]).sum()) == 1
        bad = torch.isnan(m).nonzero().view(-1)       # FP32 states: one element; 8-bit states: its block
        assert int(bad[0]) == (130 if o is opt else 128) and int(bad[-1]) == last - 1 and bool(torch.isnan(v[130]))


def test_states_of_extreme_size():
    g = torch.tensor([3e38, 1e-38, 1e-45, 0.0, -3e38, 1e19, 1e-20, -0.0] * 16, device="cuda")
    opt = cg().AdamW([128], state="8bit")
    state, p = opt.new_state(), [torch.ones(128, device="cuda")]
    cg().cgtp_adamw_step(opt, p, [g * 0.0], state, lr=1e-3, step=1)
    assert torch.equal(p[0], torch.ones(128, device="cuda")) and not state["m"].any() and not state["v"].any()
    small = torch.tensor([1e-38, 1e-30, 1e-20, -1e-25] * 32, device="cuda")
    cg().cgtp_adamw_step(opt, p, [small], state, lr=1e-3, step=1)
    m, v = cg().cgtp_adamw_state_values(opt, state)
    assert bool(torch.isfinite(m).all()) and bool(torch.isfinite(v).all()) and bool(torch.isfinite(p[0]).all())
    assert bool((v[2::4] > 0).all())


@pytest.mark.parametrize("eps", [0.0, 1e-15, 1e-12, 1e-8])
@pytest.mark.parametrize("state_kind", ["f32", "8bit"])
def test_small_eps_and_small_gradients(eps, state_kind):
    # from zero states the step is lr |g| / (|g| + eps).  FP32 keeps (1 - beta2) g^2 of g = 1e-18 as 1e-39, a
    # denormal with 19 bits: 2^-19 of v, plus the bounds above; 1e-19: 13 bits
    for size, bits in ((1.0, 20), (1e-6, 20), (1e-18, 18), (1e-19, 12)):
        g = [torch.full((200,), size, device="cuda")]
        p = [torch.zeros(200, device="cuda")]
        opt = cg().AdamW([200], state=state_kind)
        cg().cgtp_adamw_step(opt, p, g, opt.new_state(), lr=1e-2, eps=eps, step=1)
        want = 1e-2 * size / (size + eps)
        assert float((p[0] + want).abs().max()) <= 2.0 ** -bits * want, (size, float(p[0][0]), want)


def test_other_streams():
    g, p = [torch.randn(5000, device="cuda")], [torch.randn(5000, device="cuda")]
    opt = cg().AdamW([5000], state="8bit")
    runs = []
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    for stream in (None, s):
        q, state = [p[0].clone()], opt.new_state()
        torch.cuda.synchronize()
        clip = cg().cgtp_grad_norm(opt, g, 1.0, stream=stream)
        cg().cgtp_adamw_step(opt, q, g, state, lr=1e-2, clip=clip, stream=stream)
        m, v = cg().cgtp_adamw_state_values(opt, state, stream=stream)
        torch.cuda.synchronize()
        runs.append((clip, q[0], m, v))
    assert all(torch.equal(a, b) for a, b in zip(*runs))


def test_more_tensors_than_one_launch_holds():
    for count in (64, 65, 1024, 1025, 2100):
        rng = np.random.default_rng(count)
        numel = [int(v) for v in rng.integers(0, 300, size=count)]
        starts = _starts(numel)
        p = [torch.from_numpy(rng.standard_normal(k)).float().cuda() for k in numel]
        g = [torch.from_numpy(rng.standard_normal(k)).float().cuda() for k in numel]
        before = [_num(t) for t in p]
        opt = cg().AdamW(numel)
        state = opt.new_state()
        clip = cg().cgtp_grad_norm(opt, g, 1.0)
        n, coef = otr.grad_norm([_num(t) for t in g], 1.0)
        assert abs(float(clip[0]) - n) <= 64 * 2.0 ** -24 * n
        cg().cgtp_adamw_step(opt, p, g, state, lr=1e-2, step=1, clip=clip)
        m = _num(state["m"])
        for i, k in enumerate(numel):
            want = otr.adamw(before[i], _num(g[i]), np.zeros(k), np.zeros(k), 1e-2, (0.9, 0.999), 1e-8, 0.0, 1, coef)
            # from zero states: the step is lr g / (|g| + eps), 16 u of 1e-2 and 4 u of p
            assert np.all(np.abs(_num(p[i]) - want[0]) <= 2.0 ** -24 * (4 * np.abs(before[i]) + 0.32))
            assert np.all(np.abs(m[starts[i]:starts[i] + k] - want[1]) <= 70 * 2.0 ** -24 * np.abs(want[1]))


def test_norm_is_repeatable_and_exact_enough():
    rng = np.random.default_rng(8)
    numel = [3_000_001, 5, 700_000]
    for dt in (torch.float32, torch.bfloat16):
        g = [torch.from_numpy(rng.standard_normal(k)).to(dt).cuda() for k in numel]
        opt = cg().AdamW(numel, grad_dtype=dt)
        a, b = cg().cgtp_grad_norm(opt, g, 10.0), cg().cgtp_grad_norm(opt, g, 10.0)
        n, coef = otr.grad_norm([_num(t) for t in g], 10.0)
        assert torch.equal(a, b) and abs(float(a[0]) - n) <= 64 * 2.0 ** -24 * n and abs(float(a[1]) - coef) <= 66 * 2.0 ** -24 * coef
    zero = cg().cgtp_grad_norm(opt, [torch.zeros_like(t) for t in g], 10.0)
    assert float(zero[0]) == 0.0 and float(zero[1]) == 1.0


def test_refusals():
    m = cg()
    opt = m.AdamW([4, 6], state="8bit")
    state = opt.new_state()
    p = [torch.zeros(4, device="cuda"), torch.zeros(2, 3, device="cuda")]
    bad = [
        (ValueError, lambda: m.cgtp_adamw_step(opt, p[:1], p[:1], state, lr=1e-3)),
        (ValueError, lambda: m.cgtp_adamw_step(opt, [p[0], p[1].t()], p, state, lr=1e-3)),
        (TypeError, lambda: m.cgtp_adamw_step(opt, [t.double() for t in p], p, state, lr=1e-3)),
        (TypeError, lambda: m.cgtp_adamw_step(opt, p, [t.cpu() for t in p], state, lr=1e-3)),
        (ValueError, lambda: m.cgtp_adamw_step(opt, p, p, dict(state, v=state["v"][:128]), lr=1e-3)),
        (m.CgtpError, lambda: m.cgtp_adamw_step(opt, p, p, state, lr=1e-3, step=0)),
        (m.CgtpError, lambda: m.cgtp_adamw_step(opt, p, p, state, lr=1e-3, betas=(1.0, 0.9))),
        (m.CgtpError, lambda: m.cgtp_adamw_step(opt, p, p, state, lr=float("nan"))),
        (m.CgtpError, lambda: m.cgtp_adamw_step(opt, p, p, state, lr=1e-3, eps=-1.0)),
        (m.CgtpError, lambda: m.cgtp_adamw_step(opt, [None, p[1]], p, state, lr=1e-3)),
        (m.CgtpError, lambda: m.cgtp_grad_norm(opt, p, 0.0)),
        (m.CgtpError, lambda: m.AdamW([])),
        (m.CgtpError, lambda: m.AdamW([-1])),
        (m.CgtpError, lambda: m.AdamW([4], param_dtype=torch.float64, state="8bit")),
        (TypeError, lambda: m.AdamW([4], param_dtype=torch.bfloat16)),
        (m.CgtpError, lambda: m.AdamW([4], grad_dtype=torch.float64)),
    ]
    for kind, call in bad:
        with pytest.raises(kind):
            call()
    assert not state["m"].any() and not p[0].any()
