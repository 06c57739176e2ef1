"""Cases of the operators that surround a convolution in a training step: the gated residual
norm (forward and backward) and the AdamW step over many tensors (32-bit and 8-bit states,
with the global gradient norm in front of it).

Irreps rows are multiplicity-major: block i of "MULxLP" holds MUL channels of 2L+1 components.
"""

import math

import torch

own = False

DEV = "cuda"
BLOCK = 128                    # elements of one 8-bit state block
E_MIN = 40                     # smallest block exponent (biased) of the 8-bit states
M_TOP, V_TOP = 15, 31          # largest exponent field of the m and v codes
LR, BETAS, EPS, DECAY = 1e-3, (0.9, 0.999), 1e-8, 0.01
NORM_EPS = 1e-5


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def listed():
    norm = dict(act="sigmoid", pre=True, post=True, skip=True, dtype="f32", slices=False)
    opt = dict(op="adamw", state="f32", grad="f32", copies=False, clip="none", step=10)
    return [
        # the smallest graphs (molecules): one launch, nothing but latency
        dict(norm, name="fwd tiny", op="fwd", irreps="8x0e+8x1o", n=64),
        # one block of the NequIP-like workload
        dict(norm, name="fwd nequip", op="fwd", irreps="32x0e+32x1o+32x2e+32x3o", n=10000),
        # the norm in front of the first block, odd multiplicities and an odd number of nodes
        dict(norm, name="fwd first odd", op="fwd", irreps="33x0e+17x1o+5x2e", n=49999, act="none", post=False, skip=False),
        # the large radial workload in bfloat16: y feeds a bfloat16 product, gates and features
        # are column ranges of the product's output rows
        dict(norm, name="fwd uvw bf16", op="fwd", irreps="64x0e+64x1o+64x2e", n=200000, dtype="bf16", act="silu", slices=True),
        # the backward of a small batch
        dict(norm, name="bwd tiny", op="bwd", irreps="8x0e+8x1o", n=64),
        # one block of the MACE-like workload, wide rows
        dict(norm, name="bwd mace", op="bwd", irreps="128x0e+128x1o+128x2e", n=5000, act="silu", slices=True),
        # the large radial workload
        dict(norm, name="bwd uvw", op="bwd", irreps="64x0e+64x1o+64x2e", n=200000),
        # parameters of a small model: radial networks and gains, clipped
        dict(opt, name="adamw small", sizes="8x64,64x64,64x1088,128,128,128", layers=5, clip="active"),
        # a large model, bfloat16 gradients and copies of the weights
        dict(opt, name="adamw large", sizes="1536x1024,1024x1536,1024,1024,33", layers=32, grad="bf16", copies=True),
        # 8-bit states: a small model with clipping switched on but idle, as in most steps
        dict(opt, name="adamw8 small", sizes="8x64,64x64,64x1088,128,128,128", layers=5, state="8bit", clip="idle"),
        # 8-bit states: weights of the radial workload's layers, odd vectors among them
        dict(opt, name="adamw8 uvw", sizes="8x45056,64x64,64x64,64x64,192,191,7", layers=24, state="8bit"),
        # 8-bit states of a large model
        dict(opt, name="adamw8 large", sizes="1536x1024,1024x1536,1024,1024,33", layers=32, state="8bit", clip="idle"),
    ]


def draw(rng):
    if rng.random() < 0.55:
        parity = "eo"
        lmax = rng.choice([0, 1, 2, 2, 3, 3, 7])
        ls = sorted(rng.sample(range(lmax + 1), rng.randint(1, min(lmax + 1, 4))))
        top = 128 if lmax <= 3 else 24
        if rng.random() < 0.6:
            muls = [rng.choice([m for m in (4, 8, 16, 32, 64, 128) if m <= max(top, 4)])] * len(ls)
        else:
            muls = [int(round(math.exp(rng.uniform(0, math.log(top))))) for _ in ls]
        irreps = "+".join("%dx%d%s" % (m, l, parity[l % 2]) for m, l in zip(muls, ls))
        dim = sum(m * (2 * l + 1) for m, l in zip(muls, ls))
        most = min(400000, 200000 * 576 // dim)
        n = int(round(math.exp(rng.uniform(math.log(16), math.log(most)))))
        post, skip = rng.random() < 0.8, rng.random() < 0.8
        return dict(op=rng.choice(["fwd", "bwd"]), irreps=irreps, n=n, dtype=rng.choice(["f32", "f32", "bf16", "bf16all"]),
                    act=rng.choice(["none", "identity", "sigmoid", "silu"]), pre=rng.random() < 0.8 or not (post or skip),
                    post=post, skip=skip, slices=rng.random() < 0.4)
    sizes = []
    for _ in range(rng.randint(1, 9)):
        rows = int(round(math.exp(rng.uniform(0, math.log(1500)))))
        sizes.append(rng.choice(["%d" % rows, "%dx%d" % (rows, rng.choice([1, 8, 64, 128, 353, 1024]))]))
    per = sum(math.prod(map(int, s.split("x"))) for s in sizes)
    layers = max(1, min(int(round(math.exp(rng.uniform(0, math.log(64))))), 100000000 // per))
    state = rng.choice(["f32", "8bit"])
    return dict(op="adamw", state=state, grad=rng.choice(["f32", "bf16"]), copies=rng.random() < 0.5, sizes=",".join(sizes),
                layers=layers, clip=rng.choice(["none", "idle", "active"] if state == "f32" else ["none", "idle"]),
                step=rng.randint(1, 5000))


def _blocks(irreps):
    """[(multiplicity, components)] of an irreps string."""
    return [(int(t.split("x")[0]), 2 * int(t.split("x")[1][:-1]) + 1) for t in irreps.split("+")]


def _types(case):
    """Element types of the residual stream, of what comes from the product and of what goes to it."""
    f, b = torch.float32, torch.bfloat16
    return {"f32": (f, f, f), "bf16": (f, f, b), "bf16all": (b, b, b)}[case["dtype"]]


def _shapes(case):
    """Shapes of the parameter tensors."""
    return [tuple(map(int, s.split("x"))) for s in case["sizes"].split(",")] * case["layers"]


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    return _prepare_adamw(case, gen, seed) if case["op"] == "adamw" else _prepare_norm(case, gen)


def _prepare_norm(case, gen):
    blocks, n = _blocks(case["irreps"]), case["n"]
    dim, chan = sum(m * d for m, d in blocks), sum(m for m, _ in blocks)
    stream, come, go = _types(case)
    s = dict(case=case, blocks=blocks, dim=dim, chan=chan)

    def rows(width, dtype, scale):
        # node features differ in size from node to node
        x = torch.randn(n, width, device=DEV, generator=gen)
        return (x * torch.exp(0.5 * torch.randn(n, 1, device=DEV, generator=gen)) * scale).to(dtype)

    def gain(mean, spread):
        return mean + spread * torch.randn(chan, device=DEV, generator=gen)

    gated, has_z = case["act"] != "none", case["post"] or case["skip"]
    s["h"] = rows(dim, stream, 1.0) if case["skip"] or not has_z else None
    s["z"] = s["q"] = s["post"] = s["scale"] = s["pre"] = None
    if has_z:
        wide = rows((chan if gated else 0) + dim, come, 0.7)
        wide[::41] = 0                                    # nodes without neighbours
        z, q = wide[:, -dim:], wide[:, :chan] if gated else None
        # a program that keeps gates and features in one product output passes column ranges of it
        s["z"], s["q"] = (z, q) if case["slices"] else (z.contiguous(), q.contiguous() if gated else None)
        s["scale"] = gain(0.2, 0.05)
        s["post"] = gain(1.0, 0.2) if case["post"] else None
    if case["pre"]:
        s["pre"] = gain(1.0, 0.2)
    if case["op"] == "bwd":
        s["gout"] = rows(dim, stream, 1.0)
        s["gy"] = rows(dim, come, 1.0) if case["pre"] else None
        s["x"] = _plain_forward(s)[0] if has_z else s["h"]   # what the forward left
    if own:
        import clebsch_gordan_tensor_racah_gb300 as cg
        s["plan"] = cg.ResNormPlan(case["irreps"], dtype=torch.float32 if case["dtype"] == "f32" else torch.bfloat16,
                                   storage=case["dtype"] == "bf16all", act=case["act"], pre_norm=case["pre"],
                                   post_norm=case["post"], alpha=1.0, eps=NORM_EPS)
    return s


def _prepare_adamw(case, gen, seed):
    shapes = _shapes(case)
    numel = [math.prod(x) for x in shapes]
    padded = [-(-k // BLOCK) * BLOCK for k in numel]
    starts = [0]
    for k in padded:
        starts.append(starts[-1] + k)
    total = starts[-1]
    spans = torch.tensor(numel, device=DEV)
    of = torch.repeat_interleave(torch.arange(len(shapes), device=DEV), torch.tensor(padded, device=DEV), output_size=total)
    place = torch.arange(total, device=DEV) - torch.tensor(starts[:-1], device=DEV)[of]
    real = place < spans[of]
    # gradients differ in size from tensor to tensor and from element to element
    size = torch.exp(torch.randn(len(shapes), device=DEV, generator=gen) - 6)[of]
    draws = lambda: torch.randn(total, device=DEV, generator=gen) * real  # noqa: E731
    g = draws() * size * torch.exp(1.5 * torch.randn(total, device=DEV, generator=gen))
    p = 0.05 * draws()
    m = (0.3 * g + 0.1 * size * draws())
    v = g * g * (0.2 + torch.rand(total, device=DEV, generator=gen)) + 0.01 * (size * draws()) ** 2
    g = g.to(torch.float32 if case["grad"] == "f32" else torch.bfloat16)
    # gains and biases are not decayed
    scale = [1.0 if len(x) > 1 else 0.0 for x in shapes]
    s = dict(case=case, p=p, g=g, decay=torch.tensor(scale, device=DEV)[of], seed=seed * 7919 + 11,
             copy=p.to(torch.bfloat16) if case["copies"] else None)
    if case["state"] == "8bit":
        m8, me = _encode(m.abs().view(-1, BLOCK), M_TOP, 1 << 19)
        s["m"] = (m8 | ((m.view(-1, BLOCK) < 0).to(torch.int32) << 7)).to(torch.uint8).view(-1)
        v8, ve = _encode(v.view(-1, BLOCK), V_TOP, 1 << 19)
        s["v"] = torch.where(v.view(-1, BLOCK) > 0, v8.clamp(min=1), v8).to(torch.uint8).view(-1)
        s["m_exp"], s["v_exp"] = me.to(torch.uint8), ve.to(torch.uint8)
    else:
        s["m"], s["v"], s["m_exp"], s["v_exp"] = m, v, None, None
    norm = float(g.double().square().sum().sqrt())
    s["max_norm"] = {"none": None, "idle": 4.0 * norm, "active": 0.3 * norm}[case["clip"]]
    if own:
        import clebsch_gordan_tensor_racah_gb300 as cg
        cut = lambda t: None if t is None else [t[a:a + k].view(x) for a, k, x in zip(starts, numel, shapes)]  # noqa: E731
        s["opt"] = cg.AdamW(numel, grad_dtype=g.dtype, state=case["state"], decay_scale=scale)
        s["params"], s["grads"], s["copies"] = cut(p), cut(g), cut(s["copy"])
        s["state"] = dict(m=s["m"], v=s["v"], m_exp=s["m_exp"], v_exp=s["v_exp"])
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def run(s):
    op = s["case"]["op"]
    if op == "adamw":
        return _own_adamw(s) if own else _plain_adamw(s)
    if own:
        import clebsch_gordan_tensor_racah_gb300 as cg
        if op == "fwd":
            out, y = cg.cgtp_resnorm_forward(s["plan"], s["h"], s["z"], s["q"], post=s["post"], scale=s["scale"], pre=s["pre"])
        else:
            return _named_grads(cg.cgtp_resnorm_backward(s["plan"], s["gout"], s["gy"], s["x"], s["z"], s["q"], post=s["post"],
                                                         scale=s["scale"], pre=s["pre"], need_gh=s["h"] is not None))
    elif op == "fwd":
        out, y = _plain_forward(s)
    else:
        return _named_grads(_plain_backward(s))
    return dict(out=out if s["z"] is not None else None, y=y)


def _named_grads(g):
    return dict(zip(("gh", "gz", "gq", "gpost", "gscale", "gpre"), g))


def _own_adamw(s):
    import clebsch_gordan_tensor_racah_gb300 as cg
    clip = None
    if s["max_norm"] is not None:
        clip = cg.cgtp_grad_norm(s["opt"], s["grads"], s["max_norm"])
    cg.cgtp_adamw_step(s["opt"], s["params"], s["grads"], s["state"], lr=LR, betas=BETAS, eps=EPS, weight_decay=DECAY,
                       step=s["case"]["step"], copies=s["copies"], clip=clip, seed=s["seed"])
    m, v = s["m"], s["v"]
    if s["m_exp"] is not None:
        m, v = cg.cgtp_adamw_state_values(s["opt"], s["state"])
    return dict(p=s["p"], m=m, v=v, copy=s["copy"], norm=clip)


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------

def _split(x, blocks):
    """Views [n, multiplicity, components] of the irreps blocks of rows."""
    parts = torch.split(x.float(), [m * d for m, d in blocks], dim=1)
    return [p.unflatten(1, b) for p, b in zip(parts, blocks)]


def _join(parts):
    return torch.cat([p.flatten(1) for p in parts], dim=1)


def _rms(x):
    return 1.0 / torch.sqrt((x * x).mean(dim=(1, 2), keepdim=True) + NORM_EPS)


def _gate(s, derivative=False):
    """a(q) per channel, and its derivative."""
    act = s["case"]["act"]
    if act == "none":
        return None
    q = s["q"].float()
    sig = 1.0 / (1.0 + torch.exp(-q))
    if derivative:
        return {"identity": torch.ones_like(q), "sigmoid": sig * (1.0 - sig), "silu": sig * (1.0 + q * (1.0 - sig))}[act]
    return {"identity": q, "sigmoid": sig, "silu": q * sig}[act]


def _per_channel(x, blocks):
    """Per-channel factors [1 or n, channels] as [.., multiplicity, 1] of each block."""
    x = x if x.dim() == 2 else x[None]
    return [p[:, :, None] for p in torch.split(x, [m for m, _ in blocks], dim=1)]


def _plain_forward(s):
    stream, _, go = _types(s["case"])
    blocks = s["blocks"]
    out, wide = s["h"], None
    if s["z"] is not None:
        z = _split(s["z"], blocks)
        if s["case"]["post"]:
            z = [x * _rms(x) for x in z]
        w = s["scale"] if s["post"] is None else s["scale"] * s["post"]
        gate = _gate(s)
        w = w if gate is None else w * gate
        wide = _join([x * c for x, c in zip(z, _per_channel(w, blocks))])
        wide = wide if s["h"] is None else wide + s["h"].float()
        out = wide.to(stream)
    if not s["case"]["pre"]:
        return out, None
    # the norm sees the rounded stream, as the next block's backward does
    y = [x * _rms(x) * c for x, c in zip(_split(out, blocks), _per_channel(s["pre"], blocks))]
    return out, _join(y).to(go)


def _plain_backward(s):
    stream, _, go = _types(s["case"])
    blocks, case = s["blocks"], s["case"]
    gh = gz = gq = gpost = gscale = gpre = None
    d = _split(s["gout"], blocks)
    if case["pre"]:
        x, gy = _split(s["x"], blocks), _split(s["gy"], blocks)
        r = [_rms(a) for a in x]
        wy = [g * c for g, c in zip(gy, _per_channel(s["pre"], blocks))]
        d = [g + w * p - a * p * p * p * (w * a).mean(dim=(1, 2), keepdim=True) for g, w, a, p in zip(d, wy, x, r)]
        gpre = torch.cat([(g * a * p).sum(dim=(0, 2)) for g, a, p in zip(gy, x, r)])
    if s["h"] is not None:
        gh = _join(d).to(stream)
    if s["z"] is not None:
        z = _split(s["z"], blocks)
        r = [_rms(a) if case["post"] else 1.0 for a in z]
        z = [a * p for a, p in zip(z, r)]
        base = s["scale"] if s["post"] is None else s["scale"] * s["post"]
        gate = _gate(s)
        w = _per_channel(base if gate is None else base * gate, blocks)
        wd = [a * c for a, c in zip(d, w)]
        if case["post"]:
            gz = [p * (a - b * (a * b).mean(dim=(1, 2), keepdim=True)) for a, b, p in zip(wd, z, r)]
        else:
            gz = wd
        gz = _join(gz).to(go)
        along = torch.cat([(a * b).sum(dim=2) for a, b in zip(d, z)], dim=1)
        if gate is not None:
            gq = (along * base * _gate(s, derivative=True)).to(go)
            along = along * gate
        total = along.sum(dim=0)
        gscale = total if s["post"] is None else total * s["post"]
        gpost = None if s["post"] is None else total * s["scale"]
    return gh, gz, gq, gpost, gscale, gpre


def _encode(x, top, noise):
    """8-bit codes (int32) of non-negative blocks [k, BLOCK] and the blocks' exponents: top + 1 binades of
    8 steps under a power of two, then a linear range to zero; `noise` (20 bits) rounds stochastically."""
    bits = x.contiguous().view(torch.int32)
    exp = ((bits.amax(dim=1, keepdim=True) + 0xFFFFF) >> 23).clamp(min=E_MIN)
    base = exp - top
    fine = x * ((256 - base) << 23).view(torch.float32)
    small = torch.floor(fine + noise * 2.0 ** -20).to(torch.int32)
    code = torch.where(bits >= ((base + 1) << 23), ((bits + noise) >> 20) - (base << 3), small)
    return code, exp.view(-1)


def _decode(code, exp, top):
    """Values of the codes of _encode."""
    code, base = code.view(-1, BLOCK).to(torch.int32), exp.to(torch.int32).clamp(min=E_MIN)[:, None] - top
    low = code * ((base - 129 + 127) << 23).view(torch.float32)
    return torch.where(code >= 8, ((base << 23) + (code << 20)).view(torch.float32), low)


def _noise(total, seed, step):
    """32 pseudo-random bits for every state element, a function of (element, seed, step)."""
    mask = (1 << 64) - 1
    z = (seed + step * 0x9E3779B97F4A7C15) & mask
    z = ((z ^ (z >> 29)) * 0xBB67AE8584CAA73B) & mask
    z = ((z ^ (z >> 32)) * 0x9E3779B97F4A7C15) & mask
    z ^= z >> 29
    i = torch.arange(total, device=DEV)
    low = 0xFFFFFFFF
    x = ((i & low) * 0x9E3779B1 + (i >> 32) * 0x85A308D3 + (z & low)) & low
    x = ((x ^ (x >> 15)) * 0xBB67AE85) & low
    x = ((x ^ (x >> 13)) * 0x3C6EF373 + (z >> 32)) & low
    return x ^ (x >> 16)


def _plain_adamw(s):
    case = s["case"]
    g, norm = s["g"].float(), None
    if s["max_norm"] is not None:
        n = torch.sqrt((g * g).sum())
        coef = torch.where(n > s["max_norm"], s["max_norm"] / n, 1.0)
        norm = torch.stack([n, coef])
        g = g * coef
    b1, b2 = BETAS
    bits8 = s["m_exp"] is not None
    m, v = s["m"], s["v"]
    if bits8:
        sign = 1.0 - 2.0 * (m >> 7).to(torch.float32)
        m = _decode(m & 127, s["m_exp"], M_TOP).view(-1) * sign
        v = _decode(v, s["v_exp"], V_TOP).view(-1)
    m = m * b1 + g * (1.0 - b1)
    v = v * b2 + (g * g) * (1.0 - b2)
    t = case["step"]
    rate, root = LR / (1.0 - b1 ** t), 1.0 / math.sqrt(1.0 - b2 ** t)
    p = s["p"] * (1.0 - LR * DECAY * s["decay"]) - rate * m / (torch.sqrt(v) * root + EPS)
    s["p"].copy_(p)
    if s["copy"] is not None:
        s["copy"].copy_(p)
    if not bits8:
        s["m"].copy_(m)
        s["v"].copy_(v)
        return dict(p=s["p"], m=s["m"], v=s["v"], copy=s["copy"], norm=norm)
    noise = _noise(m.numel(), s["seed"], t).view(-1, BLOCK)
    m, v = m.view(-1, BLOCK), v.view(-1, BLOCK)
    mc, me = _encode(m.abs(), M_TOP, ((noise >> 16) << 4).to(torch.int32))
    vc, ve = _encode(v, V_TOP, ((noise & 0xFFFF) << 4).to(torch.int32))
    vc = torch.where(v > 0, vc.clamp(min=1), vc)
    values = _decode(mc, me, M_TOP) * torch.where(m < 0, -1.0, 1.0), _decode(vc, ve, V_TOP)
    s["m"].copy_((mc | ((m < 0).to(torch.int32) << 7)).view(-1))
    s["v"].copy_(vc.view(-1))
    s["m_exp"].copy_(me)
    s["v_exp"].copy_(ve)
    return dict(p=s["p"], m=values[0].view(-1), v=values[1].view(-1), copy=s["copy"], norm=norm)


# ---------------------------------------------------------------------------
# work and exact values
# ---------------------------------------------------------------------------

def work(case):
    if case["op"] == "adamw":
        total = sum(math.prod(x) for x in _shapes(case))
        g = 4 if case["grad"] == "f32" else 2
        each = 8 + g + 16 if case["state"] == "f32" else 8 + g + 4 + 8   # 8 bits: the values of m and v come back too
        each += 2 if case["copies"] else 0
        return dict(bytes=each * total, flops=(14 if case["state"] == "f32" else 30) * total)
    blocks, n = _blocks(case["irreps"]), case["n"]
    dim, chan = sum(m * d for m, d in blocks), sum(m for m, _ in blocks)
    a, b, c = (t.itemsize for t in _types(case))
    gated, has_z = case["act"] != "none", case["post"] or case["skip"]
    has_h = case["skip"] or not has_z
    if case["op"] == "fwd":
        wide = a * (has_h + has_z) + b * has_z + c * case["pre"]
        return dict(bytes=n * (dim * wide + (chan * b if gated and has_z else 0)), flops=8 * n * dim)
    wide = a * (1 + has_h + case["pre"]) + b * (case["pre"] + has_z) + c * has_z
    return dict(bytes=n * (dim * wide + (chan * (b + c) if gated and has_z else 0)), flops=20 * n * dim)


def exact(case, seed):
    """The definition in 64 bits: gradients by differentiating the formula, updates element by element."""
    s = prepare(case, seed)
    wide = lambda t: None if t is None else t.double()  # noqa: E731
    if case["op"] == "adamw":
        return _exact_adamw(s, case)
    leaves = {k: wide(s[k]) for k in ("h", "z", "q", "post", "scale", "pre")}
    stream = torch.float64
    if case["op"] == "fwd":
        out, y = _exact_forward(case, s["blocks"], leaves)
        if y is not None and case["dtype"] == "bf16all" and leaves["z"] is not None:
            # y is the norm of the stream as it is stored
            y = _exact_norm(out.to(torch.bfloat16).to(stream), s["blocks"], leaves["pre"])
        return dict(out=out if s["z"] is not None else None, y=y)
    g = {}
    d = wide(s["gout"])
    if case["pre"]:
        x, pre = wide(s["x"]).requires_grad_(), leaves["pre"].clone().requires_grad_()
        y = _exact_norm(x, s["blocks"], pre)
        dx, g["gpre"] = torch.autograd.grad(y, (x, pre), wide(s["gy"]))
        d = d + dx
    g["gh"] = d if s["h"] is not None else None
    if s["z"] is not None:
        names = [k for k in ("z", "q", "post", "scale") if leaves[k] is not None]
        for k in names:
            leaves[k] = leaves[k].clone().requires_grad_()
        got = torch.autograd.grad(_exact_forward(dict(case, pre=False), s["blocks"], leaves)[0], [leaves[k] for k in names], d)
        g.update({"g" + k: v for k, v in zip(names, got)})
    return {k: g.get(k) for k in ("gh", "gz", "gq", "gpost", "gscale", "gpre")}


def _exact_norm(x, blocks, gain):
    parts, at, c = [], 0, 0
    for mul, d in blocks:
        b = x[:, at:at + mul * d].reshape(-1, mul, d)
        power = torch.einsum("num,num->n", b, b) / (mul * d)
        b = b * (power + NORM_EPS).rsqrt()[:, None, None]
        parts.append((b if gain is None else b * gain[c:c + mul, None]).reshape(-1, mul * d))
        at, c = at + mul * d, c + mul
    return torch.cat(parts, 1)


def _exact_forward(case, blocks, t):
    out = t["h"]
    if t["z"] is not None:
        v = _exact_norm(t["z"], blocks, None) if case["post"] else t["z"]
        w = t["scale"] if t["post"] is None else t["scale"] * t["post"]
        if case["act"] != "none":
            w = w * {"identity": lambda q: q, "sigmoid": torch.sigmoid, "silu": torch.nn.functional.silu}[case["act"]](t["q"])
        count = torch.tensor([d for mul, d in blocks for _ in range(mul)], device=DEV)
        v = v * torch.repeat_interleave(w, count, dim=-1)
        out = v if t["h"] is None else v + t["h"]
    return out, _exact_norm(out, blocks, t["pre"]) if case["pre"] else None


def _exact_adamw(s, case):
    g, m, v, norm = s["g"].double(), s["m"], s["v"], None
    if s["m_exp"] is not None:
        def value(code, exp, top):
            code, exp = code.double(), exp.double().clamp(min=E_MIN).repeat_interleave(BLOCK)
            field, mant = torch.div(code, 8, rounding_mode="floor"), code % 8
            low = mant / 8 * torch.exp2(exp - top + 1 - 127)
            return torch.where(field > 0, (1 + mant / 8) * torch.exp2(exp - top + field - 127), low)
        sign = torch.where(m >= 128, -1.0, 1.0).double()
        m, v = sign * value(m % 128, s["m_exp"], M_TOP), value(v, s["v_exp"], V_TOP)
    if s["max_norm"] is not None:
        size = g.pow(2).sum().sqrt()
        coef = (s["max_norm"] / size).clamp(max=1.0)
        norm, g = torch.stack([size, coef]), g * coef
    m = BETAS[0] * m.double() + (1 - BETAS[0]) * g
    v = BETAS[1] * v.double() + (1 - BETAS[1]) * g.pow(2)
    t = case["step"]
    hat_m, hat_v = m / (1 - BETAS[0] ** t), v / (1 - BETAS[1] ** t)
    p = s["p"].double()
    p = p - LR * DECAY * s["decay"].double() * p - LR * hat_m / (hat_v.sqrt() + EPS)
    whole = s["m_exp"] is None     # rounded to 8 bits at random: no value in 64 bits
    return dict(p=p, m=m if whole else None, v=v if whole else None, copy=p if case["copies"] else None, norm=norm)
