"""Cases of the attention along a graph's edges: receivers attend to the states of their sources (another set
of nodes, or the same one), with a learned bias by distance buckets; and the same attention applied to the
rows of per-edge weights that a convolution reads.  Forward and backward of both.

Irreps rows are multiplicity-major: block i of "MULxLP" holds MUL channels of 2L+1 components.  The strings
of a case describe one head: the rows of a tensor hold HEADS times the multiplicity in every block, and head
h owns the h-th run of each block's channels.
"""

import math

import numpy as np
import torch

own = False

DEV = "cuda"
FAR = 5.0                      # cutoff of the synthetic distances


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def listed():
    base = dict(kv=0, degree=32, lengths="fixed", sources=0, buckets=32, bias=False, mask=False, dtype="f32")
    seven, four = "+".join(["8x0e"] * 34), "+".join(["16x0e"] * 18)
    return [
        # the smallest graphs (molecules): one launch, nothing but latency
        dict(base, name="fwd tiny", op="fwd", qk="4x0e", v="4x0e+4x1o", heads=2, n=64, degree=8, buckets=8),
        # a block as wide as the NequIP-like workload's, four heads, logits from scalars
        dict(base, name="fwd nequip", op="fwd", qk="16x0e", v="8x0e+8x1o+8x2e+8x3o", heads=4, n=10000),
        # receivers of one set read the states of a larger one, bfloat16 rows as wide as the large radial
        # workload's; cut edges are masked and some receivers lose all of theirs
        dict(base, name="fwd cross bf16", op="fwd", qk="8x0e+8x1o", v="8x0e+8x1o+8x2e", heads=8, n=50001, sources=200000,
             bias=True, mask=True, dtype="bf16"),
        # a few readout nodes read long runs of nodes; eight heads share two sets of keys and values
        dict(base, name="fwd readout", op="fwd", qk="16x0e", v="16x0e+16x1o", heads=8, kv=2, n=96, degree=2083,
             lengths="ragged", sources=49999),
        # training of a small batch, with a learned function of the distance as a bias
        dict(base, name="bwd tiny", op="bwd", qk="4x0e", v="4x0e+4x1o", heads=2, n=64, degree=8, buckets=8, bias=True),
        # training of the NequIP-like block
        dict(base, name="bwd nequip", op="bwd", qk="16x0e", v="8x0e+8x1o+8x2e+8x3o", heads=4, n=10000),
        # the wide rows in bfloat16 throughout, neighbours counted as they fall
        dict(base, name="bwd uvw bf16", op="bwd", qk="8x0e+8x1o", v="8x0e+8x1o+8x2e", heads=8, n=50001, lengths="poisson",
             sources=200000, mask=True, bias=True, dtype="bf16all"),
        # training of the readout
        dict(base, name="bwd readout", op="bwd", qk="16x0e", v="16x0e+16x1o", heads=8, kv=2, n=96, degree=2083,
             lengths="ragged", sources=49999),
        # attention on the weight rows of the NequIP-like convolution (34 paths of 32 channels)
        dict(base, name="edges fwd nequip", op="edges fwd", qk="16x0e", v=seven, heads=4, n=10000),
        # the same in bfloat16, odd counts, with hubs
        dict(base, name="edges fwd bf16", op="edges fwd", qk="16x0e", v=seven, heads=4, n=9999, lengths="hubs", mask=True,
             bias=True, dtype="bf16"),
        # weight rows of a small batch, backward
        dict(base, name="edges bwd tiny", op="edges bwd", qk="4x0e", v="+".join(["4x0e"] * 5), heads=2, n=64, degree=8, buckets=8),
        # weight rows of the MACE-like convolution (18 paths of 128 channels), backward
        dict(base, name="edges bwd mace", op="edges bwd", qk="16x0e", v=four, heads=8, n=5000, degree=40, lengths="poisson"),
    ]


def draw(rng):
    log = lambda a, b: int(round(math.exp(rng.uniform(math.log(a), math.log(b)))))  # noqa: E731
    op = rng.choice(["fwd", "bwd", "edges fwd", "edges bwd"])
    heads = rng.choice([1, 2, 3, 4, 4, 5, 8, 8, 12, 16])
    top = max(1, 64 // heads)
    mul = lambda: rng.choice([m for m in (1, 2, 4, 8, 16, 32, 64) if m <= top]) if rng.random() < 0.7 else rng.randint(1, top)  # noqa: E731

    def irreps(lmax):
        ls = sorted(rng.sample(range(lmax + 1), rng.randint(1, min(lmax + 1, 4))))
        m = mul()
        return "+".join("%dx%d%s" % (m if rng.random() < 0.8 else mul(), l, "eo"[l % 2]) for l in ls)

    qk = irreps(rng.choice([0, 0, 0, 1, 2]))
    if op.startswith("edges"):
        m = mul()
        v = "+".join(["%dx0e" % m] * max(1, min(rng.randint(1, 34), 2304 // (m * heads))))
    else:
        v = irreps(rng.choice([0, 1, 2, 2, 3, 3, 7]))
    row = heads * (_dim(qk) + _dim(v))
    edges = log(256, max(1024, min(1600000, 450000000 // row)))
    lengths = rng.choice(["fixed", "poisson", "hubs", "ragged"])
    degree = log(200, 5000) if lengths == "ragged" else rng.randint(1, 80)
    n = max(1, edges // (degree * (2 if lengths == "hubs" else 1)))
    dtype = rng.choice(["f32", "f32", "f32", "bf16", "bf16", "bf16all", "f64"])
    if op.startswith("edges") and dtype == "bf16all":
        dtype = "bf16"
    return dict(op=op, qk=qk, v=v, heads=heads, kv=0 if op.startswith("edges") or rng.random() < 0.7 else rng.choice([k for k in (1, 2, 4, 8) if heads % k == 0]),
                n=n, degree=degree, lengths=lengths, sources=max(-(-edges // 16000), log(8, 200000)), buckets=rng.choice([0, 8, 32, 33, 64, 128]),
                bias=rng.random() < 0.4, mask=rng.random() < 0.4, dtype=dtype)


def _blocks(irreps):
    """[(multiplicity, components)] of an irreps string."""
    return [(int(t.split("x")[0]), 2 * int(t.split("x")[1][:-1]) + 1) for t in irreps.split("+")]


def _dim(irreps):
    return sum(m * d for m, d in _blocks(irreps))


def _degrees(case):
    """Edges of every receiver: fixed by the case, so that seeds share their shapes."""
    rng, n, d = np.random.RandomState(case["n"] % 65521 + case["degree"]), case["n"], case["degree"]
    if case["lengths"] == "fixed":
        return np.full(n, d, dtype=np.int64)
    if case["lengths"] == "ragged":
        return rng.randint(0, 2 * d + 1, n).astype(np.int64)
    k = rng.poisson(d, n).astype(np.int64)
    if case["lengths"] == "hubs":
        # few receivers stand for many nodes: together they have about as many edges as all the others
        hubs = np.arange(0, n, 200)
        k[hubs] += d * n // len(hubs)
    return k


def _types(case):
    """Element types of q, k, v and weight rows; of results and gradients; of biases and statistics."""
    f, b, d = torch.float32, torch.bfloat16, torch.float64
    return {"f32": (f, f, f), "bf16": (b, f, f), "bf16all": (b, b, f), "f64": (d, d, d)}[case["dtype"]]


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    store, res, par = _types(case)
    degrees = _degrees(case)
    n, e, heads = case["n"], int(degrees.sum()), case["heads"]
    m, kv = case["sources"] or n, case["kv"] or heads
    dk, dv = _dim(case["qk"]), _dim(case["v"])
    edges = case["op"].startswith("edges")
    s = dict(case=case, n=n, m=m, e=e, heads=heads, kv=kv, dk=dk, dv=dv, scale=dk ** -0.5)

    def rows(count, width, dtype, size=1.0):
        x = torch.randn(count, width, device=DEV, generator=gen)
        return (x * torch.exp(0.3 * torch.randn(count, 1, device=DEV, generator=gen)) * size).to(dtype)

    deg = torch.from_numpy(degrees).to(DEV)
    s["rowptr"] = torch.cat([deg.new_zeros(1), deg.cumsum(0)]).to(torch.int32)
    s["dst"] = torch.repeat_interleave(torch.arange(n, device=DEV), deg, output_size=e)
    s["col"] = torch.randint(0, m, (e,), device=DEV, generator=gen).to(torch.int32)
    s["q"], s["k"] = rows(n, heads * dk, store), rows(m, kv * dk, store)
    s["v"] = rows(e, heads * dv, store, 0.2) if edges else rows(m, kv * dv, store)
    s["lengths"] = s["table"] = s["borders"] = s["bias"] = None
    if case["buckets"]:
        # the near half of the buckets is even in the distance, the far half in its logarithm
        k = case["buckets"]
        near = np.arange(1, k // 2 + 1) * (1.0 / (k // 2))
        far = np.exp(np.linspace(0.0, math.log(FAR), k - k // 2)[1:])
        s["borders"] = torch.from_numpy(np.concatenate([near, far])).to(torch.float32).to(DEV).to(par)
        s["lengths"] = (FAR * 1.05 * torch.rand(e, device=DEV, generator=gen) ** (1 / 3)).to(par)
        s["table"] = (0.5 * torch.randn(k, heads, device=DEV, generator=gen)).to(par)
    if case["bias"] or case["mask"]:
        s["bias"] = (0.3 * torch.randn(e, heads, device=DEV, generator=gen)).to(par)
        if case["mask"]:
            cut = (torch.rand(e, device=DEV, generator=gen) < 0.1) | (s["dst"] % 41 == 7)
            s["bias"].masked_fill_(cut[:, None], -math.inf)
    if case["op"] == "bwd":
        s["gout"] = rows(n, heads * dv, store)
        s["lse"] = _plain_forward(s)[1]            # what the forward left
    elif edges and case["op"].endswith("bwd"):
        s["gout"] = rows(e, heads * dv, res, 0.1)
        s["alpha"] = _plain_edges_forward(s)[1]
    if own:
        import clebsch_gordan_tensor_racah_gb300 as cg
        s["graph"] = cg.Graph(s["rowptr"], s["col"], n, n_src=m)
        s["plan"] = cg.AttentionPlan(case["qk"], case["v"], heads, kv_heads=kv, dtype=store, storage=case["dtype"] == "bf16all",
                                     borders=None if s["borders"] is None else s["borders"].tolist())
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def run(s):
    op = s["case"]["op"]
    if own:
        import clebsch_gordan_tensor_racah_gb300 as cg
        more = dict(lengths=s["lengths"], table=s["table"], bias=s["bias"])
        if op == "fwd":
            r = cg.cgtp_attn_forward(s["plan"], s["graph"], s["q"], s["k"], s["v"], **more)
        elif op == "bwd":
            r = cg.cgtp_attn_backward(s["plan"], s["graph"], s["gout"], s["q"], s["k"], s["v"], s["lse"],
                                      need_gbias=s["case"]["bias"], **more)
        elif op == "edges fwd":
            r = cg.cgtp_attn_edges_forward(s["plan"], s["graph"], s["q"], s["k"], s["v"], **more)
        else:
            r = cg.cgtp_attn_edges_backward(s["plan"], s["graph"], s["gout"], s["q"], s["k"], s["v"], s["alpha"],
                                            lengths=s["lengths"], need_gbias=s["case"]["bias"])
    else:
        r = {"fwd": _plain_forward, "bwd": _plain_backward, "edges fwd": _plain_edges_forward, "edges bwd": _plain_edges_backward}[op](s)
    names = {"fwd": ("out", "lse"), "edges fwd": ("w", "alpha"), "bwd": ("gq", "gk", "gv", "gtable", "gbias"),
             "edges bwd": ("gq", "gk", "gw", "gtable", "gbias")}[op]
    return dict(zip(names, r))


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------

def _wide(x):
    return x if x.dtype == torch.float64 else x.float()


def _split(x, irreps, heads):
    """Rows as [rows, heads, elements of a head]."""
    blocks = _blocks(irreps)
    parts = torch.split(_wide(x), [heads * m * d for m, d in blocks], dim=1)
    return torch.cat([p.unflatten(1, (heads, -1)) for p in parts], dim=2)


def _join(x, irreps):
    """The inverse of _split."""
    return torch.cat([p.flatten(1) for p in torch.split(x, [m * d for m, d in _blocks(irreps)], dim=2)], dim=1)


def _spread(s, x):
    """Keys or values of every head, from those that its group shares."""
    return x if s["kv"] == s["heads"] else x.repeat_interleave(s["heads"] // s["kv"], dim=1)


def _gather(s, x):
    return _spread(s, x[s["col"].long()])


def _collect(s, x):
    """Sums of edge values [e, heads, .] over the edges of each source and the heads of each group."""
    if s["kv"] != s["heads"]:
        x = x.unflatten(1, (s["kv"], -1)).sum(2)
    # long sums in 64 bits: few sources may have thousands of edges each
    wide = x.double() if s["e"] > 256 * s["m"] else x
    return torch.zeros((s["m"],) + x.shape[1:], dtype=wide.dtype, device=DEV).index_add_(0, s["col"].long(), wide).to(x.dtype)


def _receive(s, x):
    """Sums over the edges of each receiver."""
    return torch.zeros((s["n"],) + x.shape[1:], dtype=x.dtype, device=DEV).index_add_(0, s["dst"], x)


def _logits(s):
    q, k = _split(s["q"], s["case"]["qk"], s["heads"]), _split(s["k"], s["case"]["qk"], s["kv"])
    z = (q[s["dst"]] * _gather(s, k)).sum(2) * s["scale"]
    if s["table"] is not None:
        z = z + s["table"][_bucket(s)]
    return z if s["bias"] is None else z + s["bias"]


def _bucket(s):
    return (s["lengths"][:, None] >= s["borders"]).sum(1)


def _softmax(s, z):
    """Weights over each receiver's edges (zeros where nothing is left), and log of the sum of exponentials."""
    top = torch.full((s["n"], s["heads"]), -math.inf, dtype=z.dtype, device=DEV)
    top = top.scatter_reduce_(0, s["dst"][:, None].expand_as(z), z, "amax")
    shift = torch.where(top == -math.inf, 0.0, top)
    p = torch.exp(z - shift[s["dst"]])
    total = _receive(s, p)
    a = p / torch.where(total == 0, 1.0, total)[s["dst"]]
    return a, torch.log(total) + shift


def _plain_forward(s):
    a, lse = _softmax(s, _logits(s))
    v = _gather(s, _split(s["v"], s["case"]["v"], s["kv"]))
    out = _receive(s, a[:, :, None] * v)
    return _join(out, s["case"]["v"]).to(_types(s["case"])[1]), lse


def _plain_edges_forward(s):
    a, _ = _softmax(s, _logits(s))
    w = a[:, :, None] * _split(s["v"], s["case"]["v"], s["heads"])
    return _join(w, s["case"]["v"]).to(s["v"].dtype), a


def _finish(s, ds):
    """Gradients of queries, keys, table and bias for the gradient of the logits."""
    res = _types(s["case"])[1]
    q, k = _split(s["q"], s["case"]["qk"], s["heads"]), _split(s["k"], s["case"]["qk"], s["kv"])
    gq = _receive(s, ds[:, :, None] * _gather(s, k)) * s["scale"]
    gk = _collect(s, ds[:, :, None] * q[s["dst"]]) * s["scale"]
    gtable = None
    if s["table"] is not None:
        # long sums of both signs
        gtable = torch.zeros(s["table"].shape, dtype=torch.float64, device=DEV).index_add_(0, _bucket(s), ds.double()).to(s["table"].dtype)
    return _join(gq, s["case"]["qk"]).to(res), _join(gk, s["case"]["qk"]).to(res), gtable, ds if s["case"]["bias"] else None


def _plain_backward(s):
    z = _logits(s)
    p = torch.where(z == -math.inf, 0.0, torch.exp(z - s["lse"][s["dst"]]))
    g = _split(s["gout"], s["case"]["v"], s["heads"])[s["dst"]]
    dp = (g * _gather(s, _split(s["v"], s["case"]["v"], s["kv"]))).sum(2)
    gv = _collect(s, p[:, :, None] * g)
    # the mean of dp from the edges themselves: the stored result is rounded
    gq, gk, gtable, gbias = _finish(s, p * (dp - _receive(s, p * dp)[s["dst"]]))
    return gq, gk, _join(gv, s["case"]["v"]).to(_types(s["case"])[1]), gtable, gbias


def _plain_edges_backward(s):
    a, irreps, heads = s["alpha"], s["case"]["v"], s["heads"]
    g = _split(s["gout"], irreps, heads)
    dp = (g * _split(s["v"], irreps, heads)).sum(2)
    gw = _join(a[:, :, None] * g, irreps).to(_types(s["case"])[1])
    gq, gk, gtable, gbias = _finish(s, a * (dp - _receive(s, a * dp)[s["dst"]]))
    return gq, gk, gw, gtable, gbias


# ---------------------------------------------------------------------------
# work and exact values
# ---------------------------------------------------------------------------

def work(case):
    store, res, par = (t.itemsize for t in _types(case))
    n, e, heads = case["n"], int(_degrees(case).sum()), case["heads"]
    m, kv = min(case["sources"] or n, e), case["kv"] or heads
    dk, dv = _dim(case["qk"]), _dim(case["v"])
    back, edges = case["op"].endswith("bwd"), case["op"].startswith("edges")
    size = store * (n * heads * dk + m * kv * dk + (e * heads if edges else m * kv) * dv) + 4 * (n + 1 + e)
    if case["buckets"]:
        size += par * (e + case["buckets"] * heads * (2 if back else 1))
    if (case["bias"] or case["mask"]) and not (back and edges):
        size += par * e * heads
    if back:
        size += res * (n * heads * dk + m * kv * dk) + (par * e * heads if case["bias"] else 0)
        size += 2 * res * e * heads * dv + par * e * heads if edges else res * m * kv * dv + store * n * heads * dv + par * n * heads
    else:
        size += store * e * heads * dv + par * e * heads if edges else res * n * heads * dv + par * n * heads
    # a product and a sum of every element of a head: logits, results, and their gradients
    flops = e * heads * ((4 * dk + 3 * dv if edges else 6 * dk + 4 * dv) if back else (2 * dk + dv if edges else 2 * dk + 2 * dv))
    return dict(bytes=size, flops=flops)


def exact(case, seed):
    """The definition in 64 bits, a group of receivers of like length at a time, gradients by differentiating it."""
    s = prepare(case, seed)
    heads, kv, group = s["heads"], s["kv"], s["heads"] // s["kv"]
    back, edges = case["op"].endswith("bwd"), case["op"].startswith("edges")

    def index(irreps, count):
        """Columns of each head's elements, [count, elements]."""
        at, cols = 0, []
        for mul, d in _blocks(irreps):
            cols.append(at + torch.arange(count * mul * d).view(count, mul * d))
            at += count * mul * d
        return torch.cat(cols, 1).to(DEV)

    iq, ik = index(case["qk"], heads), index(case["qk"], kv)
    iv, io = index(case["v"], heads if edges else kv), index(case["v"], heads)
    q, k, v = s["q"].double()[:, iq], s["k"].double()[:, ik], s["v"].double()[:, iv]
    deg, start = (s["rowptr"][1:] - s["rowptr"][:-1]).long(), s["rowptr"][:-1].long()
    table = None if s["table"] is None else s["table"].double()
    which = None if table is None else torch.bucketize(s["lengths"], s["borders"], right=True)
    zeros = lambda *shape: torch.zeros(shape, dtype=torch.float64, device=DEV)  # noqa: E731
    out, lse = zeros(*(s["v"].shape if edges else (s["n"], heads * s["dv"]))), torch.full((s["n"], heads), -math.inf, dtype=torch.float64, device=DEV)
    alpha, gbias = zeros(s["e"], heads), zeros(s["e"], heads)
    gq, gk, gv, gtable = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v), None if table is None else torch.zeros_like(table)
    order = torch.argsort(deg, descending=True)
    lens = deg[order].tolist()
    i = 0
    while i < s["n"] and lens[i] > 0:
        take = max(1, (1 << 28) // (lens[i] * heads * (s["dk"] + s["dv"])))
        r = order[i:i + take][:max(1, sum(x > 0 for x in lens[i:i + take]))]
        i += len(r)
        place = start[r][:, None] + torch.arange(lens[i - len(r)], device=DEV)
        real = place < (start[r] + deg[r])[:, None]
        place = torch.where(real, place, start[r][:, None])
        src = s["col"][place].long()
        leaves = [q[r], k[src], v[place] if edges else v[src]]
        t = None if table is None else table[which[place]]
        b = zeros(len(r), place.shape[1], heads) if s["bias"] is None else s["bias"].double()[place]
        b = b.masked_fill(~real[:, :, None], -math.inf)
        b = b if t is None else b + t
        if back:
            leaves, b = [x.requires_grad_() for x in leaves], b.requires_grad_()
        z = torch.einsum("nkgd,njkd->njkg", leaves[0].unflatten(1, (kv, group)), leaves[1]).flatten(2) * s["scale"] + b
        dead = (z == -math.inf).all(1, keepdim=True)
        a = torch.softmax(z.masked_fill(dead, 0.0), 1).masked_fill(dead, 0.0)
        if edges:
            y = a[..., None] * leaves[2]
        else:
            y = torch.einsum("njkg,njkd->nkgd", a.unflatten(2, (kv, group)), leaves[2]).flatten(1, 2)
        at = place[real]
        if back:
            up = s["gout"].double()[:, io]
            g = torch.autograd.grad(y, leaves + [b], (up[place] * real[..., None, None]) if edges else up[r])
            gq[r] = g[0]
            gk.index_add_(0, src.flatten(), g[1].flatten(0, 1))
            if edges:
                gv[at] = g[2][real]
            else:
                gv.index_add_(0, src.flatten(), g[2].flatten(0, 1))
            gbias[at] = g[3][real]
        else:
            alpha[at] = a[real].detach()
            if edges:
                out[at[:, None, None], io] = y[real]
            else:
                out[r[:, None, None], io] = y
            lse[r] = torch.logsumexp(z, 1)
    if not back:
        return dict(w=out, alpha=alpha) if edges else dict(out=out, lse=lse)
    if gtable is not None:
        gtable.index_add_(0, which, gbias)

    def rows(x, cols, like):
        full = zeros(*like.shape)
        full[:, cols] = x
        return full

    return {"gq": rows(gq, iq, s["q"]), "gk": rows(gk, ik, s["k"]), ("gw" if edges else "gv"): rows(gv, iv, s["v"]),
            "gtable": gtable, "gbias": gbias if case["bias"] else None}
