"""Attention along a graph's edges on the GPU against the FP64 oracle.

Tolerances.  u = 2^-24 (FP32) or 2^-53 (FP64), all in units of the sums of magnitudes.
  z: dk products and sums, the scale and two biases, each relative to Z = scale sum |q k| + |T| + |b|: (dk + 5) u Z.
  a = exp(z - max) / sum: an absolute error of z is a relative one of exp (2 u of its own); numerator, sum (deg + 2
     roundings) and the maximum's logit: Ka = 2 (dk + 5) max Z + deg + 8.  lse: Ka u + 2 u |lse|.  The backward takes exp(z - lse)
     with the kernel's own lse: twice that, Kp = 2 Ka + 2 max |lse|.
  out: (Ka + deg + 4) u sum a |v|.
  dp: (dv + 2) u G, G = sum |gout v|; D = sum a dp: relative to Gm = sum a G.  ds = a (dp - D):
     Kd = Kp + dv + deg + 12 times u a (G + Gm), and |ds| <= a (G + Gm).
  gq, gk: (Kd + deg + 6) u scale sum a (G + Gm) |k| or |q|, deg the longest row of either side times the heads of
     a group; gv: (Kp + deg + 4) u sum a |gout|; table: at most 80 values of a lane and 48 columns of its CTA are added in
     the arithmetic's type, the CTAs in FP64: (Kd + 128) u sum a (G + Gm).
Results stored in bfloat16 add half a step, 2^-8 of the value.
"""

import numpy as np
import pytest

from oracle import attn as oat
from oracle.train import sizes

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

KINDS = ["f32", "f64", "bf16", "bf16s"]
NAMES = {"fwd": ("out", "lse"), "bwd": ("gq", "gk", "gv", "gtable", "gbias"), "efwd": ("w", "alpha"),
         "ebwd": ("gq", "gk", "gw", "gtable", "gbias")}
# one head's queries and values, heads, shared heads
SHAPES = [("16x0e", "8x0e+8x1o+8x2e+8x3o", 4, 4), ("4x0e", "4x0e+4x1o", 2, 2), ("8x0e+8x1o", "8x0e+8x1o+8x2e", 8, 8),
          ("16x0e", "16x0e+16x1o", 8, 2), ("1x0e", "1x0e", 1, 1), ("3x0e+1x1o", "5x0e+2x1o", 3, 1), ("5x0e", "1x7o", 5, 5),
          ("2x0e", "64x0e", 12, 4), ("64x0e", "2x0e+2x1o", 16, 16), ("1x0e", "2x0e", 64, 8), ("128x0e+128x1o", "128x0e+128x1o+128x2e", 1, 1),
          ("8x0e", "300x0e", 7, 7), ("16x0e", "+".join(["16x0e"] * 18), 8, 8), ("33x0e", "33x0e+17x1o+5x2e", 2, 1)]
DEGREES = {"few": lambda rng, n: rng.integers(0, 4, n), "usual": lambda rng, n: rng.poisson(20, n),
           "mixed": lambda rng, n: np.where(np.arange(n) % 9 == 4, rng.integers(65, 700, n), rng.integers(0, 12, n)),
           "one": lambda rng, n: np.where(np.arange(n) == n // 2, 1500, 0)}


def cg():
    import clebsch_gordan_tensor_racah_gb300 as m
    return m


def _types(kind):
    f, b, d = torch.float32, torch.bfloat16, torch.float64
    return {"f32": (f, f, f), "f64": (d, d, d), "bf16": (b, f, f), "bf16s": (b, b, f)}[kind]


def _num(t):
    return None if t is None else t.double().cpu().numpy()


def _dev(a, dtype, layout="plain"):
    """Rows on the GPU: contiguous, a column range of wider rows, or one that starts off 16 bytes."""
    t = torch.from_numpy(np.ascontiguousarray(a)).to("cuda").to(dtype)
    if layout == "plain" or t.dim() == 1:
        return t
    left, right = (8, 24) if layout == "range" else (3, 2)
    wide = torch.full((t.shape[0], t.shape[1] + left + right), 7.0, dtype=dtype, device="cuda")
    wide[:, left:left + t.shape[1]] = t
    return wide[:, left:left + t.shape[1]]


class Case:
    """Inputs, the plan and the graph of one shape, and what the oracle says."""

    def __init__(self, shape, kind="f32", degrees="usual", n=40, m=23, borders=7, bias=True, mask=False, layout="plain", seed=0, edges=False,
                 size=1.0):
        rng = np.random.default_rng(seed)
        self.qk, self.v, self.heads, self.kv = shape
        self.kind, self.edges, self.layout = kind, edges, layout
        store, self.res, self.par = _types(kind)
        deg = DEGREES[degrees](rng, n) if isinstance(degrees, str) else np.asarray(degrees)
        self.n, self.m, self.e = len(deg), m, int(deg.sum())
        self.rowptr = np.concatenate([[0], np.cumsum(deg)])
        self.dst, self.col = np.repeat(np.arange(self.n), deg), rng.integers(0, m, self.e)
        dk, dv, h, kv = sizes(self.qk)[0], sizes(self.v)[0], self.heads, self.kv
        f = lambda *s: rng.standard_normal(s)  # noqa: E731
        self.q, self.k = _dev(size * f(self.n, h * dk), store, layout), _dev(f(m, kv * dk), store, layout)
        self.x = _dev(f(self.e, h * dv) if edges else f(m, kv * dv), store, layout)
        self.gout = _dev(f(self.e if edges else self.n, h * dv), self.res if edges else store, layout)
        self.borders = np.sort(rng.uniform(0.5, 5, borders)) if borders else None
        self.lengths = _dev(rng.uniform(0, 6, self.e), self.par) if borders else None
        self.table = _dev(f(borders + 1, h), self.par) if borders else None
        b = 0.5 * f(self.e, h)
        if mask:
            b[rng.random((self.e, h)) < 0.2] = -np.inf
            b[self.dst % 5 == 2] = -np.inf
        self.bias = _dev(b, self.par) if bias or mask else None
        self.plan = cg().AttentionPlan(self.qk, self.v, h, kv_heads=kv, dtype=store, storage=kind == "bf16s", borders=self.borders)
        self.graph = cg().Graph(_dev(self.rowptr, torch.int32), _dev(self.col, torch.int32), self.n, n_src=m)
        self.more = dict(lengths=self.lengths, table=self.table, bias=self.bias)

    # -- the kernels ---------------------------------------------------------------------------------
    def run(self, op, **kw):
        c, p, g = cg(), self.plan, self.graph
        if op == "fwd":
            return c.cgtp_attn_forward(p, g, self.q, self.k, self.x, **self.more, **kw)
        if op == "efwd":
            return c.cgtp_attn_edges_forward(p, g, self.q, self.k, self.x, **self.more, **kw)
        if op == "bwd":
            lse = c.cgtp_attn_forward(p, g, self.q, self.k, self.x, **self.more)[1]
            return c.cgtp_attn_backward(p, g, self.gout, self.q, self.k, self.x, lse, need_gbias=True, **self.more, **kw)
        alpha = c.cgtp_attn_edges_forward(p, g, self.q, self.k, self.x, **self.more)[1]
        return c.cgtp_attn_edges_backward(p, g, self.gout, self.q, self.k, self.x, alpha, lengths=self.lengths, need_gbias=True, **kw)

    # -- the oracle: value, bound of the error in units of u ---------------------------------------
    def bounds(self):
        heads, kv, dst, col, n, m = self.heads, self.kv, self.dst, self.col, self.n, self.m
        q, k, x = _num(self.q), _num(self.k), _num(self.x)
        b = 0.0 if self.bias is None else _num(self.bias)
        which = None
        if self.table is not None:
            borders = np.asarray(self.borders).astype(np.float32 if self.par == torch.float32 else np.float64)
            which = oat.buckets(self.lengths.cpu().numpy(), borders)
            b = b + _num(self.table)[which]
        scale = self.plan.scale
        z, mag = oat.logits(q, k, self.qk, heads, kv, scale, dst, col, b)
        a, lse = oat.softmax(z, dst, n)
        dk, dv = sizes(self.qk)[0], sizes(self.v)[0]
        deg = max(1, np.bincount(dst, minlength=1).max(initial=0), np.bincount(col, minlength=1).max(initial=0)) * (heads // kv)
        ka = 2 * (dk + 5) * mag.max(initial=0) + deg + 8
        fin = lse[np.isfinite(lse)]
        out = {}
        xs = oat.spread(x, self.v, heads if self.edges else kv, heads)
        rows = xs if self.edges else xs[col]
        io = lambda y, count, like: oat.gather_back(y, self.v, count, like)  # noqa: E731
        wa, wm = oat.weighed(a, rows), oat.weighed(a, np.abs(rows))
        shape = (self.e if self.edges else n, heads * dv)
        if self.edges:
            out["w"] = io(wa, heads, shape), (ka + 2) * io(wm, heads, shape)
            out["alpha"] = a, ka * a
            kp = ka
        else:
            r = lambda y: io(oat.receive(y, dst, n), heads, shape)  # noqa: E731
            out["out"] = r(wa), (ka + deg + 4) * r(wm)
            out["lse"] = lse, ka + 2 * np.abs(np.where(np.isfinite(lse), lse, 0))
            kp = 2 * ka + 2 * np.abs(fin).max(initial=0)
        g = oat.spread(_num(self.gout), self.v, heads, heads)
        ge = g if self.edges else g[dst]
        dead = a == 0
        rows = np.where(dead[:, :, None], 0, rows)
        prod = np.where(dead[:, :, None], 0, ge) * rows
        dp, big = prod.sum(2), np.abs(prod).sum(2)
        ds = oat.logit_gradient(a, dp, dst, n)
        dm = a * (big + oat.receive(a * big, dst, n)[dst])
        kd = kp + dv + deg + 12
        kh, qh = oat.spread(k, self.qk, kv, heads)[col], oat.spread(q, self.qk, heads, heads)[dst]
        kh, qh = np.where(dead[:, :, None], 0, kh), np.where(dead[:, :, None], 0, qh)
        to_q = lambda y: oat.gather_back(oat.receive(y, dst, n), self.qk, heads, (n, heads * dk))  # noqa: E731
        to_k = lambda y: oat.gather_back(oat.receive(y, col, m), self.qk, kv, (m, kv * dk))  # noqa: E731
        out["gq"] = scale * to_q(ds[:, :, None] * kh), (kd + deg + 6) * scale * to_q(dm[:, :, None] * np.abs(kh))
        out["gk"] = scale * to_k(ds[:, :, None] * qh), (kd + deg + 6) * scale * to_k(dm[:, :, None] * np.abs(qh))
        ge = np.where(dead[:, :, None], 0, ge)
        if self.edges:
            out["gw"] = io(oat.weighed(a, ge), heads, shape), (kp + 4) * io(oat.weighed(a, np.abs(ge)), heads, shape)
        else:
            to_v = lambda y: io(oat.receive(y, col, m), kv, (m, kv * dv))  # noqa: E731
            out["gv"] = to_v(oat.weighed(a, ge)), (kp + deg + 4) * to_v(oat.weighed(a, np.abs(ge)))
        out["gbias"] = ds, kd * dm
        if which is not None:
            to_t = lambda y: oat.receive(y, which, len(self.borders) + 1)  # noqa: E731
            out["gtable"] = to_t(ds), (kd + 128) * to_t(dm)
        return out

    def check(self, ops):
        want = self.bounds()
        u = 2.0 ** -53 if self.kind == "f64" else 2.0 ** -24
        for op in ops:
            for name, got in zip(NAMES[op], self.run(op)):
                if name == "gtable" and self.table is None:
                    assert got is None
                    continue
                value, bound = want[name]
                # the rows of edges are stored as the weights are, their gradient in the arithmetic's type
                stored = {"w": _types(self.kind)[0], "gw": self.par, "lse": self.par, "alpha": self.par, "gtable": self.par, "gbias": self.par}
                dtype = stored.get(name, self.par if self.edges else self.res)
                assert got.dtype == dtype and tuple(got.shape) == value.shape, (op, name)
                got = _num(got)
                fin = np.isfinite(value)
                assert np.array_equal(got[~fin], value[~fin]), (op, name)
                tol = np.broadcast_to(u * bound + (2.0 ** -8 * np.abs(np.where(fin, value, 0)) if dtype == torch.bfloat16 else 0) + 1e-37, value.shape)
                bad = np.abs(got - np.where(fin, value, got)) > np.where(fin, tol, 0)
                assert not bad[fin].any(), (op, name, np.abs(got - value)[fin].max(), int(bad.sum()))


@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: f"{s[2]}of{s[3]}:{s[0]}:{s[1][:20]}")
@pytest.mark.parametrize("kind", KINDS)
def test_values_against_the_oracle(shape, kind):
    Case(shape, kind, "usual", seed=1).check(["fwd", "bwd"])


@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: f"{s[2]}of{s[3]}:{s[0]}:{s[1][:20]}")
@pytest.mark.parametrize("kind", ["f32", "f64", "bf16"])
def test_edge_rows_against_the_oracle(shape, kind):
    Case(shape, kind, "usual", seed=2, edges=True).check(["efwd", "ebwd"])


@pytest.mark.parametrize("degrees", sorted(DEGREES))
@pytest.mark.parametrize("edges", [False, True])
@pytest.mark.parametrize("shape", [SHAPES[i] for i in (0, 3, 5, 9)], ids=lambda s: f"{s[2]}of{s[3]}")
def test_rows_of_any_length(degrees, edges, shape):
    ops = ["efwd", "ebwd"] if edges else ["fwd", "bwd"]
    Case(shape, "f32", degrees, n=37, m=11, seed=3, edges=edges).check(ops)
    Case(shape, "bf16", degrees, n=61, m=301, seed=4, edges=edges, mask=True).check(ops)


@pytest.mark.parametrize("layout", ["range", "odd"])
@pytest.mark.parametrize("kind", KINDS)
def test_column_ranges_of_wider_rows(layout, kind):
    Case(SHAPES[0], kind, layout=layout, seed=5).check(["fwd", "bwd"])
    if kind != "bf16s":
        Case(SHAPES[0], kind, layout=layout, seed=6, edges=True).check(["efwd", "ebwd"])


@pytest.mark.parametrize("borders,bias", [(0, False), (0, True), (1, False), (511, True)])
@pytest.mark.parametrize("edges", [False, True])
def test_terms_of_the_logits(borders, bias, edges):
    for heads in (4, 40):
        Case(("4x0e", "4x0e+1x1o", heads, heads), "f32", "mixed", borders=borders, bias=bias, seed=7, edges=edges).check(
            ["efwd", "ebwd"] if edges else ["fwd", "bwd"])


@pytest.mark.parametrize("sizes_", [(1, 1, [1]), (1, 5, [0]), (3, 1, [0, 0, 0]), (1, 3, [3000]), (2, 4, [1, 2]), (1, 70000, [5])])
@pytest.mark.parametrize("edges", [False, True])
def test_the_smallest_graphs_and_single_receivers(sizes_, edges):
    _, m, deg = sizes_
    for shape in (SHAPES[0], SHAPES[4], SHAPES[10]):
        Case(shape, "f32", deg, m=m, seed=8, edges=edges).check(["efwd", "ebwd"] if edges else ["fwd", "bwd"])


@pytest.mark.parametrize("edges", [False, True])
def test_many_short_rows(edges):
    rng = np.random.default_rng(9)
    Case(("2x0e", "3x0e", 2, 2), "f32", rng.integers(0, 3, 20000), m=700, seed=9, edges=edges).check(["efwd", "ebwd"] if edges else ["fwd", "bwd"])
    Case(SHAPES[0], "f32", rng.integers(0, 40, 2500), m=2500, seed=9, edges=edges).check(["efwd", "ebwd"] if edges else ["fwd", "bwd"])


@pytest.mark.parametrize("edges", [False, True])
def test_masked_edges_hold_anything(edges):
    # rows that only masked edges touch hold infinities and NaN; a masked weight row too
    c = Case(SHAPES[0], "f32", "mixed", m=40, seed=10, edges=edges, mask=True)
    cut = np.flatnonzero(np.isin(c.col, range(5)))
    c.bias[torch.from_numpy(cut).cuda()] = -np.inf
    want = c.bounds()
    for s, v in zip(range(5), (np.nan, np.inf, -np.inf, 3e38, np.nan)):
        c.k[s] = v
        if not edges:
            c.x[s] = v
    if edges:
        c.x[torch.from_numpy(cut).cuda()] = np.nan
        c.gout[torch.from_numpy(cut).cuda()] = np.inf
    for op in ("efwd", "ebwd") if edges else ("fwd", "bwd"):
        for name, got in zip(NAMES[op], c.run(op)):
            value, bound = want[name]
            fin = np.isfinite(value)
            assert np.all(np.abs(_num(got) - value)[fin] <= np.broadcast_to(2.0 ** -24 * bound + 1e-37, value.shape)[fin]), (op, name)


def test_masks_of_the_lowest_value():
    # finite masks: a row of them all still sums to one, and every weight is that of the softmax
    c = Case(SHAPES[1], "f32", [6, 6, 0, 3], m=9, borders=0, seed=11)
    low = torch.finfo(torch.float32).min
    c.bias[:] = 0
    c.bias[0:6] = low
    c.bias[6:9] = low
    out, lse = c.run("fwd")
    assert torch.isfinite(out).all() and torch.isfinite(lse[:2]).all() and torch.isneginf(lse[2]).all()
    a = cg().cgtp_attn_edges_forward(cg().AttentionPlan("4x0e", "1x0e", 2), c.graph, c.q, c.k, torch.ones(c.e, 2, device="cuda"), bias=c.bias)[1]
    # the logits are lost beside the mask: it is added in the arithmetic's type, like any other bias
    assert torch.equal(a[:6], torch.full_like(a[:6], 1 / 6)) and torch.equal(a[6:9], torch.zeros_like(a[6:9]))


def test_large_logits():
    # logits of thousands: weights of zero and one, no overflow
    Case(SHAPES[0], "f32", "mixed", seed=12, size=600.0).check(["fwd"])
    c = Case(SHAPES[0], "f32", "mixed", seed=12, size=1e4)
    out, lse = c.run("fwd")
    assert torch.isfinite(out).all() and torch.isfinite(lse[torch.from_numpy(np.diff(c.rowptr) > 0).cuda()]).all()
    for t in c.run("bwd"):
        assert torch.isfinite(t).all()


def test_nan_and_infinite_logits_reach_their_receiver_only():
    c = Case(SHAPES[0], "f32", [5, 5, 200, 5], m=900, borders=0, seed=13)
    clean = c.run("fwd")[0].clone()
    for value in (np.nan, np.inf):
        c.bias[7, 1] = value
        out, lse = c.run("fwd")
        head = np.zeros(out.shape, bool)
        head[1, oat.columns(c.v, c.heads)[1]] = True
        head = torch.from_numpy(head).cuda()
        assert torch.isnan(out[head]).all() and torch.equal(out[~head], clean[~head]) and torch.isnan(lse[1, 1]) == True  # noqa: E712


def test_nan_lengths_and_borders():
    c = Case(SHAPES[1], "f32", "usual", seed=14)
    b = torch.tensor(c.borders, dtype=torch.float32, device="cuda")
    c.lengths[:7] = b          # a border belongs to the bucket above it
    c.lengths[7] = float("nan")
    c.lengths[8], c.lengths[9] = float("inf"), -1.0
    c.check(["fwd", "bwd"])


@pytest.mark.parametrize("edges", [False, True])
def test_results_repeat_bit_for_bit(edges):
    for degrees in ("mixed", "usual"):
        c = Case(SHAPES[3], "f32", degrees, n=300, m=37, seed=15, edges=edges)
        for op in ("efwd", "ebwd") if edges else ("fwd", "bwd"):
            first = [t.clone() for t in c.run(op)]
            for _ in range(3):
                assert all(torch.equal(a, b) for a, b in zip(first, c.run(op)))


@pytest.mark.parametrize("edges", [False, True])
def test_gradients_against_differences(edges):
    c = Case(("3x0e+1x1o", "2x0e+1x1o", 4, 4 if edges else 2), "f64", "usual", n=9, m=7, seed=16, edges=edges)
    fwd, bwd = ("efwd", "ebwd") if edges else ("fwd", "bwd")
    grads = dict(zip(("q", "k", "x", "table", "bias"), c.run(bwd)))
    rng = np.random.default_rng(17)
    for name, grad in grads.items():
        t = getattr(c, name)
        d = torch.from_numpy(rng.standard_normal(tuple(t.shape))).cuda()
        step, keep, vals = 1e-5, t.clone(), []
        for s in (step, -step):
            t.copy_(keep + s * d)
            vals.append(float((c.run(fwd)[0] * c.gout).sum()))
        t.copy_(keep)
        # central difference: step^2 times a third derivative of order one, plus u / step
        want = float((grad * d).sum())
        assert abs((vals[0] - vals[1]) / (2 * step) - want) <= 1e-7 * (1 + float((grad.abs() * d.abs()).sum())), name


def test_rows_of_zero_weights_are_zeros_not_leftovers():
    c = Case(SHAPES[0], "f32", "mixed", seed=18, mask=True)
    out = torch.full((c.n, c.plan.out_dim + 5), 9.0, device="cuda")
    r, lse = c.run("fwd", out=out[:, 2:2 + c.plan.out_dim])
    assert r.data_ptr() == out[:, 2:].data_ptr()
    assert (out[:, :2] == 9).all() and (out[:, 2 + c.plan.out_dim:] == 9).all()
    empty = torch.isneginf(lse).all(1)
    assert empty.any() and (r[empty] == 0).all()


def test_side_stream_capture_and_two_graphs_at_once():
    c = Case(SHAPES[0], "f32", "mixed", n=200, m=50, seed=19)
    e = Case(SHAPES[0], "f32", "mixed", n=200, m=50, seed=20, edges=True)
    want = [[t.clone() for t in x.run(op)] for x, op in ((c, "fwd"), (c, "bwd"), (e, "efwd"), (e, "ebwd"))]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = [x.run(op, stream=side) if op in ("fwd", "efwd") else None for x, op in ((c, "fwd"), (c, "bwd"), (e, "efwd"), (e, "ebwd"))]
    side.synchronize()
    for a, b in zip(want, got):
        assert b is None or all(torch.equal(x, y) for x, y in zip(a, b))
    graphs = []
    for x, op in ((c, "bwd"), (e, "ebwd"), (c, "bwd")):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            r = x.run(op)
        graphs.append((g, r))
    for (g, r) in graphs:
        for t in r:
            t.zero_()
    torch.cuda.synchronize()
    # the same plan and the same graph object, replayed on two streams at once: each call has a workspace of its own
    other = torch.cuda.Stream()
    for _ in range(5):
        for i, (g, _) in enumerate(graphs):
            with torch.cuda.stream(side if i == 0 else other):
                g.replay()
    torch.cuda.synchronize()
    for (g, r), w in zip(graphs, (want[1], want[3], want[1])):
        assert all(torch.equal(a, b) for a, b in zip(r, w))


def test_a_graph_between_two_sets():
    c = Case(SHAPES[0], "f32", "usual", n=30, m=11, seed=21)
    t_rowptr, t_eid, t_dst = c.graph.transpose()
    order = np.argsort(c.col, kind="stable")
    assert np.array_equal(t_eid.cpu().numpy(), order) and np.array_equal(t_dst.cpu().numpy(), c.dst[order])
    assert np.array_equal(t_rowptr.cpu().numpy(), np.concatenate([[0], np.cumsum(np.bincount(c.col, minlength=c.m))]))
    plan = cg().Plan("8x0e", "1x0e", "8x0e", "uvu")
    x, Y, W = (torch.zeros(s, device="cuda") for s in ((c.m, 8), (c.e, 1), (c.e, 8)))
    with pytest.raises(cg().CgtpError, match="another set"):
        cg().cgtp_conv_forward(plan, c.graph, x, Y, W)
    with pytest.raises(cg().CgtpError, match="another set"):
        cg().cgtp_conv_backward(plan, c.graph, torch.zeros(c.n, 8, device="cuda"), x, Y, W)
    rowptr, col = _dev(c.rowptr, torch.int32), _dev(c.col, torch.int32)
    with pytest.raises(cg().CgtpError, match="invalid CSR"):
        cg().Graph(rowptr, col, c.n, n_src=int(c.col.max()))
    with pytest.raises(cg().CgtpError):
        cg().Graph(rowptr, col, c.n, n_src=0)


def test_refusals():
    c = Case(SHAPES[0], "f32", "usual", seed=22)
    e = Case(SHAPES[0], "f32", "usual", seed=22, edges=True)
    f, b = cg().cgtp_attn_forward, cg().cgtp_attn_backward
    ok = dict(lengths=c.lengths, table=c.table)
    lse = f(c.plan, c.graph, c.q, c.k, c.x, **ok)[1]
    bad = [(TypeError, lambda: f(c.plan, c.graph, c.q.double(), c.k, c.x)), (TypeError, lambda: f(c.plan, c.graph, c.q.cpu(), c.k, c.x)),
           (TypeError, lambda: f(c.plan, c.graph, None, c.k, c.x)), (TypeError, lambda: f(c.plan, c.graph, c.q, c.k, None)),
           (ValueError, lambda: f(c.plan, c.graph, c.q[1:], c.k, c.x)), (ValueError, lambda: f(c.plan, c.graph, c.q, c.k[1:], c.x)),
           (ValueError, lambda: f(c.plan, c.graph, c.q[:, :-1], c.k, c.x)), (ValueError, lambda: f(c.plan, c.graph, c.q, c.k, c.x, lengths=c.lengths)),
           (ValueError, lambda: f(c.plan, c.graph, c.q, c.k, c.x, table=c.table)),
           (ValueError, lambda: f(c.plan, c.graph, c.q, c.k, c.x, lengths=c.lengths[1:], table=c.table)),
           (ValueError, lambda: f(c.plan, c.graph, c.q, c.k, c.x, lengths=c.lengths, table=c.table[1:])),
           (ValueError, lambda: f(c.plan, c.graph, c.q, c.k, c.x, lengths=c.lengths, table=c.table.t().contiguous().t())),
           (ValueError, lambda: f(c.plan, c.graph, c.q, c.k, c.x, bias=c.bias[:, :1])),
           (TypeError, lambda: f(c.plan, c.graph, c.q, c.k, c.x, bias=c.bias.double())),
           (ValueError, lambda: f(c.plan, c.graph, c.q, c.k, c.x, out=torch.empty(c.n, 3, device="cuda"))),
           (ValueError, lambda: f(c.plan, c.graph, c.q.t().contiguous().t(), c.k, c.x)),
           (ValueError, lambda: f(c.plan, c.graph, c.q[:1].expand(c.n, -1), c.k, c.x)),
           (TypeError, lambda: b(c.plan, c.graph, c.gout, c.q, c.k, c.x, None, **ok)),
           (ValueError, lambda: b(c.plan, c.graph, c.gout[:, 1:], c.q, c.k, c.x, lse, **ok)),
           (ValueError, lambda: b(c.plan, c.graph, c.gout, c.q, c.k, c.x, lse[1:], **ok)),
           (TypeError, lambda: cg().cgtp_attn_edges_backward(e.plan, e.graph, e.gout, e.q, e.k, e.x, None)),
           (ValueError, lambda: cg().cgtp_attn_edges_forward(e.plan, e.graph, e.q, e.k, e.x[1:]))]
    for kind, call in bad:
        with pytest.raises(kind):
            call()
    plain = cg().AttentionPlan(c.qk, c.v, c.heads)
    for call in (lambda: f(plain, c.graph, c.q, c.k, c.x, **ok),
                 lambda: cg().cgtp_attn_edges_backward(plain, e.graph, e.gout, e.q, e.k, e.x, torch.zeros(e.e, e.heads, device="cuda"), lengths=e.lengths)):
        with pytest.raises(ValueError):
            call()
    s = Case(SHAPES[0], "bf16s", "usual", seed=22, edges=True)
    with pytest.raises(cg().CgtpError):
        cg().cgtp_attn_edges_forward(s.plan, s.graph, s.q, s.k, s.x)
    # after all of that the calls still work
    c.check(["fwd", "bwd"])


def test_the_workspace_is_checked():
    import ctypes
    c = Case(SHAPES[0], "f32", "mixed", seed=23)
    L = cg().lib()
    need = c.plan.workspace_bytes(c.graph, "forward")
    assert need > 0 and c.plan.workspace_bytes(c.graph, "backward") > 0
    out, lse = torch.empty(c.n, c.plan.out_dim, device="cuda"), torch.empty(c.n, c.heads, device="cuda")
    ws = torch.empty(need + 16, dtype=torch.uint8, device="cuda")
    p = lambda t: ctypes.c_void_p(t.data_ptr())  # noqa: E731

    def call(at, size):
        return L.cgtp_attn_forward(c.plan.handle, c.graph.handle, p(c.q), 0, p(c.k), 0, p(c.x), 0, None, None, None, p(out), 0, p(lse),
                                   ctypes.c_void_p(at), size, None)

    torch.cuda.synchronize()
    assert call(ws.data_ptr(), need - 1) == cg().CGTP_EINVAL and call(None, need) == cg().CGTP_EINVAL
    assert call(ws.data_ptr() + 8, need) == cg().CGTP_EINVAL
    assert call(ws.data_ptr(), need) == cg().CGTP_OK
    torch.cuda.synchronize()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_attention_on_the_weights_of_a_convolution(dtype):
    """As a model runs them: attention of the receivers over their edges, the convolution with the weighed rows, and all
    the way back."""
    import oracle.conv as oconv
    import oracle.irreps as oirr
    from clebsch_gordan_tensor_racah_gb300 import workloads as wl
    spec = wl.SPECS["tiny"]
    op = oirr.make_plan(spec["in1"], spec["in2"], spec["out"], "uvu")
    w = wl.make("tiny", op.w_numel, seed=3)
    c = cg()
    plan = c.Plan(spec["in1"], spec["in2"], spec["out"], "uvu", dtype)
    heads = 2
    att = c.AttentionPlan("4x0e", c.attention_rows(plan, heads), heads, dtype=dtype, borders=c.attention_borders(8, 1.0, 5.0))
    assert att.out_dim == plan.w_numel
    rng = np.random.default_rng(4)
    t = lambda a, d=dtype: torch.from_numpy(np.ascontiguousarray(a)).cuda().to(d)  # noqa: E731
    g = c.Graph(t(w["rowptr"], torch.int32), t(w["col"], torch.int32), w["N"])
    E = g.E
    x, Y, W = t(w["x"]), t(w["Y"]), t(w["W"])
    q, k = t(rng.standard_normal((w["N"], 8))), t(rng.standard_normal((w["N"], 8)))
    lengths, table = t(rng.uniform(0, 6, E), torch.float32), t(rng.standard_normal((8, heads)), torch.float32)
    Wa, alpha = c.cgtp_attn_edges_forward(att, g, q, k, W, lengths=lengths, table=table)
    out = c.cgtp_conv_forward(plan, g, x, Y, Wa)
    # the oracle on the same (rounded) inputs
    dst = np.repeat(np.arange(w["N"]), np.diff(w["rowptr"]))
    b = _num(table)[oat.buckets(lengths.cpu().numpy(), np.float32(c.attention_borders(8, 1.0, 5.0)))]
    z, _ = oat.logits(_num(q), _num(k), "4x0e", heads, heads, 0.5, dst, w["col"], b)
    a, _ = oat.softmax(z, dst, w["N"])
    wide = oat.weighed(a, oat.spread(_num(W), c.attention_rows(plan, heads), heads, heads))
    Wr = oat.gather_back(wide, c.attention_rows(plan, heads), heads, tuple(W.shape))
    # the weighed rows: 16 roundings and an exponential of a logit below 16, stored with half a step
    assert (np.abs(_num(Wa) - Wr) <= (512 * 2.0 ** -24 + (2.0 ** -8 if dtype == torch.bfloat16 else 0)) * np.abs(Wr) + 1e-37).all()
    ref = oconv.conv_uvu_forward(op, _num(x), _num(Y), _num(Wa), w["rowptr"], w["col"])
    assert np.abs(_num(out) - ref).max() <= 1e-4 * np.abs(ref).max()   # the library's bound for a convolution
    # backward: gout -> gW' -> gW, gq, gk, gtable
    gout = t(rng.standard_normal(ref.shape))
    gWa = c.cgtp_conv_backward(plan, g, gout, x, Y, Wa)[2]
    gq, gk, gw, gtable, _ = c.cgtp_attn_edges_backward(att, g, gWa, q, k, W, alpha, lengths=lengths)
    rWa = oconv.conv_uvu_backward(op, _num(gout), _num(x), _num(Y), _num(Wa), w["rowptr"], w["col"])[2]
    rows = c.attention_rows(plan, heads)
    ge, we = oat.spread(rWa, rows, heads, heads), oat.spread(_num(W), rows, heads, heads)
    ds = oat.logit_gradient(a, (ge * we).sum(2), dst, w["N"])
    kh, qh = oat.spread(_num(k), "4x0e", heads, heads)[w["col"]], oat.spread(_num(q), "4x0e", heads, heads)[dst]
    want = (oat.gather_back(oat.receive(0.5 * ds[:, :, None] * kh, dst, w["N"]), "4x0e", heads, tuple(q.shape)),
            oat.gather_back(oat.receive(0.5 * ds[:, :, None] * qh, w["col"], w["N"]), "4x0e", heads, tuple(k.shape)),
            oat.gather_back(oat.weighed(a, ge), rows, heads, tuple(W.shape)), oat.receive(
                ds, oat.buckets(lengths.cpu().numpy(), np.float32(c.attention_borders(8, 1.0, 5.0))), 8))
    for got, ref in zip((gq, gk, gw, gtable), want):
        assert np.abs(_num(got) - ref).max() <= 1e-4 * np.abs(ref).max()


@pytest.mark.parametrize("hubs", [False, True])
@pytest.mark.parametrize("shape,kind", [(("16x0e", "4x0e+4x1o", 4, 4), "f32"), (("8x0e", "8x0e+8x1o", 4, 4), "bf16s"),
                                        (("8x0e+8x1o", "8x0e+8x1o+8x2e", 2, 2), "bf16"), (("4x0e", "4x0e", 8, 2), "f32"),
                                        (("3x0e", "1x1o", 2, 1), "f32"), (("4x0e", "2x0e", 3, 3), "f64")], ids=str)
def test_many_sources_of_few_edges(shape, kind, hubs):
    """Enough rows of both sides for one warp each, sources side by side; with hubs, whose rows are cut, and rows of more
    edges than a warp holds at once, on both sides."""
    rng = np.random.default_rng(24)
    deg = rng.poisson(14, 3000)
    deg[::50] = 0
    if hubs:
        deg[7], deg[8], deg[2999] = 700, 64, 90
    c = Case(shape, kind, deg, m=60000, seed=24)
    if hubs:
        c.col[100:900], c.col[1000:1060], c.col[2000:2050] = 59999, 5, 6
    c.col[3000:3012] = 7
    c.graph = cg().Graph(_dev(c.rowptr, torch.int32), _dev(c.col, torch.int32), c.n, n_src=c.m)
    c.check(["fwd", "bwd"])
    first = [t.clone() for t in c.run("bwd")]
    assert all(torch.equal(a, b) for a, b in zip(first, c.run("bwd")))


@pytest.mark.parametrize("edges", [False, True])
def test_the_largest_tables(edges):
    ops = ["efwd", "ebwd"] if edges else ["fwd", "bwd"]
    for heads, borders, kind in ((33, 446, "f64"), (64, 511, "f32"), (32, 511, "f64")):
        Case(("2x0e", "2x0e", heads, heads), kind, "mixed", n=12, borders=borders, seed=25, edges=edges).check(ops)
    c = Case(("2x0e", "2x0e", 33, 33), "f64", "mixed", n=12, borders=447, seed=25, edges=edges)
    c.check(ops[:1])
    with pytest.raises(cg().CgtpError, match="446 borders"):
        c.run(ops[1])


def test_rows_behind_the_first_four_gigabytes():
    """Sources at the end of tables of 5 GB give what the same sources give in tables of their own."""
    rng = np.random.default_rng(26)
    n, m, near = 40, 300000, 700
    deg = rng.poisson(20, n)
    col = rng.integers(m - near, m, deg.sum())
    c = Case(("16x0e", "1024x0e", 4, 4), "f32", deg, m=near, borders=0, seed=26)
    big = lambda t: torch.cat([torch.full((m - near, t.shape[1]), float("nan"), device="cuda"), t])  # noqa: E731
    rowptr = _dev(c.rowptr, torch.int32)
    small = cg().Graph(rowptr, _dev(col - (m - near), torch.int32), n, n_src=near)
    large = cg().Graph(rowptr, _dev(col, torch.int32), n, n_src=m)
    k, v = big(c.k), big(c.x)
    assert v.numel() * 4 > 2 ** 32
    out, lse = cg().cgtp_attn_forward(c.plan, large, c.q, k, v)
    want, wlse = cg().cgtp_attn_forward(c.plan, small, c.q, c.k, c.x)
    assert torch.equal(out, want) and torch.equal(lse, wlse)
    got = cg().cgtp_attn_backward(c.plan, large, c.gout, c.q, k, v, lse)
    ref = cg().cgtp_attn_backward(c.plan, small, c.gout, c.q, c.k, c.x, wlse)
    assert torch.equal(got[0], ref[0])
    for a, b in zip(got[1:3], ref[1:3]):
        # sums over a source's edges, at most a dozen, whose order may differ
        assert (a[:m - near] == 0).all() and torch.allclose(a[m - near:], b, rtol=0, atol=16 * 2.0 ** -24 * float(b.abs().max()))


def test_edge_rows_behind_the_first_two_billion_elements():
    n, deg, dv = 4096, 130, 1024
    c = Case(("4x0e", f"{dv}x0e", 4, 4), "f32", [2], m=64, borders=0, seed=27, edges=True)
    col = torch.randint(0, 64, (n * deg,), dtype=torch.int32, device="cuda")
    g = cg().Graph(torch.arange(0, n * deg + 1, deg, dtype=torch.int32, device="cuda"), col, n, n_src=64)
    q = torch.randn(n, 16, device="cuda")
    w = torch.randn(n * deg, 4 * dv, device="cuda")
    assert w.numel() > 2 ** 31
    out, alpha = cg().cgtp_attn_edges_forward(c.plan, g, q, c.k, w)
    tail = slice(-500, None)
    wide = lambda a: a[tail].repeat_interleave(dv, dim=1)  # noqa: E731
    assert torch.allclose(alpha.view(n, deg, 4).sum(1), torch.ones(n, 4, device="cuda"), rtol=0, atol=deg * 2.0 ** -24)
    assert torch.equal(out[tail], wide(alpha) * w[tail])
    gq, gk, gw, _, ds = cg().cgtp_attn_edges_backward(c.plan, g, out, q, c.k, w, alpha, need_gbias=True)
    assert torch.equal(gw[tail], wide(alpha) * out[tail])
    # the last receiver's gradient, from the formula in 64 bits: dv + deg + 12 roundings of sums of magnitudes
    a, dp = alpha[-deg:].double(), (out[-deg:].double() * w[-deg:].double()).view(deg, 4, dv).sum(2)
    mag = (out[-deg:].double() * w[-deg:].double()).abs().view(deg, 4, dv).sum(2)
    want = a * (dp - (a * dp).sum(0))
    assert ((ds[-deg:] - want).abs() <= (dv + deg + 12) * 2.0 ** -24 * a * (mag + (a * mag).sum(0))).all()
