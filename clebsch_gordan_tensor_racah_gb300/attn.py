"""Binding of include/cgtp_attn.h: attention along a graph's edges, of values and of per-edge weight rows.

Argument marshalling only, like the rest of the package: the computation runs in the CUDA
kernels of ``libcgtp.so``.  The calls go through ``_binding`` (csrc/binding.cpp), which checks its arguments in
native code; an argument that does not fit comes back to the checks here, which say what is wrong.
"""

import ctypes
import math

import torch

from . import _binding
from . import CGTP_BF16, CGTP_F32, CGTP_F64, _check, lib
from .train import _current, _dtype, _explain_device, _explain_rows, _explain_vector, _here, _on, _result

_binding.connect_attn(*(ctypes.cast(getattr(lib(), f), ctypes.c_void_p).value for f in (
    "cgtp_attn_workspace", "cgtp_attn_forward", "cgtp_attn_backward", "cgtp_attn_edges_forward",
    "cgtp_attn_edges_backward")))

ATTN_STORAGE = 1


def _dim(irreps):
    """Elements of a row; 1 where the library is to say what is wrong with the string."""
    try:
        blocks = [t.split("x") if "x" in t else ("1", t) for t in irreps.replace(" ", "").split("+")]
        return max(1, sum(int(mul) * (2 * int(ir[:-1]) + 1) for mul, ir in blocks))
    except ValueError:
        return 1


def attention_borders(buckets, near, far):
    """Borders of ``buckets`` distance buckets: half of them even up to ``near``, the others even in the logarithm
    from there to ``far``; the last bucket holds everything beyond."""
    if buckets < 2 or not 0 < near < far < math.inf:
        raise ValueError("at least two buckets and 0 < near < far are needed")
    half = buckets // 2
    rest = buckets - half
    return [near * (i + 1) / half for i in range(half)] + [near * (far / near) ** (i / (rest - 1)) for i in range(1, rest)]


def attention_rows(plan, heads):
    """irreps_v of an AttentionPlan for the weight rows W [E, w_numel] of a uvu convolution plan."""
    if plan.mode != "uvu":
        raise ValueError("weight rows of a uvu plan are needed")
    muls = [plan.path(p)[0][3] for p in range(plan.n_paths)]
    if any(m % heads for m in muls):
        raise ValueError(f"{heads} heads do not divide the channels of every path: {sorted(set(muls))}")
    return "+".join(f"{m // heads}x0e" for m in muls)


class AttentionPlan:
    """cgtp_attn_create: attention along the edges of a Graph.

    ``irreps_qk`` and ``irreps_v`` describe ONE head; rows hold the heads side by side in every block.  kv_heads
    (default: heads) sets of keys and values are shared by the heads.  scale: factor of the inner products (default:
    1 / sqrt(elements of a head)).  borders: ascending distances between the buckets of the bias table.

    ``dtype`` is the type of q, k, v, gout and edge rows; ``result_dtype`` of out and the gradients (``storage``, bfloat16
    only, keeps them in bfloat16); ``param_dtype`` of lengths, table, bias, lse, alpha and their gradients.
    """

    def __init__(self, irreps_qk, irreps_v, heads, kv_heads=None, dtype=None, storage=False, scale=None, borders=None):
        self.dtype = dtype or torch.float32
        code = _dtype(self.dtype, "dtype", (CGTP_F32, CGTP_F64, CGTP_BF16))
        self.heads, self.kv_heads = int(heads), int(heads if kv_heads is None else kv_heads)
        borders = [] if borders is None else [float(b) for b in borders]
        h = ctypes.c_void_p()
        args = (irreps_qk.encode(), irreps_v.encode(), self.heads, self.kv_heads, code, ATTN_STORAGE if storage else 0)
        if scale is None:
            scale = _dim(irreps_qk) ** -0.5
        _check(lib().cgtp_attn_create(ctypes.byref(h), *args, float(scale), len(borders),
                                      (ctypes.c_double * max(len(borders), 1))(*borders)))
        self._h = h
        self.device = _here()
        self.scale = float(scale)
        dk, dv = ctypes.c_int64(), ctypes.c_int64()
        _check(lib().cgtp_attn_info(h, ctypes.byref(dk), ctypes.byref(dv)))
        self.dim_qk, self.dim_v = dk.value, dv.value
        self.q_dim, self.k_dim = self.heads * self.dim_qk, self.kv_heads * self.dim_qk
        self.v_dim, self.out_dim = self.kv_heads * self.dim_v, self.heads * self.dim_v
        self.buckets = len(borders) + 1 if borders else 0
        half = self.dtype == torch.bfloat16
        self.param_dtype = torch.float32 if half else self.dtype
        self.result_dtype = self.dtype if storage else self.param_dtype
        types = [_dtype(t, "dtype", (CGTP_F32, CGTP_F64, CGTP_BF16)) for t in (self.dtype, self.result_dtype, self.param_dtype)]
        self._native = (h.value, *types, self.heads, self.kv_heads, self.dim_qk, self.dim_v, self.buckets, self.device.index)

    @property
    def handle(self):
        return self._h

    def device_bytes(self):
        """Device memory the library holds for this plan (cgtp_attn_device_bytes)."""
        nb = ctypes.c_int64()
        _check(lib().cgtp_attn_device_bytes(self._h, ctypes.byref(nb)))
        return nb.value

    def workspace_bytes(self, graph, call):
        """cgtp_attn_workspace for "forward", "backward", "edges_forward" or "edges_backward"."""
        nb = ctypes.c_int64()
        _check(lib().cgtp_attn_workspace(self._h, graph.handle, ("forward", "backward", "edges_forward", "edges_backward").index(call),
                                         ctypes.byref(nb)))
        return nb.value

    def explain(self, graph, nodes=(), edges=(), lengths=None, table=None, grids=()):
        """Raises what is wrong with a call's arguments: (name, tensor, dtype, rows, width), required unless None is in `grids`."""
        _explain_device(self.device)
        if graph.device != self.device:
            raise ValueError(f"the graph is on {graph.device}, the plan on {self.device}")
        for name, t, dtype, n, width in (*nodes, *edges):
            if t is None and n > 0:
                raise TypeError(f"{name} must be a CUDA tensor")
            _explain_rows(name, t, dtype, n, width, self.device)
        _explain_vector("lengths", lengths, self.param_dtype, graph.E, self.device)
        if table is not None and not self.buckets:
            raise ValueError("a table of biases needs a plan with borders")
        for name, t, n, width in (("table", table, self.buckets, self.heads), *grids):
            if t is None:
                continue
            _explain_rows(name, t, self.param_dtype, n, width, self.device)
            if not t.is_contiguous():
                raise ValueError(f"{name} must be contiguous")

    def __del__(self):
        h = getattr(self, "_h", None)
        if h is not None and h.value and lib is not None:
            lib().cgtp_attn_destroy(h)
            self._h = None


def _qk(plan, graph, q, k):
    return ("q", q, plan.dtype, graph.N, plan.q_dim), ("k", k, plan.dtype, graph.n_src, plan.k_dim)


def _both(lengths, table):
    if (lengths is None) != (table is None):
        raise ValueError("lengths and table: both or neither")


def cgtp_attn_forward(plan, graph, q, k, v, lengths=None, table=None, bias=None, out=None, stream=None):
    """(out, lse): attention of the graph's receivers to the states of their sources.

    q [N, q_dim], k [n_src, k_dim], v [n_src, v_dim] (column ranges of wider rows are fine) -> out [N, out_dim];
    lse [N, heads] is kept for the backward.  lengths [E] with table [buckets, heads]: bias by distance buckets.  bias
    [E, heads]: added to the logits; -inf leaves an edge out.  out: optional preallocated result."""
    if stream is not None:
        return _on(stream, cgtp_attn_forward, plan, graph, q, k, v, lengths, table, bias, out)

    def explain():
        plan.explain(graph, (*_qk(plan, graph, q, k), ("v", v, plan.dtype, graph.n_src, plan.v_dim)), (), lengths, table,
                     (("bias", bias, graph.E, plan.heads),))
        _explain_rows("out", out, plan.result_dtype, graph.N, plan.out_dim, plan.device)
        _both(lengths, table)

    r = _binding.attn_forward(plan._native, graph._native, q, k, v, lengths, table, bias, out, _current(q))
    return r if type(r) is tuple else _result(r, explain)


def cgtp_attn_backward(plan, graph, gout, q, k, v, lse, lengths=None, table=None, bias=None, need_gbias=False, stream=None):
    """(gq, gk, gv, gtable, gbias) for the gradient gout of the forward's first result.

    gtable is None without a table.  gbias [E, heads], the gradient of the logits, is None unless need_gbias."""
    if stream is not None:
        return _on(stream, cgtp_attn_backward, plan, graph, gout, q, k, v, lse, lengths, table, bias, need_gbias)

    def explain():
        plan.explain(graph, (("gout", gout, plan.dtype, graph.N, plan.out_dim), *_qk(plan, graph, q, k),
                             ("v", v, plan.dtype, graph.n_src, plan.v_dim), ("lse", lse, plan.param_dtype, graph.N, plan.heads)), (),
                     lengths, table, (("lse", lse, graph.N, plan.heads), ("bias", bias, graph.E, plan.heads)))
        _both(lengths, table)

    r = _binding.attn_backward(plan._native, graph._native, gout, q, k, v, lse, lengths, table, bias, need_gbias, _current(q))
    return r if type(r) is tuple else _result(r, explain)


def cgtp_attn_edges_forward(plan, graph, q, k, w, lengths=None, table=None, bias=None, out=None, stream=None):
    """(w', alpha): the attention's weights alpha [E, heads], and the edges' rows w [E, out_dim] times them.

    With irreps_v = attention_rows(conv_plan, heads), w' takes the place of W in cgtp_conv_forward: every message is
    weighed by its edge's attention, head by head.  out: optional preallocated w'."""
    if stream is not None:
        return _on(stream, cgtp_attn_edges_forward, plan, graph, q, k, w, lengths, table, bias, out)

    def explain():
        plan.explain(graph, _qk(plan, graph, q, k), (("w", w, plan.dtype, graph.E, plan.out_dim),), lengths, table,
                     (("bias", bias, graph.E, plan.heads),))
        _explain_rows("out", out, plan.dtype, graph.E, plan.out_dim, plan.device)
        _both(lengths, table)

    r = _binding.attn_edges_forward(plan._native, graph._native, q, k, w, lengths, table, bias, out, _current(q))
    return r if type(r) is tuple else _result(r, explain)


def cgtp_attn_edges_backward(plan, graph, gout, q, k, w, alpha, lengths=None, need_gbias=False, gw=None, stream=None):
    """(gq, gk, gw, gtable, gbias) for the gradient gout of w' (param_dtype, as convolutions give it).

    gtable is None without lengths.  gbias as in cgtp_attn_backward.  gw: optional preallocated gradient of w."""
    if stream is not None:
        return _on(stream, cgtp_attn_edges_backward, plan, graph, gout, q, k, w, alpha, lengths, need_gbias, gw)

    def explain():
        plan.explain(graph, _qk(plan, graph, q, k), (("gout", gout, plan.param_dtype, graph.E, plan.out_dim), ("w", w, plan.dtype, graph.E, plan.out_dim),
                                                     ("alpha", alpha, plan.param_dtype, graph.E, plan.heads)), lengths, None,
                     (("alpha", alpha, graph.E, plan.heads),))
        _explain_rows("gw", gw, plan.param_dtype, graph.E, plan.out_dim, plan.device)
        if lengths is not None and not plan.buckets:
            raise ValueError("lengths need a plan with borders")
        if alpha is None:
            raise TypeError("alpha must be a CUDA tensor")

    r = _binding.attn_edges_backward(plan._native, graph._native, gout, q, k, w, alpha, lengths, need_gbias, gw, _current(q))
    return r if type(r) is tuple else _result(r, explain)
