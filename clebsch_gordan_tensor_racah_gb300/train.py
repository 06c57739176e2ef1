"""Binding of include/cgtp_train.h: the gated residual norm of a block and the AdamW step.

Argument marshalling only, like the rest of the package: the computation runs in the CUDA
kernels of ``libcgtp.so``.
"""

import ctypes
import operator

import torch

from . import CGTP_BF16, CGTP_F32, CGTP_F64, _check, _ptr, lib

_Tensor = torch.Tensor
_numel, _data_ptr, _is_contiguous = _Tensor.numel, _Tensor.data_ptr, _Tensor.is_contiguous
_dtype_of, _is_cuda = operator.attrgetter("dtype"), operator.attrgetter("is_cuda")

ACTS = {"none": 0, "identity": 1, "sigmoid": 2, "silu": 3}
RESNORM_POST, RESNORM_PRE, RESNORM_STORAGE = 1, 2, 4
STATES = {"full": 0, "f32": 0, "8bit": 1}
STATE_BLOCK = 128


def _dtype(dtype, name, allowed):
    code = {torch.float32: CGTP_F32, torch.float64: CGTP_F64, torch.bfloat16: CGTP_BF16}.get(dtype)
    if code is None or code not in allowed:
        raise TypeError(f"{name}: unsupported element type {dtype}")
    return code


def _rows(t, name, dtype, n, width):
    """Device pointer and row distance of a row tensor [n, width] (a column range of wider rows is fine)."""
    if t is None:
        return None, 0
    try:
        (rows, cols), (ld, inner) = t.shape, t.stride()
    except (AttributeError, TypeError, ValueError):
        raise _misfit(t, name, dtype, n, width) from None
    if t.dtype is dtype and t.is_cuda and rows == n and cols == width and (inner == 1 or width == 1 or n == 0):
        if n <= 1:
            return t.data_ptr(), 0
        if ld >= width:
            return t.data_ptr(), ld
    raise _misfit(t, name, dtype, n, width)


def _misfit(t, name, dtype, n, width):
    """What is wrong with a row tensor that _rows refused."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        return TypeError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        return TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != (n, width):
        return ValueError(f"{name} must have shape ({n}, {width}), got {tuple(t.shape)}")
    return ValueError(f"{name}: elements of a row must be contiguous and rows must not overlap")


def _vector(t, name, dtype, width):
    """Device pointer of a contiguous tensor [width] or None."""
    if t is None:
        return None
    if isinstance(t, torch.Tensor) and t.dtype is dtype and t.is_cuda and t.shape == (width,) and t.is_contiguous():
        return t.data_ptr()
    if isinstance(t, torch.Tensor) and t.shape != (width,):
        raise ValueError(f"{name} must have shape ({width},), got {tuple(t.shape)}")
    return _ptr(t, name, dtype)


def _current(stream, device):
    """cudaStream_t of `stream`, or of the device's current stream."""
    return stream.cuda_stream if stream is not None else torch._C._cuda_getCurrentRawStream(device.index)


class ResNormPlan:
    """cgtp_resnorm_create: the norms, gate and residual around a block of irreps features.

    ``stream_dtype`` is the type of h, out, gout, gh; ``in_dtype`` of z, q, gy (what comes from a
    product); ``out_dtype`` of y, gz, gq (what goes to one); ``param_dtype`` of post, scale, pre and
    their gradients.  ``storage`` (bfloat16 only) keeps every row tensor in bfloat16.
    """

    def __init__(self, irreps, dtype=None, storage=False, act="none", pre_norm=True, post_norm=True, alpha=1.0,
                 eps=1e-5):
        dtype = dtype or torch.float32
        code = _dtype(dtype, "dtype", (CGTP_F32, CGTP_F64, CGTP_BF16))
        if act not in ACTS:
            raise ValueError(f"act must be one of {sorted(ACTS)}")
        flags = (RESNORM_POST if post_norm else 0) | (RESNORM_PRE if pre_norm else 0) | (RESNORM_STORAGE if storage else 0)
        h = ctypes.c_void_p()
        _check(lib().cgtp_resnorm_create(ctypes.byref(h), irreps.encode(), code, flags, ACTS[act], float(alpha), float(eps)))
        self._h = h
        dim, channels, blocks = ctypes.c_int64(), ctypes.c_int64(), ctypes.c_int()
        _check(lib().cgtp_resnorm_info(h, ctypes.byref(dim), ctypes.byref(channels), ctypes.byref(blocks)))
        self.dim, self.channels, self.n_blocks = dim.value, channels.value, blocks.value
        self.act, self.pre_norm, self.post_norm = act, bool(pre_norm), bool(post_norm)
        half = dtype == torch.bfloat16
        self.out_dtype = dtype
        self.stream_dtype = self.in_dtype = torch.float32 if half and not storage else dtype
        self.param_dtype = torch.float32 if half else dtype

    @property
    def handle(self):
        return self._h

    def device_bytes(self):
        """Device memory the library holds for this plan (cgtp_resnorm_device_bytes)."""
        nb = ctypes.c_int64()
        _check(lib().cgtp_resnorm_device_bytes(self._h, ctypes.byref(nb)))
        return nb.value

    def __del__(self):
        h = getattr(self, "_h", None)
        if h is not None and h.value:
            lib().cgtp_resnorm_destroy(h)
            self._h = None


def cgtp_resnorm_forward(plan, h, z=None, q=None, post=None, scale=None, pre=None, out=None, y=None, stream=None):
    """(out, y) with out = alpha h + scale a(q) post rms(z) z and y = pre rms(out) out.

    z = None: y is the norm of h and the first result is h itself.  h = None: no residual.  y is
    None for plans with pre_norm = False.  Row tensors [N, dim] (q: [N, channels]) may be column
    ranges of wider ones."""
    ref = h if h is not None else z
    if ref is None:
        raise ValueError("h or z must be given")
    n, dim, chan, device = ref.shape[0], plan.dim, plan.channels, ref.device
    st, it, ot, pt, empty = plan.stream_dtype, plan.in_dtype, plan.out_dtype, plan.param_dtype, torch.empty
    # operands are checked before results are allocated
    hp, zp, qp = _rows(h, "h", st, n, dim), _rows(z, "z", it, n, dim), _rows(q, "q", it, n, chan)
    if z is not None and out is None:
        out = empty((n, dim), dtype=st, device=device)
    if plan.pre_norm and y is None:
        y = empty((n, dim), dtype=ot, device=device)
    status = lib().cgtp_resnorm_forward(
        plan.handle, n, *hp, *zp, *qp, _vector(post, "post", pt, chan), _vector(scale, "scale", pt, chan),
        _vector(pre, "pre", pt, chan), *_rows(out, "out", st, n, dim), *_rows(y, "y", ot, n, dim), _current(stream, device))
    if status:
        _check(status)
    return (out if z is not None else h), y


def cgtp_resnorm_backward(plan, gout, gy, x, z=None, q=None, post=None, scale=None, pre=None, need_gh=True,
                          outs=None, stream=None):
    """(gh, gz, gq, gpost, gscale, gpre) for the gradients gout (or None) and gy of the results.

    x is what the forward returned first.  gz and gq are None without z or a gate; gpost, gscale
    and gpre are None where that factor is.  outs: optional preallocated results in that order
    (column ranges of wider rows are fine for gh, gz and gq)."""
    ref = gout if gout is not None else gy
    if ref is None:
        raise ValueError("gout or gy must be given")
    n, dim, chan, device = ref.shape[0], plan.dim, plan.channels, ref.device
    st, it, ot, pt, empty = plan.stream_dtype, plan.in_dtype, plan.out_dtype, plan.param_dtype, torch.empty
    gp, yp, xp = _rows(gout, "gout", st, n, dim), _rows(gy, "gy", it, n, dim), _rows(x, "x", st, n, dim)
    zp, qp = _rows(z, "z", it, n, dim), _rows(q, "q", it, n, chan)
    if outs is not None:
        gh, gz, gq, gpost, gscale, gpre = outs
        sums = _vector(gpost, "gpost", pt, chan), _vector(gscale, "gscale", pt, chan), _vector(gpre, "gpre", pt, chan)
    else:
        gh = empty((n, dim), dtype=st, device=device) if need_gh else None
        gz = empty((n, dim), dtype=ot, device=device) if z is not None else None
        gq = empty((n, chan), dtype=ot, device=device) if z is not None and plan.act != "none" else None
        gpost = None if post is None else empty(chan, dtype=pt, device=device)
        gscale = None if scale is None else empty(chan, dtype=pt, device=device)
        gpre = None if pre is None else empty(chan, dtype=pt, device=device)
        sums = [None if g is None else g.data_ptr() for g in (gpost, gscale, gpre)]
    status = lib().cgtp_resnorm_backward(
        plan.handle, n, *gp, *yp, *xp, *zp, *qp, _vector(post, "post", pt, chan), _vector(scale, "scale", pt, chan),
        _vector(pre, "pre", pt, chan), *_rows(gh, "gh", st, n, dim), *_rows(gz, "gz", ot, n, dim),
        *_rows(gq, "gq", ot, n, chan), *sums, _current(stream, device))
    if status:
        _check(status)
    return gh, gz, gq, gpost, gscale, gpre


class AdamW:
    """cgtp_adamw_create: AdamW over tensors of ``numel`` elements each.

    state "f32" (or "full": the parameters' type) or "8bit".  decay_scale: factor of the weight
    decay for each tensor (0: not decayed)."""

    def __init__(self, numel, param_dtype=None, grad_dtype=None, state="f32", decay_scale=None):
        self.param_dtype = param_dtype or torch.float32
        self.grad_dtype = grad_dtype or self.param_dtype
        if state not in STATES:
            raise ValueError(f"state must be one of {sorted(STATES)}")
        self.numel = [int(k) for k in numel]
        self.state = "8bit" if STATES[state] else "full"
        n = len(self.numel)
        sizes = (ctypes.c_int64 * max(n, 1))(*self.numel)
        if decay_scale is not None:
            if len(decay_scale) != n:
                raise ValueError("one decay_scale per tensor")
            decay_scale = (ctypes.c_float * max(n, 1))(*decay_scale)
        h = ctypes.c_void_p()
        _check(lib().cgtp_adamw_create(ctypes.byref(h), n, sizes, decay_scale,
                                       _dtype(self.param_dtype, "param_dtype", (CGTP_F32, CGTP_F64)),
                                       _dtype(self.grad_dtype, "grad_dtype", (CGTP_F32, CGTP_F64, CGTP_BF16)),
                                       STATES[state]))
        self._h = h
        total = ctypes.c_int64()
        _check(lib().cgtp_adamw_info(h, ctypes.byref(total)))
        self.state_numel = total.value
        self._list = ctypes.c_void_p * max(n, 1)

    @property
    def handle(self):
        return self._h

    def new_state(self, device="cuda"):
        """Initial states: dict of m, v, m_exp, v_exp (the last two None unless 8-bit)."""
        eight = self.state == "8bit"
        dt = torch.uint8 if eight else self.param_dtype
        zeros = lambda k: torch.zeros(k, dtype=dt, device=device)  # noqa: E731
        return dict(m=zeros(self.state_numel), v=zeros(self.state_numel),
                    m_exp=zeros(self.state_numel // STATE_BLOCK) if eight else None,
                    v_exp=zeros(self.state_numel // STATE_BLOCK) if eight else None)

    def device_bytes(self):
        """Device memory the library holds for this optimizer (cgtp_adamw_device_bytes)."""
        nb = ctypes.c_int64()
        _check(lib().cgtp_adamw_device_bytes(self._h, ctypes.byref(nb)))
        return nb.value

    def pointers(self, tensors, name, dtype):
        """HOST array of the tensors' device pointers; their number and sizes are the optimizer's."""
        given = [t for t in tensors if t is not None]
        sizes = self.numel
        if len(given) != len(tensors):
            sizes = [k for k, t in zip(sizes, tensors) if t is not None]
        try:
            # whole lists at C speed: a step has hundreds of small tensors
            fits = (len(tensors) == len(self.numel) and list(map(_numel, given)) == sizes
                    and all(map(_is_contiguous, given)) and all(map(_is_cuda, given))
                    and (not given or set(map(_dtype_of, given)) == {dtype}))
            if fits:
                if len(given) == len(tensors):
                    return self._list(*map(_data_ptr, given))
                return self._list(*[None if t is None else t.data_ptr() for t in tensors])
        except TypeError:
            pass
        raise self._misfit(tensors, name, dtype)

    def _misfit(self, tensors, name, dtype):
        """What is wrong with a list of tensors that `pointers` refused."""
        if len(tensors) != len(self.numel):
            return ValueError(f"{name}: {len(self.numel)} tensors expected, got {len(tensors)}")
        for t, k in zip(tensors, self.numel):
            if t is None:
                continue
            if not isinstance(t, torch.Tensor) or t.dtype != dtype or not t.is_cuda:
                return TypeError(f"{name} must be {dtype} CUDA tensors")
            if t.numel() != k or not t.is_contiguous():
                return ValueError(f"{name}: a contiguous tensor of {k} elements expected, got {tuple(t.shape)}")
        return TypeError(f"{name} must be {dtype} CUDA tensors")

    def states(self, state):
        """Device pointers of m, v, m_exp, v_exp after checks of type and size."""
        n, eight = self.state_numel, self.state == "8bit"
        dt = torch.uint8 if eight else self.param_dtype
        if eight and (state["m_exp"] is None or state["v_exp"] is None):
            raise ValueError("8-bit states need m_exp and v_exp")
        blocks = n // STATE_BLOCK
        return (_vector(state["m"], "state m", dt, n), _vector(state["v"], "state v", dt, n),
                _vector(state["m_exp"], "state m_exp", dt, blocks) if eight else None,
                _vector(state["v_exp"], "state v_exp", dt, blocks) if eight else None)

    def __del__(self):
        h = getattr(self, "_h", None)
        if h is not None and h.value:
            lib().cgtp_adamw_destroy(h)
            self._h = None


def cgtp_grad_norm(opt, grads, max_norm=float("inf"), out=None, stream=None):
    """Tensor [norm of all gradients, min(1, max_norm / norm)]; None gradients count as zero."""
    found = opt.pointers(grads, "grads", opt.grad_dtype)
    if out is None:
        given = next((t for t in grads if t is not None), None)
        out = torch.empty(2, dtype=opt.param_dtype, device="cuda" if given is None else given.device)
    _check(lib().cgtp_grad_norm(opt.handle, found, float(max_norm), _vector(out, "out", opt.param_dtype, 2),
                                _current(stream, out.device)))
    return out


def cgtp_adamw_step(opt, params, grads, state, lr, betas=(0.9, 0.999), eps=1e-8, weight_decay=0.0, step=1,
                    copies=None, clip=None, seed=0, stream=None):
    """One AdamW step in place.  A None gradient skips its tensor.  copies: bfloat16 tensors (or None)
    that receive the new parameters.  clip: result of cgtp_grad_norm.  seed: rounding of 8-bit states."""
    _check(lib().cgtp_adamw_step(
        opt.handle, opt.pointers(params, "params", opt.param_dtype), opt.pointers(grads, "grads", opt.grad_dtype),
        None if copies is None else opt.pointers(copies, "copies", torch.bfloat16), *opt.states(state), float(lr),
        float(betas[0]), float(betas[1]), float(eps), float(weight_decay), int(step), int(seed) & 0xFFFFFFFFFFFFFFFF,
        _vector(clip, "clip", opt.param_dtype, 2), _current(stream, state["m"].device)))


def cgtp_adamw_state_values(opt, state, stream=None):
    """(m, v) as the FP32 values the 8-bit states stand for (the states themselves otherwise)."""
    if opt.state != "8bit":
        return state["m"], state["v"]
    m, v = (torch.empty(opt.state_numel, dtype=torch.float32, device=state[k].device) for k in ("m", "v"))
    p = opt.states(state)
    _check(lib().cgtp_adamw_state_values(opt.handle, p[0], p[1], p[2], p[3], m.data_ptr(), v.data_ptr(),
                                         _current(stream, m.device)))
    return m, v
