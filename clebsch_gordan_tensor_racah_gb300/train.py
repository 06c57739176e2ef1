"""Binding of include/cgtp_train.h: the gated residual norm of a block and the AdamW step.

Argument marshalling only, like the rest of the package: the computation runs in the CUDA
kernels of ``libcgtp.so``.  The calls of a training step go through ``_binding`` (csrc/binding.cpp),
which checks its arguments in native code; an argument that does not fit comes back to the
checks here, which say what is wrong.
"""

import ctypes

import torch

from . import _binding
from . import CGTP_BF16, CGTP_F32, CGTP_F64, _check, _ptr, lib

_binding.connect(*(ctypes.cast(getattr(lib(), f), ctypes.c_void_p).value for f in (
    "cgtp_resnorm_forward", "cgtp_resnorm_backward", "cgtp_adamw_step", "cgtp_grad_norm", "cgtp_adamw_state_values")))

ACTS = {"none": 0, "identity": 1, "sigmoid": 2, "silu": 3}
RESNORM_POST, RESNORM_PRE, RESNORM_STORAGE = 1, 2, 4
STATES = {"full": 0, "f32": 0, "8bit": 1}
STATE_BLOCK = 128


def _dtype(dtype, name, allowed):
    code = {torch.float32: CGTP_F32, torch.float64: CGTP_F64, torch.bfloat16: CGTP_BF16}.get(dtype)
    if code is None or code not in allowed:
        raise TypeError(f"{name}: unsupported element type {dtype}")
    return code


def _here():
    """The current device: the one that a plan or optimizer is made on."""
    return torch.device("cuda", torch.cuda.current_device())


def _explain_device(device):
    """Raises where calls of a plan or optimizer of `device` would be launched on another one."""
    if _here() != device:
        raise ValueError(f"the plan or optimizer is on {device}, the current device is {_here()}")


def _explain_rows(name, t, dtype, n, width, device):
    """Raises where a row tensor (or None) does not fit."""
    if t is None:
        return
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.device != device:
        raise ValueError(f"{name} must be on {device}, got {t.device}")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != (n, width):
        raise ValueError(f"{name} must have shape ({n}, {width}), got {tuple(t.shape)}")
    if (t.stride(1) != 1 and width > 1 and n > 0) or (n > 1 and t.stride(0) < width):
        raise ValueError(f"{name}: elements of a row must be contiguous and rows must not overlap")


def _explain_vector(name, t, dtype, width, device):
    """Raises where a contiguous tensor [width] (or None) does not fit."""
    if t is None:
        return
    _ptr(t, name, dtype)
    if t.device != device:
        raise ValueError(f"{name} must be on {device}, got {t.device}")
    if t.shape != (width,):
        raise ValueError(f"{name} must have shape ({width},), got {tuple(t.shape)}")


def _explain_list(name, tensors, numel, dtype, device):
    """Raises where a list of tensors (or None) does not fit the optimizer's."""
    if len(tensors) != len(numel):
        raise ValueError(f"{name}: {len(numel)} tensors expected, got {len(tensors)}")
    for t, k in zip(tensors, numel):
        if t is None:
            continue
        if not isinstance(t, torch.Tensor) or t.dtype != dtype or not t.is_cuda:
            raise TypeError(f"{name} must be {dtype} CUDA tensors")
        if t.device != device:
            raise ValueError(f"{name} must be on {device}, got {t.device}")
        if t.numel() != k or not t.is_contiguous():
            raise ValueError(f"{name}: a contiguous tensor of {k} elements expected, got {tuple(t.shape)}")


def _result(r, explain):
    """A native call's results, or its refusal as an exception."""
    if r is NotImplemented:
        explain()
        raise TypeError("arguments of unexpected types")
    if type(r) is int:
        _check(r)
    return r


def _on(stream, call, *args, **kwargs):
    """`call` with `stream` as the current one, so that its results belong to that stream."""
    with torch.cuda.stream(stream):
        return call(*args, **kwargs)


def _current(t):
    """cudaStream_t of the current stream of a tensor's device."""
    return torch._C._cuda_getCurrentRawStream(t.device.index) if getattr(t, "is_cuda", False) else 0


class ResNormPlan:
    """cgtp_resnorm_create: the norms, gate and residual around a block of irreps features.

    ``stream_dtype`` is the type of h, out, gout, gh; ``in_dtype`` of z, q, gy (what comes from a
    product); ``out_dtype`` of y, gz, gq (what goes to one); ``param_dtype`` of post, scale, pre and
    their gradients.  ``storage`` (bfloat16 only) keeps every row tensor in bfloat16.

    The plan owns the partial sums of the parameter gradients: its backwards must not overlap on the GPU.  Give
    each stream that runs them at the same time a plan of its own.
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
        self.device = _here()
        dim, channels, blocks = ctypes.c_int64(), ctypes.c_int64(), ctypes.c_int()
        _check(lib().cgtp_resnorm_info(h, ctypes.byref(dim), ctypes.byref(channels), ctypes.byref(blocks)))
        self.dim, self.channels, self.n_blocks = dim.value, channels.value, blocks.value
        self.act, self.pre_norm, self.post_norm = act, bool(pre_norm), bool(post_norm)
        half = dtype == torch.bfloat16
        self.out_dtype = dtype
        self.stream_dtype = self.in_dtype = torch.float32 if half and not storage else dtype
        self.param_dtype = torch.float32 if half else dtype
        types = [_dtype(t, "dtype", (CGTP_F32, CGTP_F64, CGTP_BF16))
                 for t in (self.stream_dtype, self.in_dtype, self.out_dtype, self.param_dtype)]
        self._native = (h.value, *types, self.dim, self.channels, int(self.pre_norm), int(act != "none"), self.device.index)

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
        if h is not None and h.value and lib is not None:
            lib().cgtp_resnorm_destroy(h)
            self._h = None


def cgtp_resnorm_forward(plan, h, z=None, q=None, post=None, scale=None, pre=None, out=None, y=None, stream=None):
    """(out, y) with out = alpha h + scale a(q) post rms(z) z and y = pre rms(out) out.

    z = None: y is the norm of h and the first result is h itself.  h = None: no residual.  y is
    None for plans with pre_norm = False.  Row tensors [N, dim] (q: [N, channels]) may be column
    ranges of wider ones."""
    if stream is not None:
        return _on(stream, cgtp_resnorm_forward, plan, h, z, q, post, scale, pre, out, y)
    ref = h if h is not None else z
    if ref is None:
        raise ValueError("h or z must be given")

    def explain():
        _explain_device(plan.device)
        n, dim, chan = ref.shape[0], plan.dim, plan.channels
        for name, t, dtype, width in (("h", h, plan.stream_dtype, dim), ("z", z, plan.in_dtype, dim), ("q", q, plan.in_dtype, chan),
                                      ("out", out, plan.stream_dtype, dim), ("y", y, plan.out_dtype, dim)):
            _explain_rows(name, t, dtype, n, width, plan.device)
        for name, t in (("post", post), ("scale", scale), ("pre", pre)):
            _explain_vector(name, t, plan.param_dtype, chan, plan.device)

    r = _binding.resnorm_forward(plan._native, h, z, q, post, scale, pre, out, y, _current(ref))
    return r if type(r) is tuple else _result(r, explain)


def cgtp_resnorm_backward(plan, gout, gy, x, z=None, q=None, post=None, scale=None, pre=None, need_gh=True,
                          outs=None, stream=None):
    """(gh, gz, gq, gpost, gscale, gpre) for the gradients gout (or None) and gy of the results.

    Without z the stream is h itself and alpha does not enter gh.  x is what the forward returned first.  gz and gq are None without z or a gate; gpost, gscale
    and gpre are None where that factor is.  outs: optional preallocated results in that order
    (column ranges of wider rows are fine for gh, gz and gq)."""
    if stream is not None:
        return _on(stream, cgtp_resnorm_backward, plan, gout, gy, x, z, q, post, scale, pre, need_gh, outs)
    ref = gout if gout is not None else gy
    if ref is None:
        raise ValueError("gout or gy must be given")
    outs = None if outs is None else tuple(outs)

    def explain():
        _explain_device(plan.device)
        n, dim, chan = ref.shape[0], plan.dim, plan.channels
        gh, gz, gq, *sums = outs or (None,) * 6
        for name, t, dtype, width in (("gout", gout, plan.stream_dtype, dim), ("gy", gy, plan.in_dtype, dim),
                                      ("x", x, plan.stream_dtype, dim), ("z", z, plan.in_dtype, dim), ("q", q, plan.in_dtype, chan),
                                      ("gh", gh, plan.stream_dtype, dim), ("gz", gz, plan.out_dtype, dim), ("gq", gq, plan.out_dtype, chan)):
            _explain_rows(name, t, dtype, n, width, plan.device)
        for name, t in zip(("post", "scale", "pre", "gpost", "gscale", "gpre"), (post, scale, pre, *sums)):
            _explain_vector(name, t, plan.param_dtype, chan, plan.device)

    r = _binding.resnorm_backward(plan._native, gout, gy, x, z, q, post, scale, pre, need_gh, outs, _current(ref))
    return r if type(r) is tuple else _result(r, explain)


class AdamW:
    """cgtp_adamw_create: AdamW over tensors of ``numel`` elements each.

    state "f32" (or "full": the parameters' type) or "8bit".  decay_scale: factor of the weight
    decay for each tensor (0: not decayed).

    The optimizer owns the partial sums of the gradient norm: its norms must not overlap on the GPU."""

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
        self.device = _here()
        total = ctypes.c_int64()
        _check(lib().cgtp_adamw_info(h, ctypes.byref(total)))
        self.state_numel = total.value
        self._sizes = sizes                     # read by the native calls
        self._native = (h.value, _dtype(self.param_dtype, "param_dtype", (CGTP_F32, CGTP_F64)),
                        _dtype(self.grad_dtype, "grad_dtype", (CGTP_F32, CGTP_F64, CGTP_BF16)), STATES[state],
                        self.state_numel, n, ctypes.addressof(sizes), self.device.index)

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

    def explain(self, lists, state=None, clip=None):
        """Raises what is wrong with the arguments of a step."""
        _explain_device(self.device)
        for name, tensors, dtype in lists:
            if tensors is not None:
                _explain_list(name, tensors, self.numel, dtype, self.device)
        if state is not None:
            n, eight = self.state_numel, self.state == "8bit"
            for name in ("m", "v") + (("m_exp", "v_exp") if eight else ()):
                if state[name] is None:
                    raise ValueError(f"state {name} is missing")
                _explain_vector("state " + name, state[name], torch.uint8 if eight else self.param_dtype,
                                n // STATE_BLOCK if name.endswith("exp") else n, self.device)
        _explain_vector("norm and coefficient", clip, self.param_dtype, 2, self.device)

    def __del__(self):
        h = getattr(self, "_h", None)
        if h is not None and h.value and lib is not None:
            lib().cgtp_adamw_destroy(h)
            self._h = None


def cgtp_grad_norm(opt, grads, max_norm=float("inf"), out=None, stream=None):
    """Tensor [norm of all gradients, min(1, max_norm / norm)]; None gradients count as zero."""
    if stream is not None:
        return _on(stream, cgtp_grad_norm, opt, grads, max_norm, out)
    ref = out if out is not None else next((g for g in grads if g is not None), None)
    if ref is None:
        out = ref = torch.empty(2, dtype=opt.param_dtype, device="cuda")
    r = _binding.grad_norm(opt._native, grads, max_norm, out, _current(ref))
    return r if type(r) is torch.Tensor else _result(r, lambda: opt.explain([("grads", grads, opt.grad_dtype)], clip=out))


def cgtp_adamw_step(opt, params, grads, state, lr, betas=(0.9, 0.999), eps=1e-8, weight_decay=0.0, step=1,
                    copies=None, clip=None, seed=0, stream=None):
    """One AdamW step in place.  A None gradient skips its tensor.  copies: bfloat16 tensors (or None)
    that receive the new parameters.  clip: result of cgtp_grad_norm.  seed: rounding of 8-bit states.

    lr, step and seed are taken at the call: a captured graph repeats the captured step's bias correction and rounding
    bits, so a training loop calls the step outside its graphs."""
    if stream is not None:
        return _on(stream, cgtp_adamw_step, opt, params, grads, state, lr, betas, eps, weight_decay, step, copies, clip, seed)
    r = _binding.adamw_step(opt._native, params, grads, copies, state["m"], state["v"], state["m_exp"], state["v_exp"], lr, betas[0],
                            betas[1], eps, weight_decay, step, seed, clip, _current(state["m"]))
    if r is not None:
        _result(r, lambda: opt.explain([("params", params, opt.param_dtype), ("grads", grads, opt.grad_dtype),
                                        ("copies", copies, torch.bfloat16)], state, clip))


def cgtp_adamw_state_values(opt, state, stream=None):
    """(m, v) as the FP32 values the 8-bit states stand for (the states themselves otherwise)."""
    if opt.state != "8bit":
        return state["m"], state["v"]
    if stream is not None:
        return _on(stream, cgtp_adamw_state_values, opt, state)
    r = _binding.state_values(opt._native, state["m"], state["v"], state["m_exp"], state["v_exp"], _current(state["m"]))
    return r if type(r) is tuple else _result(r, lambda: opt.explain([], state))
