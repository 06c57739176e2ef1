"""FP64 oracle of the operators of a training step: the gated residual norm, AdamW and the
8-bit state codes.  NumPy, one definition per function, nothing shared with the kernels."""

import math

import numpy as np


def parse(irreps):
    """[(multiplicity, 2l+1)] of an irreps string."""
    out = []
    for term in irreps.replace(" ", "").split("+"):
        mul, ir = term.split("x") if "x" in term else ("1", term)
        out.append((int(mul), 2 * int(ir[:-1]) + 1))
    return out


def sizes(irreps):
    b = parse(irreps)
    return sum(m * d for m, d in b), sum(m for m, _ in b)


def gate(act, q):
    """a(q) and a'(q)."""
    if act == "none":
        return np.ones_like(q), np.zeros_like(q)
    if act == "identity":
        return q, np.ones_like(q)
    with np.errstate(over="ignore"):
        s = 1.0 / (1.0 + np.exp(-q))
    if act == "sigmoid":
        return s, s * (1 - s)
    return q * s, s + q * s * (1 - s)


def _blocks(irreps):
    off = coff = 0
    for mul, d in parse(irreps):
        yield slice(off, off + mul * d), slice(coff, coff + mul), mul, d
        off, coff = off + mul * d, coff + mul


def _f64(v):
    return None if v is None else np.asarray(v, dtype=np.float64)


def resnorm_forward(irreps, h=None, z=None, q=None, post=None, scale=None, pre=None, act="none", pre_norm=True,
                    post_norm=True, alpha=1.0, eps=1e-5):
    """(out, y): out = alpha h + scale a(q) post rms(z) z, y = pre rms(out) out."""
    h, z, q, post, scale, pre = map(_f64, (h, z, q, post, scale, pre))
    dim, chan = sizes(irreps)
    one = np.ones(chan)
    post, scale, pre = (one if v is None else v for v in (post, scale, pre))
    n = (h if h is not None else z).shape[0]
    out, y = np.zeros((n, dim)), np.zeros((n, dim))
    for e, c, mul, d in _blocks(irreps):
        if z is None:
            o = h[:, e].reshape(n, mul, d)
        else:
            b = z[:, e].reshape(n, mul, d)
            r = 1 / np.sqrt((b ** 2).mean(axis=(1, 2), keepdims=True) + eps) if post_norm else 1.0
            a = gate(act, q[:, c])[0] if act != "none" else 1.0
            o = (scale[c] * post[c] * a)[..., None] * b * r if act != "none" else (scale[c] * post[c])[:, None] * b * r
            if h is not None:
                o = o + alpha * h[:, e].reshape(n, mul, d)
        out[:, e] = o.reshape(n, mul * d)
        y[:, e] = (pre[c][:, None] * o / np.sqrt((o ** 2).mean(axis=(1, 2), keepdims=True) + eps)).reshape(n, mul * d)
    return out, (y if pre_norm else None)


def resnorm_backward(irreps, gout, gy, x, z=None, q=None, post=None, scale=None, pre=None, act="none", pre_norm=True,
                     post_norm=True, alpha=1.0, eps=1e-5):
    """(gh, gz, gq, gpost, gscale, gpre), in the order of summation of the definition."""
    gout, gy, x, z, q, post, scale, pre = map(_f64, (gout, gy, x, z, q, post, scale, pre))
    dim, chan = sizes(irreps)
    one = np.ones(chan)
    post, scale, pre = (one if v is None else v for v in (post, scale, pre))
    n = (gout if gout is not None else gy).shape[0]
    gh, gz, gq = np.zeros((n, dim)), np.zeros((n, dim)), np.zeros((n, chan))
    gpost, gscale, gpre = np.zeros(chan), np.zeros(chan), np.zeros(chan)
    for e, c, mul, d in _blocks(irreps):
        g = np.zeros((n, mul, d)) if gout is None else gout[:, e].reshape(n, mul, d)
        if pre_norm:
            b, k = x[:, e].reshape(n, mul, d), gy[:, e].reshape(n, mul, d)
            p = 1 / np.sqrt((b ** 2).mean(axis=(1, 2), keepdims=True) + eps)
            w = k * pre[c][:, None]
            g = g + p * w - p ** 3 * b * (w * b).mean(axis=(1, 2), keepdims=True)
            gpre[c] = (p * b * k).sum(axis=(0, 2))
        gh[:, e] = (1.0 if z is None else alpha) * g.reshape(n, mul * d)     # without z the stream is h itself
        if z is None:
            continue
        b = z[:, e].reshape(n, mul, d)
        r = 1 / np.sqrt((b ** 2).mean(axis=(1, 2), keepdims=True) + eps) if post_norm else np.ones((n, 1, 1))
        a, da = gate(act, q[:, c]) if act != "none" else (np.ones((n, mul)), np.zeros((n, mul)))
        v = g * (scale[c] * post[c] * a)[..., None]      # gradient of r z
        gz[:, e] = (r * v - (r ** 3 * b * (v * b).mean(axis=(1, 2), keepdims=True) if post_norm else 0.0)).reshape(n, mul * d)
        along = (g * r * b).sum(axis=2)
        gq[:, c] = along * scale[c] * post[c] * da
        gpost[c] = (along * a * scale[c]).sum(axis=0)
        gscale[c] = (along * a * post[c]).sum(axis=0)
    return gh, gz, gq, gpost, gscale, gpre


# ---------------------------------------------------------------------------
# AdamW
# ---------------------------------------------------------------------------

BLOCK, E_MIN = 128, 40


def code_table(top):
    """Values of all codes of a block with exponent 127 (largest exponent field `top`), in units where
    the block's power of two is 1: field 0 is linear."""
    code = np.arange(8 * (top + 1))
    field, mant = code // 8, code % 8
    return np.where(field == 0, mant / 8 * 2.0 ** (1 - top), (1 + mant / 8) * 2.0 ** (field - top))


def state_values(code, exp, top, signed):
    """Values of uint8 codes [k * BLOCK] with block exponents [k]."""
    code = np.asarray(code, dtype=np.int64)
    e = np.maximum(np.repeat(np.asarray(exp, dtype=np.int64), BLOCK), E_MIN)
    v = code_table(top)[code & 127 if signed else code] * np.exp2(e - 127.0)
    v = np.where(e == 255, np.nan, v)
    return np.where(code & 128, -v, v) if signed else v


def adamw(p, g, m, v, lr, betas, eps, decay, step, coef=1.0):
    """(p, m, v) after one step in FP64."""
    p, g, m, v = map(_f64, (p, g, m, v))
    g = coef * g
    m = betas[0] * m + (1 - betas[0]) * g
    v = betas[1] * v + (1 - betas[1]) * g * g
    hat_m, hat_v = m / (1 - betas[0] ** step), v / (1 - betas[1] ** step)
    return p * (1 - lr * decay) - lr * hat_m / (np.sqrt(hat_v) + eps), m, v


def grad_norm(grads, max_norm):
    n = math.sqrt(sum(float((np.asarray(g, dtype=np.float64) ** 2).sum()) for g in grads))
    return n, min(1.0, max_norm / n) if n else 1.0
