"""FP64 oracle of the attention along a graph's edges, of values and of edge rows, with the sums of magnitudes that
bound a computation's rounding.  NumPy, straight from the definition, nothing shared with the kernels."""

import numpy as np

from .train import parse


def columns(irreps, heads):
    """[heads, elements]: columns of each head's elements in rows of `heads` heads."""
    out, at = [], 0
    for mul, d in parse(irreps):
        out.append(at + np.arange(heads * mul * d).reshape(heads, mul * d))
        at += heads * mul * d
    return np.concatenate(out, axis=1)


def spread(x, irreps, count, heads):
    """Rows of `count` (shared) heads as [rows, heads, elements]."""
    x = np.asarray(x, dtype=np.float64)[:, columns(irreps, count)]
    return np.repeat(x, heads // count, axis=1)


def gather_back(x, irreps, count, shape):
    """The adjoint of spread."""
    rows, heads, d = x.shape
    out = np.zeros(shape)
    out[:, columns(irreps, count)] = x.reshape(rows, count, heads // count, d).sum(2)
    return out


def buckets(lengths, borders):
    """Number of borders <= r (0 for NaN)."""
    with np.errstate(invalid="ignore"):
        return (np.asarray(borders)[None, :] <= np.asarray(lengths)[:, None]).sum(1)


def logits(q, k, irreps, heads, kv, scale, dst, col, bias=0.0):
    """(z [E, heads], magnitudes of its terms); -inf where the bias is."""
    a, b = spread(q, irreps, heads, heads)[dst], spread(k, irreps, kv, heads)[col]
    bias = np.broadcast_to(np.asarray(bias, dtype=np.float64), (len(dst), heads))
    shut = bias == -np.inf
    open_ = np.where(shut, 0.0, bias)
    z = np.where(shut, -np.inf, scale * np.where(shut[:, :, None], 0.0, a * b).sum(2) + open_)
    return z, scale * np.where(shut[:, :, None], 0.0, np.abs(a * b)).sum(2) + np.abs(open_)


def softmax(z, dst, n):
    """(a, lse): weights over each receiver's edges, zeros and -inf where nothing is left."""
    top = np.full((n, z.shape[1]), -np.inf)
    np.maximum.at(top, dst, z)
    shift = np.where(top == -np.inf, 0.0, top)
    p = np.exp(z - shift[dst])
    total = np.zeros_like(top)
    np.add.at(total, dst, p)
    with np.errstate(divide="ignore"):
        return p / np.where(total == 0, 1.0, total)[dst], np.log(total) + shift


def receive(x, dst, n):
    out = np.zeros((n,) + x.shape[1:])
    np.add.at(out, dst, x)
    return out


def weighed(a, x):
    """a x, where a weight of zero takes nothing from x, whatever it holds."""
    return np.where(a[:, :, None] == 0, 0.0, a[:, :, None] * np.where(a[:, :, None] == 0, 0.0, x))


def logit_gradient(a, dp, dst, n):
    """ds = a (dp - sum over the receiver's edges of a dp)."""
    dp = np.where(a == 0, 0.0, dp)
    return a * (dp - receive(a * dp, dst, n)[dst])
