"""Attention: refusals that need no GPU, the bucket borders, and the oracle against direct loops."""

import ctypes
import math
import os
import re

import numpy as np
import pytest

import clebsch_gordan_tensor_racah_gb300 as cg
from oracle import attn as oat

torch = pytest.importorskip("torch")


def _create(irreps_qk=b"4x0e", irreps_v=b"4x0e+4x1o", heads=2, kv=2, dtype=cg.CGTP_F32, flags=0, scale=0.5, borders=()):
    h = ctypes.c_void_p()
    s = cg.lib().cgtp_attn_create(ctypes.byref(h), irreps_qk, irreps_v, heads, kv, dtype, flags, scale, len(borders),
                                  (ctypes.c_double * max(1, len(borders)))(*borders))
    if h.value:
        cg.lib().cgtp_attn_destroy(h)
    return s


@pytest.mark.parametrize("kw", [dict(irreps_qk=None), dict(irreps_qk=b""), dict(irreps_qk=b"4x"), dict(irreps_v=b"4x0e+"), dict(irreps_v=b"0x0e"),
                                dict(heads=0), dict(heads=65), dict(heads=-1), dict(kv=0), dict(kv=3), dict(heads=2, kv=4), dict(heads=3, kv=2), dict(dtype=9),
                                dict(flags=2), dict(flags=1), dict(dtype=cg.CGTP_F64, flags=1), dict(scale=math.nan), dict(scale=math.inf),
                                dict(borders=(2.0, 1.0)), dict(borders=(1.0, math.nan)), dict(borders=(1.0, math.inf)),
                                dict(borders=tuple(range(512)))])
def test_plans_that_cannot_be_are_refused(kw):
    assert _create(**kw) == cg.CGTP_EINVAL


def test_rows_too_long_are_refused():
    assert _create(irreps_v=b"4097x0e") == cg.CGTP_EUNSUPPORTED
    assert _create(irreps_qk=b"8193x0e", heads=1, kv=1) == cg.CGTP_EUNSUPPORTED
    assert _create(irreps_v=b"200000000x7e", heads=64, kv=1) in (cg.CGTP_EINVAL, cg.CGTP_EUNSUPPORTED)


def test_null_handles_are_refused():
    L, n = cg.lib(), ctypes.c_int64()
    none = [None] * 40
    assert L.cgtp_attn_create(None, b"1x0e", b"1x0e", 1, 1, 0, 0, 1.0, 0, None) == cg.CGTP_EINVAL
    assert L.cgtp_attn_info(None, ctypes.byref(n), None) == cg.CGTP_EINVAL
    assert L.cgtp_attn_workspace(None, None, 0, ctypes.byref(n)) == cg.CGTP_EINVAL
    assert L.cgtp_attn_device_bytes(None, ctypes.byref(n)) == cg.CGTP_EINVAL
    for f in (L.cgtp_attn_forward, L.cgtp_attn_backward, L.cgtp_attn_edges_forward, L.cgtp_attn_edges_backward):
        args = [0 if a is ctypes.c_int64 else None for a, _ in zip(f.argtypes, none)]
        assert f(*args) == cg.CGTP_EINVAL
    L.cgtp_attn_destroy(None)


def test_every_entry_point_of_the_header_is_exported():
    root = os.path.dirname(os.path.dirname(cg.__file__))
    names = re.findall(r"\b(cgtp_(?:attn|graph)_\w+)\(", open(os.path.join(root, "include", "cgtp_attn.h")).read())
    assert len(set(names)) == 10 and set(names) <= set(cg.EXPORTS)
    assert all(hasattr(cg.lib(), n) for n in names)


def test_borders():
    b = cg.attention_borders(32, 1.0, 5.0)
    assert len(b) == 31 and b == sorted(b) and b[15] == 1.0 and b[-1] == pytest.approx(5.0)
    assert np.allclose(np.diff(b[:16]), 1 / 16) and np.allclose(np.diff(np.log(b[15:])), math.log(5.0) / 15)
    assert cg.attention_borders(2, 1.0, 5.0) == [1.0]
    assert list(oat.buckets([0.0, 1.0, 1.5, np.nan, 9.0], [1.0, 2.0])) == [0, 1, 1, 0, 2]
    for bad in ((1, 1.0, 5.0), (8, 0.0, 5.0), (8, 5.0, 5.0), (8, 1.0, math.inf), (8, math.nan, 5.0)):
        with pytest.raises(ValueError):
            cg.attention_borders(*bad)


def test_oracle_against_loops():
    rng = np.random.default_rng(0)
    heads, kv, qk, v = 4, 2, "2x0e+1x1o", "1x0e+2x1o"
    n, m, deg = 3, 4, [3, 0, 2]
    dst, col = np.repeat(np.arange(n), deg), rng.integers(0, m, sum(deg))
    q, k, x = rng.standard_normal((n, heads * 5)), rng.standard_normal((m, kv * 5)), rng.standard_normal((m, kv * 7))
    z, _ = oat.logits(q, k, qk, heads, kv, 0.3, dst, col)
    a, lse = oat.softmax(z, dst, n)
    out = oat.gather_back(oat.receive(oat.weighed(a, oat.spread(x, v, kv, heads)[col]), dst, n), v, heads, (n, heads * 7))
    want = np.zeros_like(out)
    for i in range(n):
        es = np.flatnonzero(dst == i)
        for h in range(heads):
            g = h // 2
            qh = np.concatenate([q[i, 2 * h:2 * h + 2], q[i, 8 + 3 * h:11 + 3 * h]])
            zs = np.array([0.3 * qh @ np.concatenate([k[col[e], 2 * g:2 * g + 2], k[col[e], 4 + 3 * g:7 + 3 * g]]) for e in es])
            if not len(es):
                assert lse[i, h] == -np.inf
                continue
            p = np.exp(zs - zs.max())
            for w, e in zip(p / p.sum(), es):
                want[i, h] += w * x[col[e], g]
                want[i, 4 + 6 * h:10 + 6 * h] += w * x[col[e], 2 + 6 * g:8 + 6 * g]
            assert np.isclose(lse[i, h], np.log(p.sum()) + zs.max())
    assert np.allclose(out, want)


def test_weights_turn_with_nothing():
    # the inner products of irreps rows do not change under a rotation of both (here: about the axis that mixes two
    # components of l = 1)
    rng = np.random.default_rng(1)
    q, k = rng.standard_normal((5, 2 + 6)), rng.standard_normal((5, 2 + 6))
    c, s = math.cos(0.7), math.sin(0.7)
    R = np.array([[c, 0, s], [0, 1, 0], [-s, 0, c]])

    def turned(x):
        y = x.copy()
        y[:, 2:] = (x[:, 2:].reshape(5, 2, 3) @ R.T).reshape(5, 6)
        return y

    dst, col = np.arange(5), np.arange(5)[::-1]
    z0, _ = oat.logits(q, k, "1x0e+1x1o", 2, 2, 1.0, dst, col)
    z1, _ = oat.logits(turned(q), turned(k), "1x0e+1x1o", 2, 2, 1.0, dst, col)
    assert np.allclose(z0, z1)
