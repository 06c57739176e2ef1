"""Refusals of the training-step operators that need no GPU, at the C boundary."""

import ctypes

import clebsch_gordan_tensor_racah_gb300 as cg


def test_resnorm_create_rejects_bad_arguments_before_device_work():
    L = cg.lib()
    h = ctypes.c_void_p()
    inf, nan = float("inf"), float("nan")
    cases = [
        (b"8x0e+", 0, 0, 0, 1.0, 1e-5, cg.CGTP_EINVAL),       # empty term
        (b"8x9e", 0, 0, 0, 1.0, 1e-5, cg.CGTP_EINVAL),        # l > 7
        (b"0x0e", 0, 0, 0, 1.0, 1e-5, cg.CGTP_EINVAL),        # a block without channels
        (b"8x0e", 3, 0, 0, 1.0, 1e-5, cg.CGTP_EINVAL),        # unknown type
        (b"8x0e", 0, 8, 0, 1.0, 1e-5, cg.CGTP_EINVAL),        # unknown flag
        (b"8x0e", 0, 0, 4, 1.0, 1e-5, cg.CGTP_EINVAL),        # unknown gate
        (b"8x0e", 0, 0, -1, 1.0, 1e-5, cg.CGTP_EINVAL),
        (b"8x0e", 0, 0, 0, 1.0, -1e-5, cg.CGTP_EINVAL),       # negative eps
        (b"8x0e", 0, 0, 0, 1.0, nan, cg.CGTP_EINVAL),
        (b"8x0e", 0, 0, 0, inf, 1e-5, cg.CGTP_EINVAL),
        (b"60000x7o+60000x7o", 0, 0, 0, 1.0, 1e-5, cg.CGTP_EUNSUPPORTED),   # rows too long
    ]
    for irreps, dtype, flags, act, alpha, eps, want in cases:
        st = L.cgtp_resnorm_create(ctypes.byref(h), irreps, dtype, flags, act, alpha, eps)
        assert st == want, (irreps, st, L.cgtp_last_error())
        assert not h.value
    assert L.cgtp_resnorm_create(None, b"8x0e", 0, 0, 0, 1.0, 1e-5) == cg.CGTP_EINVAL
    assert L.cgtp_resnorm_create(ctypes.byref(h), None, 0, 0, 0, 1.0, 1e-5) == cg.CGTP_EINVAL


def test_adamw_create_rejects_bad_arguments_before_device_work():
    L = cg.lib()
    h = ctypes.c_void_p()
    sizes = (ctypes.c_int64 * 2)(4, 4)
    less = (ctypes.c_int64 * 2)(4, -4)
    huge = (ctypes.c_int64 * 2)(4, 1 << 40)
    nan = (ctypes.c_float * 2)(1.0, float("nan"))
    cases = [
        (0, sizes, None, 0, 0, 0, cg.CGTP_EINVAL),
        (2, None, None, 0, 0, 0, cg.CGTP_EINVAL),
        (2, less, None, 0, 0, 0, cg.CGTP_EINVAL),
        (2, huge, None, 0, 0, 0, cg.CGTP_EUNSUPPORTED),
        (2, sizes, nan, 0, 0, 0, cg.CGTP_EINVAL),
        (2, sizes, None, 2, 2, 0, cg.CGTP_EINVAL),            # bfloat16 parameters
        (2, sizes, None, 1, 0, 0, cg.CGTP_EINVAL),            # FP32 gradients of FP64 parameters
        (2, sizes, None, 0, 0, 2, cg.CGTP_EINVAL),            # unknown state
        (2, sizes, None, 1, 1, 1, cg.CGTP_EUNSUPPORTED),      # 8-bit states of FP64 parameters
    ]
    for n, numel, decay, pd, gd, state, want in cases:
        st = L.cgtp_adamw_create(ctypes.byref(h), n, numel, decay, pd, gd, state)
        assert st == want, (n, st, L.cgtp_last_error())
        assert not h.value


def test_null_handles_rejected():
    L = cg.lib()
    z = ctypes.c_void_p()
    assert L.cgtp_resnorm_forward(None, 1, z, 0, z, 0, z, 0, z, z, z, z, 0, z, 0, z) == cg.CGTP_EINVAL
    assert L.cgtp_resnorm_info(None, None, None, None) == cg.CGTP_EINVAL
    assert L.cgtp_adamw_step(None, z, z, z, z, z, z, z, 0.0, 0.9, 0.9, 0.0, 0.0, 1, 0, z, z) == cg.CGTP_EINVAL
    assert L.cgtp_grad_norm(None, z, 1.0, z, z) == cg.CGTP_EINVAL
    assert L.cgtp_adamw_state_values(None, z, z, z, z, z, z, z) == cg.CGTP_EINVAL
    L.cgtp_resnorm_destroy(None)
    L.cgtp_adamw_destroy(None)
