"""CPU-only checks of the 16-bit products' C calls: bad arguments are rejected
on the host before the device is touched, empty calls are no-ops, workspace
sizes grow with what is asked for."""
import ctypes

import pytest

from test_abi import FAKE, MX_ERR_INVALID_ARGUMENT, MX_ERR_MISALIGNED, MX_ERR_UNSUPPORTED_SHAPE, MX_OK

BF16, FP16, FP32 = 0, 1, 2
BIG = (1 << 31) - 1023   # one above the largest size


@pytest.fixture(scope="module")
def lib():
    import moe_grouped_gemm_mx_b200 as mx   # sets the argument types
    return mx._lib


def test_linear_act(lib):
    def f(x=FAKE, w=FAKE, bias=None, res=None, z=None, y=FAKE, m=4, n=16, k=32, dtype=BF16, act=0):
        return lib.mx_linear_act(x, w, bias, res, z, y, m, n, k, dtype, act, None, None)
    assert f(m=-1) == f(n=-8) == f(k=-8) == MX_ERR_INVALID_ARGUMENT
    assert f(dtype=FP32) == f(dtype=-1) == f(dtype=3) == MX_ERR_INVALID_ARGUMENT
    assert f(act=-1) == f(act=5) == MX_ERR_INVALID_ARGUMENT
    assert f(k=0) == f(k=36) == f(n=20) == MX_ERR_UNSUPPORTED_SHAPE
    assert f(m=BIG) == f(n=1 << 31) == f(k=1 << 31) == f(k=(1 << 27) + 8) == MX_ERR_UNSUPPORTED_SHAPE
    assert f(x=None) == f(w=None) == f(y=None) == MX_ERR_INVALID_ARGUMENT
    for name in ("x", "w", "bias", "res", "z", "y"):
        assert f(**{name: FAKE + 8}) == MX_ERR_MISALIGNED
    assert f(x=None, w=None, y=None, m=0) == f(x=None, w=None, y=None, n=0) == MX_OK
    assert f(m=0, k=20) == MX_ERR_UNSUPPORTED_SHAPE


def test_linear_act_backward(lib):
    ws = lib.mx_linear_act_backward_workspace_bytes
    assert ws(0, 8) == ws(8, 0) == ws(-1, 8) == 0
    assert ws(1, 8) == ws(1024, 8) == 0 and ws(1025, 8) == 9 * 32 and ws(8192, 4096) == 64 * 4096 * 4

    def f(dy=FAKE, z=FAKE, x=FAKE, w=FAKE, dz=FAKE, dx=FAKE, dw=FAKE, db=FAKE, m=4, n=16, k=32, dtype=BF16, act=1, work=FAKE,
          size=1 << 20):
        return lib.mx_linear_act_backward(dy, z, x, w, dz, dx, dw, db, m, n, k, dtype, act, work, size, None, None)
    assert f(m=-1) == f(dtype=FP32) == f(act=7) == MX_ERR_INVALID_ARGUMENT
    assert f(k=0) == f(k=33) == f(n=9) == f(m=BIG) == MX_ERR_UNSUPPORTED_SHAPE
    assert f(m=(1 << 27) + 1) == f(n=(1 << 27) + 8) == MX_ERR_UNSUPPORTED_SHAPE   # dw sums over m, dx over n
    assert f(dy=None) == f(z=None) == f(dz=None) == MX_ERR_INVALID_ARGUMENT
    assert f(x=None) == f(w=None) == MX_ERR_INVALID_ARGUMENT            # dw wants x, dx wants w
    big = {"m": 2000, "n": 16}
    assert f(work=None, **big) == f(size=16 * 16 * 4 - 1, **big) == MX_ERR_INVALID_ARGUMENT  # dbias wants the workspace
    for name in ("dy", "z", "x", "w", "dz", "dx", "dw", "db", "work"):
        assert f(**{name: FAKE + 4}) == MX_ERR_MISALIGNED
    assert f(dx=None, dw=None, db=None) == MX_OK                        # nothing wanted
    assert f(m=0, dx=None, dw=None, db=None) == f(n=0, dx=None) == MX_OK


def test_grouped_ragged(lib):
    calls = {
        "forward": lambda a, b, off, g, m, n, k, t, d: lib.mx_grouped_gemm_ragged(a, b, off, g, m, n, k, t, d, None, None),
        "dgrad": lambda a, b, off, g, m, n, k, t, d: lib.mx_grouped_gemm_ragged_dgrad(a, b, off, g, m, n, k, t, d, None, None),
        "wgrad": lambda a, b, off, g, m, n, k, t, d: lib.mx_grouped_gemm_ragged_wgrad(a, b, off, g, m, n, k, t, t, d, None, None),
    }
    for name, f in calls.items():
        assert f(FAKE, FAKE, FAKE, -1, 4, 16, 32, BF16, FAKE) == MX_ERR_INVALID_ARGUMENT
        assert f(FAKE, FAKE, FAKE, 2, -1, 16, 32, BF16, FAKE) == MX_ERR_INVALID_ARGUMENT
        assert f(FAKE, FAKE, FAKE, 2, 4, 16, 32, FP32, FAKE) == MX_ERR_INVALID_ARGUMENT
        for bad in ((2, 4, 0, 32), (2, 4, 16, 0), (2, 4, 12, 32), (2, 4, 16, 36), (1025, 4, 16, 32), (2, BIG, 16, 32)):
            assert f(FAKE, FAKE, FAKE, *bad, FP16, FAKE) == MX_ERR_UNSUPPORTED_SHAPE, (name, bad)
        assert f(None, FAKE, FAKE, 2, 4, 16, 32, BF16, FAKE) == MX_ERR_INVALID_ARGUMENT
        assert f(FAKE, None, FAKE, 2, 4, 16, 32, BF16, FAKE) == MX_ERR_INVALID_ARGUMENT
        assert f(FAKE, FAKE, None, 2, 4, 16, 32, BF16, FAKE) == MX_ERR_INVALID_ARGUMENT
        assert f(FAKE, FAKE, FAKE, 2, 4, 16, 32, BF16, None) == MX_ERR_INVALID_ARGUMENT
        assert f(FAKE + 8, FAKE, FAKE, 2, 4, 16, 32, BF16, FAKE) == MX_ERR_MISALIGNED
        assert f(FAKE, FAKE + 2, FAKE, 2, 4, 16, 32, BF16, FAKE) == MX_ERR_MISALIGNED
        assert f(FAKE, FAKE, FAKE + 2, 2, 4, 16, 32, BF16, FAKE) == MX_ERR_MISALIGNED
        assert f(FAKE, FAKE, FAKE, 2, 4, 16, 32, BF16, FAKE + 8) == MX_ERR_MISALIGNED
        assert f(None, None, None, 0, 4, 16, 32, BF16, None) == MX_OK
    for name in ("forward", "dgrad"):
        assert calls[name](None, None, None, 2, 0, 16, 32, BF16, None) == MX_OK
    over = (1 << 27) + 8
    assert calls["forward"](FAKE, FAKE, FAKE, 2, 4, 16, over, BF16, FAKE) == MX_ERR_UNSUPPORTED_SHAPE
    assert calls["dgrad"](FAKE, FAKE, FAKE, 2, 4, over, 16, BF16, FAKE) == MX_ERR_UNSUPPORTED_SHAPE
    assert calls["wgrad"](FAKE, FAKE, FAKE, 2, over, 16, 16, BF16, FAKE) == MX_ERR_UNSUPPORTED_SHAPE
    w = lib.mx_grouped_gemm_ragged_wgrad
    assert w(FAKE, FAKE, FAKE, 2, 4, 16, 32, BF16, FP16, FAKE, None, None) == MX_ERR_INVALID_ARGUMENT
    assert w(FAKE, FAKE, FAKE, 2, 4, 16, 32, FP16, BF16, FAKE, None, None) == MX_ERR_INVALID_ARGUMENT
    assert w(None, None, None, 2, 0, 16, 32, FP16, FP32, None, None, None) == MX_ERR_INVALID_ARGUMENT  # zeros to write


def test_orthogonalize(lib):
    ws = lib.mx_orthogonalize_workspace_bytes
    assert ws(0, 8, 8, BF16, 5) == ws(1, 0, 8, BF16, 5) == ws(1, 8, (1 << 20) + 1, BF16, 5) == ws(1, 8, 8, BF16, 0) == 0
    assert ws(2, 64, 128, BF16, 5) > ws(1, 64, 128, BF16, 5) > ws(1, 64, 128, BF16, 3)
    usual = (3.4445, -4.7750, 2.0315)

    def f(g=FAKE, t=BF16, out=FAKE, batch=1, m=16, n=24, steps=5, coeffs=None, eps=1e-7, work=FAKE, size=1 << 30):
        flat = usual * 5 if coeffs is None else coeffs
        arr = (ctypes.c_float * max(1, len(flat)))(*flat)
        return lib.mx_orthogonalize(g, t, out, batch, m, n, steps, arr, eps, work, size, None, None)
    assert f(batch=-1) == f(m=-1) == f(n=-1) == MX_ERR_INVALID_ARGUMENT
    assert f(t=FP16) == f(t=3) == f(steps=0) == f(steps=17, coeffs=usual * 17) == MX_ERR_INVALID_ARGUMENT
    assert f(eps=-1.0) == f(eps=float("nan")) == f(eps=float("inf")) == MX_ERR_INVALID_ARGUMENT
    assert f(steps=1, coeffs=(4.5, 0.0, 0.0)) == MX_ERR_INVALID_ARGUMENT            # singular values above 3.9
    assert f(steps=3, coeffs=(2.5, 0.0, 0.0) * 3) == MX_ERR_INVALID_ARGUMENT        # on the way
    assert f(steps=1, coeffs=(20.0, -60.0, 40.0)) == MX_ERR_INVALID_ARGUMENT       # |a + b s^2 + c s^4| above 15.5
    assert f(steps=1, coeffs=(3.8, 0.0, 0.0), g=None, out=None, work=None, batch=0) == MX_OK
    assert f(steps=1, coeffs=(float("inf"), 0.0, 0.0)) == MX_ERR_INVALID_ARGUMENT
    assert f(batch=65536) == f(m=(1 << 20) + 1) == f(n=(1 << 20) + 1) == MX_ERR_UNSUPPORTED_SHAPE
    assert f(g=None) == f(out=None) == f(work=None) == f(size=100) == MX_ERR_INVALID_ARGUMENT
    assert f(g=FAKE + 8) == f(out=FAKE + 8) == f(work=FAKE + 16) == MX_ERR_MISALIGNED
    assert f(g=None, out=None, work=None, batch=0) == f(g=None, out=None, work=None, m=0) == MX_OK
    assert lib.mx_orthogonalize(FAKE, BF16, FAKE, 1, 8, 8, 5, None, 1e-7, FAKE, 1 << 30, None, None) == MX_ERR_INVALID_ARGUMENT


def test_orthogonalize_workspace_serves_other_step_counts(lib):
    """From four steps on (fewer may do with less) the number of steps does not change the size."""
    ws = lib.mx_orthogonalize_workspace_bytes
    for batch, m, n in ((1, 1, 1), (3, 129, 257), (70, 300, 200)):
        assert len({ws(batch, m, n, BF16, steps) for steps in range(4, 17)}) == 1
        assert len({ws(batch, m, n, FP32, steps) for steps in range(1, 17)}) == 1
