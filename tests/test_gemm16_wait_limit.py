"""A wait bound far below the kernels' legitimate waits, in the ragged products
and both forms of the orthogonalisation: the call reports MX_DEV_TIMEOUT, ends,
writes nothing outside its output, and the next call is right."""
import contextlib

import pytest
import torch

from gemm16_util import guarded, normal

pytestmark = pytest.mark.gpu

BF16, FP32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def mx():
    import moe_grouped_gemm_mx_b200 as m
    return m


@contextlib.contextmanager
def limit(mx, ns):
    mx.mx_set_wait_limit_ns(ns)
    try:
        yield
    finally:
        mx.mx_set_wait_limit_ns(0)


def times_out_and_recovers(mx, call, shape, dtype):
    """call(out, status), whose waits for its first accumulator take hundreds of microseconds."""
    want, _ = guarded(shape, dtype)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    call(want, status)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    out, intact = guarded(shape, dtype)
    with limit(mx, 1000):
        call(out, status)
        torch.cuda.synchronize()
    assert int(status.item()) & mx.MX_DEV_TIMEOUT and intact()
    status.zero_()
    call(out, status)
    torch.cuda.synchronize()
    assert int(status.item()) == 0 and intact() and torch.equal(out, want)


LONG = 1 << 18


@pytest.mark.parametrize("cfg", ["0", "1", "2"])
def test_ragged_forward_and_input_gradient(mx, cfg, monkeypatch):
    monkeypatch.setenv("MX_GEMM16_CONFIG", cfg)
    off = torch.tensor([0, 40, 40, 300], dtype=torch.int32, device="cuda")
    a, b = normal((300, LONG), BF16, 1), normal((3, 264, LONG), BF16, 2, 0.002)
    times_out_and_recovers(mx, lambda o, s: mx.mx_grouped_gemm_ragged(a, b, off, d=o, dev_status=s), (300, 264), BF16)
    bt = b.view(3, LONG, 264)
    times_out_and_recovers(mx, lambda o, s: mx.mx_grouped_gemm_ragged_dgrad(a, bt, off, da=o, dev_status=s), (300, 264), BF16)


@pytest.mark.parametrize("out_dtype", [BF16, FP32], ids=["bf16", "fp32"])
def test_ragged_weight_gradient(mx, out_dtype):
    """Groups that end inside a step of the tensor core's (their rows are cleared by a warp of its own)."""
    rows = LONG + 71
    off = torch.tensor([0, 33, LONG, rows], dtype=torch.int32, device="cuda")
    dd, a = normal((rows, 264), BF16, 3, 0.01), normal((rows, 136), BF16, 4)
    times_out_and_recovers(mx, lambda o, s: mx.mx_grouped_gemm_ragged_wgrad(dd, a, off, db=o, dev_status=s),
                           (3, 264, 136), out_dtype)


@pytest.mark.parametrize("cfg", ["0", "1"])
def test_orthogonalize_general_form(mx, cfg, monkeypatch):
    """The first product sums over the long side; those behind it work on what it left."""
    monkeypatch.setenv("MX_GEMM16_CONFIG", cfg)
    g = normal((1, 136, LONG), BF16, 5)
    times_out_and_recovers(mx, lambda o, s: mx.mx_orthogonalize(g, steps=3, out=o, dev_status=s), (1, 136, LONG), BF16)


@pytest.mark.parametrize("shape", [(1, 128, 6144), (3, 32, 7168), (2, 2000, 100), (1, 16, 64)], ids=str)
def test_orthogonalize_one_launch_form(mx, shape):
    """Its products take about as long as a wait's first look, so that a wait may
    or may not run out: either it is reported or the result is the usual one."""
    g = normal(shape, FP32, 6)
    want = mx.mx_orthogonalize(g, steps=16, coeffs=(1.5, -0.5, 0.0))
    for ns in (1, 200, 1000, 5000):
        for _ in range(5):
            out, intact = guarded(shape, BF16)
            status = torch.zeros(1, dtype=torch.int32, device="cuda")
            with limit(mx, ns):
                mx.mx_orthogonalize(g, steps=16, coeffs=(1.5, -0.5, 0.0), out=out, dev_status=status)
                torch.cuda.synchronize()
            assert intact()
            assert int(status.item()) == mx.MX_DEV_TIMEOUT or (int(status.item()) == 0 and torch.equal(out, want))
    assert torch.equal(mx.mx_orthogonalize(g, steps=16, coeffs=(1.5, -0.5, 0.0)), want)
