"""mx_linear_act and its backward pass on the GPU against 64-bit references:
both kernels and every split of K, sizes around the tiles' edges, both types,
every activation, bias, residual and pre-activation, gradients against the
formulas and against differences, captured graphs and two streams at once."""
import contextlib
import os
import subprocess
import sys

import pytest
import torch

from gemm16_util import SENTINEL, U, TINY, act_ref, close, guarded, normal, product_tol, sum_error

pytestmark = pytest.mark.gpu

BF16, FP16 = torch.bfloat16, torch.float16
ACTS = ["none", "relu", "silu", "gelu", "gelu_tanh"]


@pytest.fixture(scope="module")
def mx():
    import moe_grouped_gemm_mx_b200 as m
    return m


@contextlib.contextmanager
def config(value):
    """Force a kernel (None: the library's choice)."""
    if value is None:
        yield
        return
    os.environ["MX_GEMM16_CONFIG"] = str(value)
    try:
        yield
    finally:
        del os.environ["MX_GEMM16_CONFIG"]


def forward_ref(x, w, bias, residual, act):
    """y, z and what each may be off by (u of the output type apart)."""
    xd, wd = x.double(), w.double()
    k = x.shape[1]
    z = xd @ wd.T
    mass = xd.abs() @ wd.abs().T
    if bias is not None:
        z = z + bias.double()
        mass = mass + bias.double().abs()
    dz = sum_error(k) * mass
    y = act_ref(z, act)[0]
    # no activation's slope exceeds 1.13; its own evaluation is within 2^-19 of |z|
    dy = 1.13 * dz + (2.0 ** -19 * (z.abs() + dz) if act != "none" else 0.0)
    if residual is not None:
        y = y + residual.double()
        dy = dy + 2.0 ** -23 * (y.abs() + residual.double().abs())
    return y, dy, z, dz


def check_forward(mx, m, n, k, dtype, act, bias=True, residual=True, want_z=True, seed=0):
    x = normal((m, k), dtype, seed)
    w = normal((n, k), dtype, seed + 1, k ** -0.5)
    b = normal((n,), dtype, seed + 2, 0.3) if bias else None
    r = normal((m, n), dtype, seed + 3) if residual else None
    y, y_intact = guarded((m, n), dtype)
    z, z_intact = guarded((m, n), dtype) if want_z else (None, lambda: True)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    mx.mx_linear_act(x, w, bias=b, residual=r, activation=act, z=z, y=y, dev_status=status)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    ry, dy, rz, dz = forward_ref(x, w, b, r, act)
    u = U[dtype]
    close(y, ry, u * ry.abs() + (1 + u) * dy + TINY[dtype], f"y {m}x{n}x{k} {act}")
    if want_z:
        close(z, rz, u * rz.abs() + (1 + u) * dz + TINY[dtype], f"z {m}x{n}x{k}")
    assert y_intact() and z_intact(), "wrote outside an output"


SMALL = [(1, 8, 8), (1, 2112, 1024), (2, 16, 24), (31, 40, 56), (64, 128, 64), (65, 136, 72), (128, 128, 128),
         (129, 264, 200), (255, 256, 136), (300, 520, 1032)]


@pytest.mark.parametrize("cfg", [0, 1, 2, 4, 8])
@pytest.mark.parametrize("shape", SMALL, ids=lambda s: "x".join(map(str, s)))
def test_forward_every_kernel(mx, cfg, shape):
    with config(cfg):
        check_forward(mx, *shape, BF16, "silu", seed=cfg)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("dtype", [BF16, FP16], ids=["bf16", "fp16"])
@pytest.mark.parametrize("cfg", [0, 2])
def test_forward_types_and_activations(mx, cfg, dtype, act):
    with config(cfg):
        check_forward(mx, 200, 392, 328, dtype, act)


@pytest.mark.parametrize("cfg", [0, 1, 4])
@pytest.mark.parametrize("parts", [(False, False, False), (True, False, False), (False, True, False), (False, False, True),
                                   (True, False, True), (False, True, True)], ids=str)
def test_forward_optional_parts(mx, cfg, parts):
    bias, residual, want_z = parts
    with config(cfg):
        check_forward(mx, 140, 280, 264, FP16, "gelu", bias, residual, want_z)


@pytest.mark.parametrize("shape", [(1, 2112, 7168), (64, 2112, 7168), (1037, 7168, 2048), (2050, 4104, 136), (4100, 2560, 520),
                                   (2560, 2568, 7168)], ids=lambda s: "x".join(map(str, s)))
def test_forward_as_chosen(mx, shape):
    """The library's own choice of kernel, up to several tiles per CTA pair."""
    check_forward(mx, *shape, BF16, "gelu_tanh", seed=5)


def test_forward_keeps_special_values(mx):
    """A NaN or an infinity in a row of x stays in that row; relu passes NaN on."""
    for cfg in (0, 2):
        with config(cfg):
            x = normal((300, 256), BF16, 1)
            w = normal((264, 256), BF16, 2, 0.1)
            clean = mx.mx_linear_act(x, w, activation="relu")
            x[7, 3] = float("nan")
            x[140, 200] = float("inf")
            y = mx.mx_linear_act(x, w, activation="relu")
            assert bool(torch.isnan(y[7]).all())
            assert not bool(torch.isfinite(y[140]).all())
            rest = torch.ones(300, dtype=torch.bool)
            rest[[7, 140]] = False
            assert torch.equal(y[rest], clean[rest])


def test_forward_in_place_residual(mx):
    for cfg in (0, 4):
        with config(cfg):
            x, w, r = normal((333, 264), BF16, 1), normal((520, 264), BF16, 2, 0.06), normal((333, 520), BF16, 3)
            want = mx.mx_linear_act(x, w, residual=r, activation="silu")
            got = mx.mx_linear_act(x, w, residual=r, activation="silu", y=r)
            assert got is r and torch.equal(got, want)


@pytest.mark.parametrize("cfg", [1, 2, 8])
@pytest.mark.parametrize("shape", [(129, 136, 264), (333, 520, 520)], ids=lambda s: "x".join(map(str, s)))
def test_forward_in_place_residual_by_tile(mx, cfg, shape):
    """The same where other lanes store than those that read the residual."""
    m, n, k = shape
    with config(cfg):
        x, w, r = normal((m, k), FP16, 1), normal((n, k), FP16, 2, 0.06), normal((m, n), FP16, 3)
        want = mx.mx_linear_act(x, w, residual=r, activation="gelu")
        got = mx.mx_linear_act(x, w, residual=r, activation="gelu", y=r)
        assert got is r and torch.equal(got, want)


def test_results_do_not_vary(mx):
    """The same call gives the same bits (split sums meet in a fixed order)."""
    for cfg in (0, 8):
        with config(cfg):
            x, w = normal((70, 4096), BF16, 1), normal((1032, 4096), BF16, 2, 0.02)
            first = mx.mx_linear_act(x, w)
            for _ in range(10):
                assert torch.equal(mx.mx_linear_act(x, w), first)


# ---------------------------------------------------------------- backward

def check_backward(mx, m, n, k, dtype, act, seed=0, bias=True):
    x = normal((m, k), dtype, seed)
    w = normal((n, k), dtype, seed + 1, k ** -0.5)
    z = normal((m, n), dtype, seed + 2, 2.0)
    dy = normal((m, n), dtype, seed + 3, 0.1)
    dx, ix = guarded((m, k), dtype)
    dw, iw = guarded((n, k), dtype)
    db, ib = guarded((n,), dtype)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    mx.mx_linear_act_backward(dy, x, w, z=z if act != "none" else None, activation=act, dx=dx, dw=dw,
                              dbias=db if bias else None, dev_status=status)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    u = U[dtype]
    zd, g = z.double(), dy.double()
    dz = g * act_ref(zd, act)[1]
    # act' is evaluated to 2^-18 (1 + |z|); dz is rounded once before the products
    slope_err = g.abs() * 2.0 ** -18 * (1 + zd.abs()) if act != "none" else torch.zeros_like(g)
    dz_err = slope_err + (u * dz.abs() + TINY[dtype] if act != "none" else 0.0)
    xd, wd = x.double(), w.double()
    rx, rw, rb = dz @ wd, dz.T @ xd, dz.sum(0)
    close(dx, rx, product_tol(rx, dz.abs() @ wd.abs(), n, dtype) + 1.01 * (dz_err @ wd.abs()), f"dx {m}x{n}x{k} {act}")
    close(dw, rw, product_tol(rw, dz.abs().T @ xd.abs(), m, dtype) + 1.01 * (dz_err.T @ xd.abs()),
          f"dw {m}x{n}x{k} {act}")
    if bias:
        # FP32 sums in chunks: m additions at most, 2^-24 of the sum of magnitudes each
        tol = u * rb.abs() + 1.01 * (slope_err.sum(0) + (m + 64) * 2.0 ** -24 * dz.abs().sum(0)) + TINY[dtype]
        close(db, rb, tol, f"dbias {m}x{n} {act}")
    assert ix() and iw() and ib(), "wrote outside an output"


@pytest.mark.parametrize("cfg", [None, 0, 1, 4])
@pytest.mark.parametrize("shape", [(1, 8, 8), (7, 64, 128), (128, 128, 128), (129, 136, 264), (333, 1000, 776), (70, 520, 72)],
                         ids=lambda s: "x".join(map(str, s)))
def test_backward(mx, cfg, shape):
    with config(cfg):
        check_backward(mx, *shape, BF16, "gelu")


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("dtype", [BF16, FP16], ids=["bf16", "fp16"])
def test_backward_types_and_activations(mx, dtype, act):
    check_backward(mx, 515, 264, 392, dtype, act)


def test_backward_large(mx):
    check_backward(mx, 4100, 2568, 1032, BF16, "silu")


def test_backward_parts(mx):
    """Frozen weights, no input gradient, gradients into given tensors, dz handed out."""
    x, w = normal((200, 136), BF16, 1), normal((72, 136), BF16, 2)
    z, dy = normal((200, 72), BF16, 3), normal((200, 72), BF16, 4)
    dx, dw, db = mx.mx_linear_act_backward(dy, x, w, z=z, activation="relu", bias_grad=True)
    only_x = mx.mx_linear_act_backward(dy, None, w, z=z, activation="relu")
    only_w = mx.mx_linear_act_backward(dy, x, None, z=z, activation="relu")
    assert only_x[1] is None and only_x[2] is None and torch.equal(only_x[0], dx)
    assert only_w[0] is None and only_w[2] is None and torch.equal(only_w[1], dw)
    dz = torch.empty_like(dy)
    again = mx.mx_linear_act_backward(dy, x, w, z=z, activation="relu", bias_grad=True, dz=dz)
    assert torch.equal(dz, torch.where(z > 0, dy, torch.zeros_like(dy)))
    assert all(torch.equal(a, b) for a, b in zip(again, (dx, dw, db)))


def test_empty(mx):
    x, w = torch.empty((0, 64), dtype=BF16, device="cuda"), normal((32, 64), BF16, 1)
    assert mx.mx_linear_act(x, w).shape == (0, 32)
    dx, dw, db = mx.mx_linear_act_backward(torch.empty((0, 32), dtype=BF16, device="cuda"), x, w, bias_grad=True)
    assert dx.shape == (0, 64) and bool((dw == 0).all()) and bool((db == 0).all())
    w0 = torch.empty((0, 64), dtype=BF16, device="cuda")
    dx, dw, _ = mx.mx_linear_act_backward(torch.empty((5, 0), dtype=BF16, device="cuda"), normal((5, 64), BF16, 2), w0)
    assert bool((dx == 0).all()) and dw.shape == (0, 64)


@pytest.mark.parametrize("act", ACTS)
def test_gradient_against_differences(mx, act):
    """The backward pass against central differences of the 64-bit forward at the
    16-bit inputs: L = sum(c * y), along random directions.  z is the 64-bit
    pre-activation rounded to FP16, as the forward keeps it; its rounding moves
    act' by at most 2^-11 |z| max|act''| (under 1.2 for every smooth one).  relu's
    kink is kept away from: every |z| is at least 2^-6."""
    m, n, k = 24, 40, 48
    x, w, b = normal((m, k), FP16, 1), normal((n, k), FP16, 2, 0.2), normal((n,), FP16, 3, 0.3)
    c = normal((m, n), FP16, 4)

    def value(xd, wd, bd):
        return (c.double() * act_ref(xd @ wd.T + bd, act)[0]).sum().item()

    zd = x.double() @ w.double().T + b.double()
    if act == "relu":
        c = torch.where(zd.abs() >= 2.0 ** -6, c, torch.zeros_like(c))
    dx, dw, db = mx.mx_linear_act_backward(c, x, w, z=zd.to(FP16), activation=act, bias_grad=True)
    dz = c.double().abs() * 1.13
    h = 1e-5
    for i, (t, got) in enumerate(((x, dx), (w, dw), (b, db))):
        d = normal(t.shape, torch.float32, 10 + i).double()
        args = [x.double(), w.double(), b.double()]
        args[i] = args[i] + h * d
        up = value(*args)
        args[i] = args[i] - 2 * h * d
        down = value(*args)
        want = (up - down) / (2 * h)
        have = (got.double() * d).sum().item()
        # each element's error: its own rounding, dz's rounding and z's rounding
        per = dz * 2.0 ** -11 + c.double().abs() * 1.2 * 2.0 ** -11 * (zd.abs() + 1)
        spread = (per @ w.double().abs(), per.T @ x.double().abs(), per.sum(0))[i]
        tol = ((spread + 2.0 ** -11 * got.double().abs() + 2.0 ** -13) * d.abs()).sum().item() + 1e-6 * abs(want)
        assert abs(have - want) <= tol, (act, i, have, want, tol)


# ---------------------------------------------------------------- streams and graphs

def test_captured_and_replayed(mx):
    """Forward and backward captured into one graph, replayed on new inputs,
    beside an uncaptured call of the same tensors."""
    m, n, k = 200, 264, 136
    x, w, b = normal((m, k), BF16, 1), normal((n, k), BF16, 2, 0.1), normal((n,), BF16, 3)
    dy = normal((m, n), BF16, 4)

    def step():
        y, z = mx.mx_linear_act(x, w, bias=b, activation="gelu", return_z=True)
        return (y, z) + tuple(mx.mx_linear_act_backward(dy, x, w, z=z, activation="gelu", bias_grad=True))

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for seed in (20, 30):
        x.copy_(normal((m, k), BF16, seed))
        dy.copy_(normal((m, n), BF16, seed + 1))
        graph.replay()
        want = step()
        torch.cuda.synchronize()
        for got, ref in zip(out, want):
            assert torch.equal(got, ref)


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("act", ["relu", "silu", "gelu", "gelu_tanh"])
def test_activations_over_the_whole_range(mx, dtype, act):
    """y and dz for z from the type's smallest to its largest numbers.  A product
    with one term is exact, so z is.  y is off by its rounding and 2^-19 |z| (the
    activation's evaluation), dz by its rounding and 2^-19 (the derivative's, at
    most 1.13 large); results below 2^-126 may become zero."""
    top = torch.finfo(dtype).max
    e = torch.arange(-24 if dtype is FP16 else -120, 15 if dtype is FP16 else 127, dtype=torch.float64)
    mags = torch.cat([torch.zeros(1, dtype=torch.float64), 2.0 ** e, 1.375 * 2.0 ** e[2:-1],
                      torch.tensor([top, 5.5, 9.0, 13.0, 30.0, 100.0], dtype=torch.float64)])
    mags = mags.to(dtype)
    vals = torch.cat([mags, -mags])
    vals = torch.cat([vals, vals.new_zeros((-len(vals)) % 8)]).cuda()
    n = len(vals)
    x = torch.zeros(1, 8, dtype=dtype, device="cuda")
    x[0, 0] = 1
    w = torch.zeros(n, 8, dtype=dtype, device="cuda")
    w[:, 0] = vals
    y, z = mx.mx_linear_act(x, w, activation=act, return_z=True)
    assert torch.equal(z[0], vals)
    zd = vals.double()
    inner = zd.clamp(-1e4, 1e4)  # (beyond it every activation is z or 0, its slope 1 or 0)
    ref, slope = act_ref(inner, act)
    ref = torch.where(zd > 1e4, zd, torch.where(zd < -1e4, torch.zeros_like(zd), ref))
    u = U[dtype]
    close(y[0], ref, u * ref.abs() + 2.0 ** -19 * zd.abs() + TINY[dtype] + 2.0 ** -126, f"y {act}")
    dz = torch.empty(1, n, dtype=dtype, device="cuda")
    mx.mx_linear_act_backward(torch.ones(1, n, dtype=dtype, device="cuda"), x, None, z=z, activation=act, dz=dz)
    close(dz[0], slope, u * slope.abs() + 2.0 ** -19 + TINY[dtype], f"dz {act}")


def test_relu_passes_on_what_a_nan_gets(mx):
    z = torch.tensor([[float("nan"), 1.0, -1.0, 0.0, float("inf"), float("-inf"), -0.0, 2.0]], dtype=BF16, device="cuda")
    dy = torch.arange(1, 9, dtype=torch.float32, device="cuda").to(BF16).view(1, 8)
    dz = torch.empty_like(dy)
    mx.mx_linear_act_backward(dy, torch.ones(1, 8, dtype=BF16, device="cuda"), None, z=z, activation="relu", dz=dz)
    assert dz[0].tolist() == [1, 2, 0, 0, 5, 0, 0, 8]


FIRST_CALL = """
import sys
import torch
import moe_grouped_gemm_mx_b200 as mx
torch.manual_seed(0)
x = torch.randn(256, 512, device="cuda").bfloat16()
w = torch.randn(264, 512, device="cuda").bfloat16()
b = torch.randn(4, 264, 512, device="cuda").bfloat16()
off = torch.tensor([0, 60, 60, 200, 256], dtype=torch.int32, device="cuda")
g = torch.randn(2, 32, 700, device="cuda")
calls = {
    "linear": lambda: [mx.mx_linear_act(x, w, activation="silu")],
    "backward": lambda: list(mx.mx_linear_act_backward(x @ w.T, x, w, bias_grad=True)),
    "ragged": lambda: [mx.mx_grouped_gemm_ragged(x, b, off)],
    "wgrad": lambda: [mx.mx_grouped_gemm_ragged_wgrad(x, x, off, out_dtype=torch.float32)],
    "orthogonalize": lambda: [mx.mx_orthogonalize(g)],
    "general": lambda: [mx.mx_orthogonalize(x)],
}
call = calls[sys.argv[1]]
x @ w.T  # the library's own handles exist before the capture
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    got = call()
graph.replay()
torch.cuda.synchronize()
assert mx.read_internal_status() == 0
for a, e in zip(got, call()):
    assert torch.equal(a, e), (a - e).abs().max()
print("ok")
"""


@pytest.mark.parametrize("which", ["linear", "backward", "ragged", "wgrad", "orthogonalize", "general"])
def test_first_call_of_a_process_is_captured(mx, which):
    """What a first call sets up on the host (kernel attributes, the internal
    status word, what the choice of a kernel asks the device) is allowed in a capture."""
    done = subprocess.run([sys.executable, "-c", FIRST_CALL, which], capture_output=True, text=True, timeout=300,
                          cwd=os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
    assert done.returncode == 0 and "ok" in done.stdout, done.stdout[-2000:] + done.stderr[-2000:]


def test_two_streams_at_once(mx):
    """Calls on two streams at the same time, workspaces of their own, give what
    one after the other gives."""
    data = [(normal((900, 520), BF16, s), normal((1032, 520), BF16, s + 1, 0.05), normal((900, 1032), BF16, s + 2)) for s in (1, 7)]

    def go(d, stream=None):
        y, z = mx.mx_linear_act(d[0], d[1], activation="silu", return_z=True, stream=stream)
        return (y,) + tuple(mx.mx_linear_act_backward(d[2], d[0], d[1], z=z, activation="silu", bias_grad=True, stream=stream))

    want = [go(d) for d in data]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in data]
    for _ in range(5):
        got = [[go(d, s) for _ in range(3)] for d, s in zip(data, streams)]
        torch.cuda.synchronize()
        for runs, ref in zip(got, want):
            for run in runs:
                assert all(torch.equal(a, b) for a, b in zip(run, ref))


def test_stream_by_pointer(mx):
    """The stream may be a raw pointer, and what the call allocates belongs to it."""
    x, w = normal((300, 264), BF16, 1), normal((136, 264), BF16, 2, 0.1)
    want = mx.mx_linear_act(x, w, activation="silu")
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = [mx.mx_linear_act(x, w, activation="silu", stream=side.cuda_stream) for _ in range(20)]
    torch.cuda.synchronize()
    assert all(torch.equal(g, want) for g in got)


def test_wait_timeout_reported(mx):
    """A wait bound far below the kernels' legitimate waits: the call reports
    MX_DEV_TIMEOUT, writes nothing outside its output and leaves the context
    usable."""
    x, w = normal((256, 65536 * 4), BF16, 1), normal((512, 65536 * 4), BF16, 2, 0.002)
    for cfg in (0, 1):
        with config(cfg):
            y, intact = guarded((256, 512), BF16)
            status = torch.zeros(1, dtype=torch.int32, device="cuda")
            mx.mx_set_wait_limit_ns(1000)
            try:
                mx.mx_linear_act(x, w, y=y, dev_status=status)
                torch.cuda.synchronize()
            finally:
                mx.mx_set_wait_limit_ns(0)
            assert int(status.item()) & mx.MX_DEV_TIMEOUT and intact()
            status.zero_()
            mx.mx_linear_act(x, w, y=y, dev_status=status)
            torch.cuda.synchronize()
            assert int(status.item()) == 0 and intact()
            ref = x.double() @ w.double().T
            close(y, ref, product_tol(ref, x.double().abs() @ w.double().abs().T, x.shape[1], BF16), "after the timeout")


def test_more_elements_than_32_bits_count(mx):
    """An output of 2.4e9 elements: rows behind the 2^31st element are right, in the
    forward pass and in dz (the residual, the pre-activation and the bias sums cross it too)."""
    m, n, k = 600 * 1024 + 8, 4096, 64
    x, w, b = normal((m, k), BF16, 1), normal((n, k), BF16, 2, 0.125), normal((n,), BF16, 3)
    r = torch.empty((m, n), dtype=BF16, device="cuda").fill_(0.5)
    y, z = mx.mx_linear_act(x, w, bias=b, residual=r, activation="relu", return_z=True)
    rows = torch.tensor([0, 1, 524286, 524287, 524288, 524289, m - 130, m - 1], device="cuda")
    ry, dy, rz, dz = forward_ref(x[rows], w, b, r[rows], "relu")
    close(y[rows], ry, U[BF16] * ry.abs() + 1.01 * dy, "y")
    close(z[rows], rz, U[BF16] * rz.abs() + 1.01 * dz, "z")
    del r
    g = y                      # any gradient: the outputs themselves
    dzt = torch.empty_like(z)
    dx, dw, db = mx.mx_linear_act_backward(g, x, w, z=z, activation="relu", bias_grad=True, dz=dzt)
    assert torch.equal(dzt[rows], torch.where(z[rows] > 0, g[rows], torch.zeros_like(g[rows])))
    ref = dzt[rows].double() @ w.double()
    close(dx[rows], ref, product_tol(ref, dzt[rows].double().abs() @ w.double().abs(), n, BF16), "dx")
    cols = torch.tensor([0, 7, 2048, 4095], device="cuda")
    sub = dzt[:, cols].double()
    ref = sub.T @ x.double()
    close(dw[cols], ref, product_tol(ref, sub.abs().T @ x.double().abs(), m, BF16), "dw")
    ref = sub.sum(0)
    close(db[cols], ref, U[BF16] * ref.abs() + (m + 64) * 2.0 ** -24 * sub.abs().sum(0), "dbias")


def test_empty_setting_is_no_setting(mx, monkeypatch):
    x, w = normal((70, 520), BF16, 1), normal((264, 520), BF16, 2, 0.05)
    want = mx.mx_linear_act(x, w)
    monkeypatch.setenv("MX_GEMM16_CONFIG", "")
    assert torch.equal(mx.mx_linear_act(x, w), want)
    monkeypatch.setenv("MX_GEMM16_CONFIG", "no")
    assert torch.equal(mx.mx_linear_act(x, w), want)


def test_python_refusals(mx):
    x, w = normal((16, 64), BF16, 1), normal((32, 64), BF16, 2)
    with pytest.raises(TypeError):
        mx.mx_linear_act(x.float(), w)
    with pytest.raises(TypeError):
        mx.mx_linear_act(x, w.half())
    with pytest.raises(ValueError):
        mx.mx_linear_act(x, w[:, :32].contiguous())
    with pytest.raises(ValueError):
        mx.mx_linear_act(x.t(), w)
    with pytest.raises(ValueError):
        mx.mx_linear_act(x, w, activation="tanh")
    with pytest.raises(ValueError):
        mx.mx_linear_act(x, w, bias=torch.zeros(31, dtype=BF16, device="cuda"))
    with pytest.raises(ValueError):
        mx.mx_linear_act(x.cpu(), w)
    with pytest.raises(ValueError):                                                 # dz without an activation
        mx.mx_linear_act_backward(normal((16, 32), BF16, 3), x, w, dz=normal((16, 32), BF16, 3))
    with pytest.raises(mx.MXError):
        mx.mx_linear_act(normal((16, 60), BF16, 1), normal((32, 60), BF16, 2))      # k % 8
    with pytest.raises(mx.MXError):
        mx.mx_linear_act(x, normal((30, 64), BF16, 2))                              # n % 8
    with pytest.raises(ValueError):
        mx.mx_linear_act_backward(normal((16, 32), BF16, 3), x, w, activation="relu")  # no z
    with pytest.raises(mx.MXError):
        mx.mx_linear_act_backward(normal((1100, 32), BF16, 3), normal((1100, 64), BF16, 1), w, bias_grad=True,
                                  workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
