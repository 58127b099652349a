"""Sums of many values of one sign into 16 bits, against 64 bits, with a tolerance
that does not grow with their length.

The tensor core's accumulator truncates: each 16 terms may lose 2^-22 of the sum
so far (one truncated addition, doubled as in gemm16_util), always in one
direction.  The kernels therefore add what one accumulator holds of a long sum,
at most 2^15 terms of it, to FP32 sums that are rounded: the whole is off by
(2^15 / 16 + 16) 2^-22 of the sum and, for the rounded additions of up to 2^22 / 2^13
parts, 2^9 times 2^-24; on top the rounding of the result."""
import pytest
import torch

from gemm16_util import SENTINEL, U, close, guarded

pytestmark = pytest.mark.gpu

BF16, FP16, FP32 = torch.bfloat16, torch.float16, torch.float32
SUM_ERROR = (2 ** 15 / 16 + 16) * 2.0 ** -22 + 2.0 ** 9 * 2.0 ** -24


@pytest.fixture(scope="module")
def mx():
    import moe_grouped_gemm_mx_b200 as m
    return m


@pytest.fixture
def forced(monkeypatch):
    def force(cfg):
        if cfg is not None:
            monkeypatch.setenv("MX_GEMM16_CONFIG", cfg)
    return force


def positive(shape, dtype, seed, scale=1.0):
    """Values between half and one and a half times `scale`."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return ((torch.rand(shape, generator=gen, device="cuda") + 0.5) * scale).to(dtype)


def near(got, ref, what):
    u = U[got.dtype]
    close(got, ref, (u + SUM_ERROR * (1 + u)) * ref.abs(), what)


@pytest.mark.parametrize("cfg", [None, "0", "1", "2", "8"])
@pytest.mark.parametrize("rows,dtype", [(2 ** 15, FP16), (2 ** 15 + 1, FP16), (2 ** 20 + 37, FP16), (2 ** 22 + 5, BF16)],
                         ids=["2^15", "2^15+1", "2^20+37", "2^22+5-bf16"])
def test_weight_gradient(mx, forced, cfg, rows, dtype):
    forced(cfg)
    n, k = 72, 136
    x, dy = positive((rows, k), dtype, 1), positive((rows, n), dtype, 2, 2.0 ** -10)
    dw, intact = guarded((n, k), dtype)
    mx.mx_linear_act_backward(dy, x, None, dw=dw)
    near(dw, dy.double().T @ x.double(), f"dw over {rows}")
    assert intact()


@pytest.mark.parametrize("cfg", [None, "0", "1", "4"])
@pytest.mark.parametrize("parts", ["plain", "bias", "residual", "all"])
def test_linear(mx, forced, cfg, parts):
    """Every part of the epilogue behind a long sum; rows and columns that end inside a tile."""
    forced(cfg)
    m, n, k = 140, 328, 2 ** 20 + 24
    x, w = positive((m, k), FP16, 3), positive((n, k), FP16, 4, 2.0 ** -10)
    bias = positive((n,), FP16, 5, 100.0) if parts in ("bias", "all") else None
    residual = positive((m, n), FP16, 6, 100.0) if parts in ("residual", "all") else None
    y, intact_y = guarded((m, n), FP16)
    z, intact_z = guarded((m, n), FP16) if parts == "all" else (None, lambda: True)
    mx.mx_linear_act(x, w, bias=bias, residual=residual, activation="none" if parts == "plain" else "silu", y=y, z=z)
    ref = x.double() @ w.double().T + (0.0 if bias is None else bias.double())
    if z is not None:
        near(z, ref, "z")
    near(y, ref + (0.0 if residual is None else residual.double()), "y")  # silu of a thousand is the thousand
    assert intact_y() and intact_z()


def test_linear_in_place_residual(mx):
    m, n, k = 300, 520, 2 ** 16 + 8
    x, w, r = positive((m, k), BF16, 1), positive((n, k), BF16, 2, 2.0 ** -16), positive((m, n), BF16, 3)
    want = mx.mx_linear_act(x, w, residual=r)
    got = mx.mx_linear_act(x, w, residual=r, y=r)
    assert got is r and torch.equal(got, want)


@pytest.mark.parametrize("cfg", [None, "0", "1", "2"])
def test_ragged_forward_and_input_gradient(mx, forced, cfg):
    forced(cfg)
    counts, k, n = [33, 0, 290, 1], 2 ** 20 + 8, 136
    off = torch.tensor([3, 36, 36, 326, 327], dtype=torch.int32, device="cuda")
    rows = 330
    a, b = positive((rows, k), FP16, 1), positive((4, n, k), FP16, 2, 2.0 ** -10)
    for name, call, w in (("d", lambda out: mx.mx_grouped_gemm_ragged(a, b, off, d=out), b),
                          ("da", lambda out: mx.mx_grouped_gemm_ragged_dgrad(a, b.view(4, k, n), off, da=out),
                           b.view(4, k, n).transpose(1, 2))):
        out, intact = guarded((rows, n), FP16)
        out.fill_(SENTINEL)
        call(out)
        at = 3
        for e, c in enumerate(counts):
            if c:
                near(out[at:at + c], a[at:at + c].double() @ w[e].double().T, f"{name} of expert {e}")
            at += c
        assert bool((out[:3] == SENTINEL).all()) and bool((out[327:] == SENTINEL).all()) and intact()


@pytest.mark.parametrize("dtype,out_dtype", [(FP16, FP16), (BF16, BF16), (FP16, FP32)], ids=["fp16", "bf16", "fp32"])
def test_ragged_weight_gradient(mx, dtype, out_dtype):
    """Experts with none, few, tens of thousands and a million rows, rows outside the groups."""
    counts = [1, 2 ** 20 + 5, 0, 40007, 300, 2 ** 15, 8192, 8193, 16384, 16385]
    n, k = 264, 392
    rows = 7 + sum(counts) + 9
    off = torch.tensor([7 + sum(counts[:i]) for i in range(len(counts) + 1)], dtype=torch.int32, device="cuda")
    dd, a = positive((rows, n), dtype, 3, 2.0 ** -10), positive((rows, k), dtype, 4)
    for t in (dd, a):
        t[:7] = float("nan")
        t[-9:] = float("inf")
    db, intact = guarded((len(counts), n, k), out_dtype)
    mx.mx_grouped_gemm_ragged_wgrad(dd, a, off, db=db)
    at = 7
    for e, c in enumerate(counts):
        near(db[e], dd[at:at + c].double().T @ a[at:at + c].double(), f"expert {e} of {c} rows")
        at += c
    assert intact()


@pytest.mark.parametrize("dtype", [BF16, FP16], ids=["bf16", "fp16"])
def test_ragged_weight_gradient_in_32_bits(mx, dtype):
    """FP32 results add a part of 512 rows at a time: (512 / 16 + 16) 2^-22 of the sum for the
    parts, 2^-24 for each addition and the last rounding.  (One accumulator would lose 3e-5
    of 5003 rows, three times that.)  More tiles than CTA pairs, sums of one part and of
    many, ends inside a step of 16 in the first part and in later ones."""
    counts = [511, 512, 513, 0, 1024, 1025, 3, 5003, 2 ** 16 + 3, 1536]
    n, k = 1288, 1032
    first, rows = 5, 5 + sum(counts) + 4
    off = torch.tensor([first + sum(counts[:i]) for i in range(len(counts) + 1)], dtype=torch.int32, device="cuda")
    dd, a = positive((rows, n), dtype, 3, 0.125), positive((rows, k), dtype, 4)
    for t in (dd, a):
        t[:first] = float("nan")
        t[-4:] = float("inf")
    db, intact = guarded((len(counts), n, k), FP32)
    mx.mx_grouped_gemm_ragged_wgrad(dd, a, off, db=db)
    for e, c in enumerate(counts):
        at = first + sum(counts[:e])
        ref = dd[at:at + c].double().T @ a[at:at + c].double()
        tol = (512 / 16 + 16) * 2.0 ** -22 + (-(-c // 512) + 1) * 2.0 ** -24
        close(db[e], ref, tol * ref.abs(), f"expert {e} of {c} rows")
    assert intact()


def test_several_tiles_a_pair(mx):
    """More 256 x 256 tiles than CTA pairs: sums of one part and of several take turns in a pair's accumulators."""
    counts = [20000, 0, 300, 17001, 16384, 9000, 40003]
    n, k = 1288, 1032
    off = torch.tensor([sum(counts[:i]) for i in range(len(counts) + 1)], dtype=torch.int32, device="cuda")
    dd, a = positive((sum(counts), n), FP16, 3, 2.0 ** -10), positive((sum(counts), k), FP16, 4)
    db = mx.mx_grouped_gemm_ragged_wgrad(dd, a, off)
    for e, c in enumerate(counts):
        at = sum(counts[:e])
        near(db[e], dd[at:at + c].double().T @ a[at:at + c].double(), f"expert {e} of {c} rows")


@pytest.mark.parametrize("cfg", [None, "0", "1", "8"])
@pytest.mark.parametrize("shape", [(1, 1, 2 ** 20), (2, 2 ** 20 - 3, 1)], ids=str)
def test_orthogonalize_long_side(mx, forced, cfg, shape):
    """One row or column: its Gram matrix is one sum of squares, A = 1, and a step gives
    (a + b A + c A^2) X.  A sum too small by a part d, and A's rounding to FP16 (2^-11),
    change that factor by |b + 2 c| = 0.72 times them of 0.70; its own rounding to FP16 is
    2^-11 more.  X's roundings to BF16 (2^-8 at most) average out over a million
    elements, those of equal values among them apart: five times 2^-9 / 1000 is left for them."""
    forced(cfg)
    batch, m, n = shape
    gen = torch.Generator(device="cuda").manual_seed(7)
    g = torch.randn(shape, generator=gen, device="cuda").to(BF16)
    a, b, c = 3.4445, -4.7750, 2.0315
    got = mx.mx_orthogonalize(g, steps=1, coeffs=(a, b, c)).double()
    for i in range(batch):
        x = g[i].double()
        x = x / (torch.linalg.vector_norm(x) + 1e-7)
        ref = (a + b + c) * x
        assert float(torch.linalg.vector_norm(got[i] - ref) / torch.linalg.vector_norm(ref)) < 2.0 ** -8
        along = float((got[i] * ref).sum() / (ref * ref).sum()) - 1.0
        assert abs(along) <= 0.72 / 0.70 * (SUM_ERROR + 2.0 ** -11) + 2.0 ** -11 + 5.0 * 2.0 ** -9 / 1000, along
