"""mx_orthogonalize where eps is much larger than the matrix: X starts at |G| / eps
and grows by a factor of |a| a step, down to ratios where no FP16 number could
hold it as it is.

What the result may be off by, of its norm, in the 64-bit iteration's terms: its
rounding to BF16 (of independent errors up to 2^-8 of each element the norm is at most
2^-8 / sqrt 3), in each of the last three steps the rounding of X to FP16 (2^-11 / sqrt 3)
and that of the product's factor (2^-11, the same for all elements); the steps
before them keep X to 22 bits."""
import math

import pytest
import torch

from gemm16_util import guarded

pytestmark = pytest.mark.gpu

BF16, FP32 = torch.bfloat16, torch.float32
COEFFS = (3.4445, -4.7750, 2.0315)
BOUND = 2.0 ** -8 / math.sqrt(3) + 3 * 2.0 ** -11 * (1 + 1 / math.sqrt(3))
RATIOS = [1.0, 0.1, 0.06, 1e-2, 1e-3, 1e-4, 5e-6, 5e-7, 1e-9, 1e-13, 1e-20, 1e-30]


@pytest.fixture(scope="module")
def mx():
    import moe_grouped_gemm_mx_b200 as m
    return m


def exact(g, coeffs, eps):
    x = g.double() / (torch.linalg.vector_norm(g.double()) + eps)
    flip = x.shape[0] > x.shape[1]
    x = x.T if flip else x
    for a, b, c in coeffs:
        p = x @ x.T
        px = p @ x
        x = a * x + b * px + c * (p @ px)
    return x.T if flip else x


def batch_of(shape, dtype, eps, ratios, seed):
    """One matrix for each ratio of norm to eps, a zero one behind them."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    m, n = shape
    g = torch.randn(len(ratios) + 1, m, n, generator=gen, device="cuda", dtype=torch.float64)
    g += 0.5 * torch.randn(len(ratios) + 1, m, 1, generator=gen, device="cuda", dtype=torch.float64)
    for i, r in enumerate(ratios):
        g[i] *= r * eps / torch.linalg.vector_norm(g[i])
    g[-1] = 0.0
    return g.to(dtype)


def check(mx, g, coeffs, eps):
    out, intact = guarded(g.shape, BF16)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    mx.mx_orthogonalize(g, steps=len(coeffs), coeffs=coeffs, eps=eps, out=out, dev_status=status)
    torch.cuda.synchronize()
    assert int(status.item()) == 0 and intact()
    for i in range(g.shape[0] - 1):
        ref = exact(g[i], coeffs, eps)
        off = float(torch.linalg.vector_norm(out[i].double() - ref) / torch.linalg.vector_norm(ref))
        assert off <= BOUND, f"ratio {RATIOS[i]}: {off:.3g} off, bound {BOUND:.3g}"
    assert bool((out[-1] == 0).all())


@pytest.mark.parametrize("form", ["", "general"])
@pytest.mark.parametrize("eps", [1e-7, 1.0], ids=str)
@pytest.mark.parametrize("dtype", [BF16, FP32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("shape", [(64, 520), (1000, 72), (33, 77), (264, 392), (301, 257)], ids=str)
def test_small_against_eps(mx, shape, dtype, eps, form, monkeypatch):
    monkeypatch.setenv("MX_ORTHO_CONFIG", form)
    check(mx, batch_of(shape, dtype, eps, RATIOS, 1), [COEFFS] * 5, eps)


@pytest.mark.parametrize("form", ["", "general"])
@pytest.mark.parametrize("steps", [1, 2, 3, 4])
def test_steps(mx, steps, form, monkeypatch):
    monkeypatch.setenv("MX_ORTHO_CONFIG", form)
    check(mx, batch_of((96, 200), BF16, 1.0, RATIOS, 2), [COEFFS] * steps, 1.0)


@pytest.mark.parametrize("form", ["", "general"])
@pytest.mark.parametrize("steps", [8, 12, 16])
def test_many_steps(mx, steps, form, monkeypatch):
    """Steps that bring X up from nothing.  The usual coefficients have |s p'(s) / p(s)| up
    to 2 where p(s) is near one, so that after that point each step of theirs may double
    an error; these have p'(1) = 0."""
    monkeypatch.setenv("MX_ORTHO_CONFIG", form)
    check(mx, batch_of((96, 200), BF16, 1.0, RATIOS, 2), [(1.875, -1.25, 0.375)] * steps, 1.0)


@pytest.mark.parametrize("form", ["", "general"])
def test_coefficients_that_shrink(mx, form, monkeypatch):
    """X falls by 8 in some steps and grows in others."""
    monkeypatch.setenv("MX_ORTHO_CONFIG", form)
    coeffs = [(0.125, 0.0, 0.0), (0.125, 0.0, 0.0), (3.0, -3.0, 1.0), (0.125, 0.01, 0.0), (3.8, 0.0, 0.0), (2.0, -1.5, 0.5)]
    check(mx, batch_of((72, 136), BF16, 1.0, RATIOS, 3), coeffs, 1.0)


@pytest.mark.parametrize("cfg", ["0", "1", "8"])
def test_every_kernel(mx, cfg, monkeypatch):
    monkeypatch.setenv("MX_ORTHO_CONFIG", "general")
    monkeypatch.setenv("MX_GEMM16_CONFIG", cfg)
    for dtype in (BF16, FP32):
        check(mx, batch_of((264, 520), dtype, 1.0, RATIOS, 4), [COEFFS] * 5, 1.0)


@pytest.mark.parametrize("form", ["", "general"])
def test_no_linear_term(mx, form, monkeypatch):
    """a = 0: a small X falls with its cube, past what the products can resolve.  The result stays
    finite; where it is large, each step triples an error and adds three FP16 roundings
    of its own (13 times 3 times 2^-11 in three steps), where it is small, FP16's smallest steps
    in A and B, held times 2^12, leave less than 1e-7 of X a step."""
    monkeypatch.setenv("MX_ORTHO_CONFIG", form)
    coeffs = [(0.0, 1.0, 0.0)] * 3
    g = batch_of((72, 136), BF16, 1.0, RATIOS, 5)
    got = mx.mx_orthogonalize(g, steps=3, coeffs=coeffs, eps=1.0).double()
    assert bool(torch.isfinite(got).all())
    for i, r in enumerate(RATIOS):
        ref = exact(g[i], coeffs, 1.0)
        off = float(torch.linalg.vector_norm(got[i] - ref))
        assert off <= (2.0 ** -8 + 39 * 2.0 ** -11) * float(torch.linalg.vector_norm(ref)) + 3e-7 * r, (r, off)
