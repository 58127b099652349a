"""mx_orthogonalize element by element, and the general form with many tiles for
each pair of CTAs.

An element may be off by its rounding to BF16 (2^-8 of it) and by what the other
roundings leave, which spreads over all elements alike: six times the root
mean square of the error of the method's model in test_orthogonalize.  (That
contains the rounding to BF16 and is about three times the rest of it: some
eighteen standard deviations, of a few million elements.)  An element that is wholly wrong is off by
its own size, a hundred times that."""
import pytest
import torch

from gemm16_util import guarded
from test_orthogonalize import COEFFS, check, exact, model, momentum

BF16, FP32 = torch.bfloat16, torch.float32
DTYPES = pytest.mark.parametrize("dtype", [BF16, FP32], ids=["bf16", "fp32"])


@pytest.fixture(scope="module")
def mx():
    import moe_grouped_gemm_mx_b200 as m
    return m


def check_elements(g, got, steps=5, what=""):
    coeffs = [COEFFS] * steps
    for i in range(g.shape[0]):
        ref = exact(g[i], coeffs, 1e-7)
        rms = float((model(g[i], coeffs, 1e-7) - ref).square().mean().sqrt())
        err = (got[i].double() - ref).abs()
        over = err - 2.0 ** -8 * ref.abs()
        assert bool(torch.isfinite(err).all()) and float(over.max()) <= 6.0 * rms, \
            f"{what} matrix {i}: {float(over.max()):.3g} over at {divmod(int(over.argmax()), ref.shape[1])}, rms {rms:.3g}"


def test_a_wrong_element_shows():
    """On the CPU: the model's own result with one element lost stays within the bound of the norm, not within this one."""
    gen = torch.Generator().manual_seed(1)
    g = torch.randn(1, 1024, 1792, generator=gen).to(BF16)
    got = model(g[0], [COEFFS] * 2, 1e-7)[None]
    check_elements(g, got, 2)
    at = (got[0].abs() - got[0].square().mean().sqrt()).abs().argmin()   # one of usual size
    got[0].view(-1)[at] = 0.0
    check(g, got, [COEFFS] * 2)
    with pytest.raises(AssertionError):
        check_elements(g, got, 2)


@pytest.mark.gpu
@DTYPES
@pytest.mark.parametrize("shape", [(2, 64, 1000), (1, 500, 128), (3, 264, 392), (1, 1024, 1792), (2, 769, 401)], ids=str)
def test_every_element(mx, shape, dtype):
    g = momentum(*shape, dtype, seed=2)
    check_elements(g, mx.mx_orthogonalize(g), what=str(shape))


@pytest.mark.gpu
@DTYPES
@pytest.mark.parametrize("cfg", ["0", "1", "2", "8"])
def test_every_kernel(mx, cfg, dtype, monkeypatch):
    monkeypatch.setenv("MX_ORTHO_CONFIG", "general")
    monkeypatch.setenv("MX_GEMM16_CONFIG", cfg)
    for shape in ((2, 300, 520), (1, 520, 296), (2, 71, 77), (1, 640, 641)):
        g = momentum(*shape, dtype, seed=3)
        check_elements(g, mx.mx_orthogonalize(g), what=f"{shape} {cfg}")


@pytest.mark.gpu
@DTYPES
@pytest.mark.parametrize("shape", [(2, 1537, 2561), (2, 2561, 1537), (3, 1288, 2304)], ids=str)
def test_many_tiles_a_pair(mx, shape, dtype, monkeypatch):
    """154 tiles and more over 74 pairs: a warp's staging tile, which holds C, then the low half, then
    the result, is used again by the next tile while the last store may still read it."""
    monkeypatch.setenv("MX_GEMM16_CONFIG", "0")
    g = momentum(*shape, dtype, seed=4)
    out, intact = guarded(shape, BF16)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    mx.mx_orthogonalize(g, out=out, dev_status=status)
    torch.cuda.synchronize()
    assert int(status.item()) == 0 and intact()
    check_elements(g, out, what=str(shape))
    check(g, out, [COEFFS] * 5, what=str(shape))
    assert torch.equal(mx.mx_orthogonalize(g), out)


@pytest.mark.gpu
def test_both_sides_longer_than_an_accumulator_takes(mx, monkeypatch):
    """Every product sums over more than 2^14: the epilogues behind parts of a sum, with C, its low half,
    the result's low half and the mirrored tiles."""
    m, n, steps = 16392, 16400, 4
    g = torch.randn(m, n, generator=torch.Generator(device="cuda").manual_seed(5), device="cuda")
    coeffs = [COEFFS] * steps
    ref = exact(g, coeffs, 1e-7)
    rms = float((model(g, coeffs, 1e-7) - ref).square_().mean().sqrt())
    for cfg in ("0", "1"):
        monkeypatch.setenv("MX_GEMM16_CONFIG", cfg)
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        got = mx.mx_orthogonalize(g, steps=steps, dev_status=status)
        assert int(status.item()) == 0
        err = got.double().sub_(ref).abs_()
        assert float(err.square().mean().sqrt()) <= 1.3 * rms
        assert float(err.sub_(ref.abs(), alpha=2.0 ** -8).max()) <= 6.0 * rms
