"""mx_orthogonalize on the GPU against the iteration in 64 bits.

What the result may be off by: the same iteration is run in 64 bits with every
rounding that the method makes (FP16 operands held times powers of two, X as a
sum of two FP16 numbers while three or more steps follow, BF16 at the end), and its distance from
the exact one is the method's own error on that input.  A kernel's roundings
fall differently (its FP32 sums move values across rounding borders) but have
the same size, so its Frobenius error may be 1.3 times the model's; a matrix of
few elements, whose error is no average, gets one BF16 half step (2^-8) and as
much again on top."""
import math

import pytest
import torch

from gemm16_util import guarded, normal

pytestmark = pytest.mark.gpu

BF16, FP32 = torch.bfloat16, torch.float32
COEFFS = (3.4445, -4.7750, 2.0315)


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


def model(g, coeffs, eps):
    """The iteration with the method's roundings."""
    def fp16(v, scale):
        return (v * scale).to(torch.float16).double() / scale

    gd = g.double()
    f = float(torch.linalg.vector_norm(gd)) + eps
    flip = gd.shape[0] > gd.shape[1]
    gd = gd.T if flip else gd
    sx = 2.0 ** round(0.5 * math.log2(gd.shape[1]))
    two = 2.0 ** math.floor(math.log2(f))
    hi = fp16(gd / two, sx)
    low = fp16(gd / two - hi, sx) if g.dtype == FP32 else torch.zeros_like(hi)
    hi, low = hi * two / f, low * two / f
    has_low = g.dtype == FP32
    steps = len(coeffs)
    for i, (a, b, c) in enumerate(coeffs):
        p = fp16(hi @ hi.T, 4096.0)
        low_out = i < steps - 3
        if has_low or low_out:
            x = a * (hi + low) + fp16(b * p + c * (p @ p), 4096.0) @ hi
        else:
            x = fp16(a * torch.eye(p.shape[0], dtype=torch.float64, device=p.device) + b * p + c * (p @ p), 4096.0) @ hi
        hi = fp16(x, sx)
        low = fp16(x - hi, sx) if low_out else torch.zeros_like(hi)
        has_low = low_out
    x = x.to(BF16).double()
    return x.T if flip else x


def momentum(batch, m, n, dtype, seed, scale=1e-3):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    r = max(1, min(m, n) // 8)
    g = torch.randn(batch, m, r, generator=gen, device="cuda") @ torch.randn(batch, r, n, generator=gen, device="cuda")
    return ((g / r ** 0.5 + 0.3 * torch.randn(batch, m, n, generator=gen, device="cuda")) * scale).to(dtype)


def check(g, got, coeffs, eps=1e-7, what=""):
    gs, os = (g, got) if g.dim() == 3 else (g[None], got[None])
    for i in range(gs.shape[0]):
        ref = exact(gs[i], coeffs, eps)
        norm = torch.linalg.vector_norm(ref)
        own = float(torch.linalg.vector_norm(model(gs[i], coeffs, eps) - ref) / norm)
        off = float(torch.linalg.vector_norm(os[i].double() - ref) / norm)
        bound = 1.3 * own + (2.0 ** -7 if ref.numel() < 1024 else 0.0)
        assert off <= bound, f"{what} matrix {i}: {off:.3g} off, the method's own error is {own:.3g}"


SHAPES = [(1, 1, 1), (1, 1, 40), (1, 40, 1), (2, 3, 5), (1, 16, 16), (3, 24, 200), (2, 200, 24), (1, 127, 129), (2, 128, 128),
          (1, 129, 257), (2, 264, 136), (1, 333, 1000), (3, 257, 77), (1, 32, 7168)]


@pytest.mark.parametrize("dtype", [BF16, FP32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_shapes(mx, shape, dtype):
    g = momentum(*shape, dtype, seed=1)
    out, intact = guarded(shape, BF16)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    mx.mx_orthogonalize(g, out=out, dev_status=status)
    torch.cuda.synchronize()
    assert int(status.item()) == 0 and intact()
    check(g, out, [COEFFS] * 5, what=str(shape))


EDGES = [(1, 16, 64), (1, 17, 65), (1, 2, 128), (2, 64, 129), (1, 65, 385), (1, 128, 768), (1, 127, 1025), (1, 64, 7168),
         (1, 128, 6144), (1, 128, 6145), (1, 33, 7169), (20, 40, 700), (3, 1000, 128), (1, 3000, 100), (40, 128, 96),
         (3, 31, 7167), (5, 7, 9), (2, 50, 1001), (2, 50, 1002), (2, 50, 1004), (3, 5, 67), (4, 129, 63), (1, 3, 449)]


@pytest.mark.parametrize("dtype", [BF16, FP32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("shape", EDGES, ids=lambda s: "x".join(map(str, s)))
def test_one_launch_form(mx, shape, dtype, monkeypatch):
    """Around the sizes where the matrix just fits a cluster, both orientations,
    more matrices than clusters; the general form gives the same within both errors."""
    g, _ = guarded(shape, dtype)               # what lies next to the matrices is not theirs
    g.copy_(momentum(*shape, dtype, seed=21))
    out, intact = guarded(shape, BF16)
    mx.mx_orthogonalize(g, out=out)
    torch.cuda.synchronize()
    assert intact()
    check(g, out, [COEFFS] * 5, what=str(shape))
    monkeypatch.setenv("MX_ORTHO_CONFIG", "general")
    check(g, mx.mx_orthogonalize(g), [COEFFS] * 5, what=f"{shape} general")


@pytest.mark.parametrize("dtype", [BF16, FP32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_shapes_general_form(mx, shape, dtype, monkeypatch):
    monkeypatch.setenv("MX_ORTHO_CONFIG", "general")
    g = momentum(*shape, dtype, seed=1)
    out, intact = guarded(shape, BF16)
    mx.mx_orthogonalize(g, out=out)
    torch.cuda.synchronize()
    assert intact()
    check(g, out, [COEFFS] * 5, what=str(shape))


@pytest.mark.parametrize("cfg", ["0", "1", "4"])
def test_every_kernel(mx, cfg, monkeypatch):
    monkeypatch.setenv("MX_ORTHO_CONFIG", "general")
    monkeypatch.setenv("MX_GEMM16_CONFIG", cfg)
    for shape in ((2, 300, 520), (1, 520, 296), (2, 71, 77), (1, 640, 641)):
        for dtype in (BF16, FP32):
            g = momentum(*shape, dtype, seed=2)
            check(g, mx.mx_orthogonalize(g), [COEFFS] * 5, what=f"{shape} {cfg}")


@pytest.mark.parametrize("shape", [(2, 1024, 1792), (1, 2056, 1032), (4, 768, 768)], ids=str)
def test_large(mx, shape):
    g = momentum(*shape, BF16, seed=3)
    check(g, mx.mx_orthogonalize(g), [COEFFS] * 5)


@pytest.mark.parametrize("steps", [1, 2, 3, 4, 6, 8])
@pytest.mark.parametrize("dtype", [BF16, FP32], ids=["bf16", "fp32"])
def test_steps(mx, steps, dtype):
    g = momentum(1, 136, 200, dtype, seed=4)
    check(g, mx.mx_orthogonalize(g, steps=steps), [COEFFS] * steps)


def test_coefficients_per_step(mx):
    coeffs = [(3.9, -8.0, 4.9), (3.4445, -4.7750, 2.0315), (1.875, -1.25, 0.375), (1.5, -0.5, 0.0)]
    g = momentum(2, 96, 160, BF16, seed=5)
    check(g, mx.mx_orthogonalize(g, steps=4, coeffs=coeffs), coeffs)


def test_two_dimensions_in_place_and_workspace(mx):
    g = momentum(1, 136, 264, BF16, seed=6)[0].contiguous()
    want = mx.mx_orthogonalize(g)
    assert want.shape == g.shape
    need = mx.mx_orthogonalize_workspace_bytes(1, 136, 264)
    big = torch.full((need + 512,), 0x5A, dtype=torch.uint8, device="cuda")
    at = (256 - big.data_ptr() % 256) % 256
    view = big[at:at + need]
    got = mx.mx_orthogonalize(g, workspace=view)
    assert torch.equal(got, want) and bool((big[:at] == 0x5A).all()) and bool((big[at + need:] == 0x5A).all())
    assert torch.equal(mx.mx_orthogonalize(g, out=g), want)


@pytest.mark.parametrize("form", ["", "general"])
@pytest.mark.parametrize("shape", [(64, 136), (136, 64), (60, 77), (136, 140)], ids=str)
def test_special_matrices(mx, shape, form, monkeypatch):
    """Zeros give zeros; a NaN or an infinity spoils its own matrix only; norms at
    the ends of the types' ranges."""
    monkeypatch.setenv("MX_ORTHO_CONFIG", form)
    g = momentum(6, *shape, FP32, seed=7, scale=1.0)
    g[1] = 0.0
    g[2, 3, 5] = float("nan")
    g[3, 0, 0] = float("inf")
    g[4] *= 1e30
    g[5] *= 1e-30
    got = mx.mx_orthogonalize(g, eps=0.0)
    assert bool((got[1] == 0).all())
    assert bool(torch.isnan(got[2]).all()) and bool(torch.isnan(got[3]).all())
    check(g[0], got[0], [COEFFS] * 5, 0.0)
    check(g[4], got[4], [COEFFS] * 5, 0.0, "huge")
    check(g[5], got[5], [COEFFS] * 5, 0.0, "tiny")
    small = momentum(1, *shape, BF16, seed=8, scale=1e-9)      # eps counts
    check(small, mx.mx_orthogonalize(small), [COEFFS] * 5)


def test_strong_and_weak_directions(mx):
    """Singular values four decades apart: where a method that rounds X to 11 bits
    at every step is off by percents."""
    gen = torch.Generator(device="cuda").manual_seed(9)
    m, n = 256, 512
    strong = torch.randn(m, 4, generator=gen, device="cuda") @ torch.randn(4, n, generator=gen, device="cuda")
    g = (strong + 0.003 * torch.randn(m, n, generator=gen, device="cuda")).to(BF16)
    got = mx.mx_orthogonalize(g)
    check(g, got, [COEFFS] * 5)
    ref = exact(g, [COEFFS] * 5, 1e-7)
    assert float(torch.linalg.vector_norm(got.double() - ref) / torch.linalg.vector_norm(ref)) < 4e-3


def test_batch_is_independent_and_repeatable(mx):
    g = momentum(5, 200, 328, BF16, seed=10)
    first = mx.mx_orthogonalize(g)
    for _ in range(5):
        assert torch.equal(mx.mx_orthogonalize(g), first)
    order = torch.tensor([3, 1, 4, 0, 2], device="cuda")
    assert torch.equal(mx.mx_orthogonalize(g[order].contiguous()), first[order])


def test_captured_and_two_streams(mx):
    g = momentum(2, 136, 264, BF16, seed=11)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        mx.mx_orthogonalize(g)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = mx.mx_orthogonalize(g)
    for seed in (12, 13):
        g.copy_(momentum(2, 136, 264, BF16, seed=seed))
        graph.replay()
        assert torch.equal(out, mx.mx_orthogonalize(g))
    data = [momentum(2, 520, 648, BF16, seed=s) for s in (14, 15)]
    want = [mx.mx_orthogonalize(d) for d in data]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in data]
    got = [[mx.mx_orthogonalize(d, stream=s) for _ in range(4)] for d, s in zip(data, streams)]
    torch.cuda.synchronize()
    assert all(torch.equal(r, w) for runs, w in zip(got, want) for r in runs)


def test_more_elements_than_32_bits_count(mx):
    """A batch of 2.2e9 elements: its last matrices are right."""
    batch, m, n = 66, 4096, 8192
    g = torch.empty((batch, m, n), dtype=BF16, device="cuda").fill_(1e-3)
    g[0] = momentum(1, m, n, BF16, seed=31)[0]
    g[-1] = momentum(1, m, n, BF16, seed=32)[0]
    got = mx.mx_orthogonalize(g, steps=2)
    for i in (0, batch - 1):
        check(g[i], got[i], [COEFFS] * 2, what=f"matrix {i}")


def test_empty(mx):
    for shape in ((0, 8, 8), (2, 0, 8), (2, 8, 0)):
        assert mx.mx_orthogonalize(torch.empty(shape, dtype=BF16, device="cuda")).shape == shape


def test_python_refusals(mx):
    g = momentum(1, 16, 24, BF16, seed=1)[0].contiguous()
    with pytest.raises(TypeError):
        mx.mx_orthogonalize(g.half())
    with pytest.raises(ValueError):
        mx.mx_orthogonalize(g.t())
    with pytest.raises(ValueError):
        mx.mx_orthogonalize(g, steps=0)
    with pytest.raises(ValueError):
        mx.mx_orthogonalize(g, steps=4, coeffs=[COEFFS] * 3)
    with pytest.raises(mx.MXError):
        mx.mx_orthogonalize(g, coeffs=(8.0, 0.0, 0.0))      # singular values would leave FP16's range
    with pytest.raises(mx.MXError):
        mx.mx_orthogonalize(g, coeffs=(float("nan"), 0.0, 0.0))
    with pytest.raises(mx.MXError):
        mx.mx_orthogonalize(g, eps=-1.0)
    with pytest.raises(mx.MXError):
        mx.mx_orthogonalize(g, workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError):
        mx.mx_orthogonalize(g, out=torch.empty((24, 16), dtype=BF16, device="cuda"))
