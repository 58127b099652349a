"""16-bit products grouped by expert over ragged row ranges, with both
gradients, against 64-bit references on the GPU: empty experts, experts of one
row, sizes around the tiles' edges, rows outside the groups left as they were,
what lies next to a group kept out of it, bad offsets, and the whole chain from
the router's table to the gradients."""
import contextlib
import os

import pytest
import torch

import mx_inputs
from gemm16_util import SENTINEL, U, close, guarded, normal, product_tol

pytestmark = pytest.mark.gpu

BF16, FP16, FP32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module")
def mx():
    import moe_grouped_gemm_mx_b200 as m
    return m


@contextlib.contextmanager
def config(value):
    if value is None:
        yield
        return
    os.environ["MX_GEMM16_CONFIG"] = str(value)
    try:
        yield
    finally:
        del os.environ["MX_GEMM16_CONFIG"]


def offsets_of(counts, first=0):
    return torch.tensor([first] + [first + sum(counts[:i + 1]) for i in range(len(counts))], dtype=torch.int32, device="cuda")


def check(mx, counts, n, k, dtype, first=0, behind=0, seed=0, out_dtype=None):
    """Forward, input gradient and weight gradient of one routing; rows before
    `first` and `behind` rows after the last group hold NaN in the operands."""
    off = offsets_of(counts, first)
    m = first + sum(counts) + behind
    lo, hi = first, first + sum(counts)
    a, b = normal((m, k), dtype, seed), normal((len(counts), n, k), dtype, seed + 1, k ** -0.5)
    dd = normal((m, n), dtype, seed + 2, 0.1)
    for t in (a, dd):
        t[:lo] = float("nan")
        t[hi:] = float("inf")
    d, i1 = guarded((m, n), dtype)
    da, i2 = guarded((m, k), dtype)
    out_dtype = dtype if out_dtype is None else out_dtype
    db, i3 = guarded((len(counts), n, k), out_dtype)
    d.fill_(SENTINEL)
    da.fill_(SENTINEL)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    mx.mx_grouped_gemm_ragged(a, b, off, d=d, dev_status=status)
    mx.mx_grouped_gemm_ragged_dgrad(dd, b, off, da=da, dev_status=status)
    mx.mx_grouped_gemm_ragged_wgrad(dd, a, off, db=db, dev_status=status)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    at = lo
    for e, rows in enumerate(counts):
        s = slice(at, at + rows)
        at += rows
        ad, bd, gd = a[s].double(), b[e].double(), dd[s].double()
        if rows:
            r = ad @ bd.T
            close(d[s], r, product_tol(r, ad.abs() @ bd.abs().T, k, dtype), f"d of expert {e} ({rows} rows)")
            r = gd @ bd
            close(da[s], r, product_tol(r, gd.abs() @ bd.abs(), n, dtype), f"da of expert {e} ({rows} rows)")
        r = gd.T @ ad
        close(db[e], r, product_tol(r, gd.abs().T @ ad.abs(), max(rows, 1), out_dtype), f"db of expert {e} ({rows} rows)")
        if not rows:
            assert bool((db[e] == 0).all())
    for t in (d, da):
        assert bool((t[:lo] == SENTINEL).all()) and bool((t[hi:] == SENTINEL).all()), "rows outside the groups changed"
    assert i1() and i2() and i3(), "wrote outside an output"


ROUTINGS = {
    "one": [1],
    "ones": [1, 1, 0, 1],
    "edges": [127, 128, 129, 0, 255, 256, 257],
    "tails of K steps": [15, 16, 17, 31, 33, 1, 64, 65, 111, 113, 0, 200],
    "empty ends": [0, 0, 70, 0, 300, 0],
    "all in one": [0, 700, 0, 0],
}


@pytest.mark.parametrize("cfg", [None, 0, 1, 2])
@pytest.mark.parametrize("routing", list(ROUTINGS), ids=lambda s: s.replace(" ", "-"))
def test_routings(mx, cfg, routing):
    with config(cfg):
        check(mx, ROUTINGS[routing], 264, 136, BF16, seed=3)


@pytest.mark.parametrize("cfg", [0, 1, 4])
@pytest.mark.parametrize("nk", [(8, 8), (64, 256), (128, 72), (520, 328)], ids=str)
def test_sizes_and_rows_outside(mx, cfg, nk):
    with config(cfg):
        check(mx, [33, 0, 150, 7], *nk, FP16, first=13, behind=29, seed=4)


@pytest.mark.parametrize("dtype", [BF16, FP16], ids=["bf16", "fp16"])
def test_weight_gradient_in_32_bits(mx, dtype):
    check(mx, [70, 0, 1, 260, 129], 136, 392, dtype, out_dtype=FP32, first=3, behind=5)


def test_many_groups(mx):
    gen = torch.Generator().manual_seed(0)
    counts = torch.randint(0, 9, (1024,), generator=gen).tolist()
    check(mx, counts, 72, 64, BF16, first=2, behind=2)


def test_several_tiles_a_pair(mx):
    """More 256 x 256 tiles than CTA pairs: the accumulators alternate, the epilogue overlaps."""
    check(mx, [1500, 3, 900, 700, 0, 1100], 1560, 1032, BF16, seed=9)


def test_neighbours_stay_out_of_a_weight_gradient(mx):
    """An expert whose rows are infinite spoils its own gradient only, at every
    remainder of its neighbours' row counts modulo 16."""
    for tail in range(1, 17):
        counts = [112 + tail, 40, 16 + tail]
        off = offsets_of(counts)
        m = sum(counts)
        a, dd = normal((m, 136), BF16, tail), normal((m, 72), BF16, 50 + tail)
        want = mx.mx_grouped_gemm_ragged_wgrad(dd, a, off)
        lo = counts[0]
        a[lo:lo + 40] = float("inf")
        dd[lo:lo + 40] = float("nan")
        got = mx.mx_grouped_gemm_ragged_wgrad(dd, a, off)
        assert torch.equal(got[0], want[0]) and torch.equal(got[2], want[2]), tail
        assert bool(torch.isnan(got[1]).all())


def test_no_rows(mx):
    b = normal((3, 64, 32), BF16, 1)
    off = torch.zeros(4, dtype=torch.int32, device="cuda")
    assert mx.mx_grouped_gemm_ragged(torch.empty((0, 32), dtype=BF16, device="cuda"), b, off).shape == (0, 64)
    db = mx.mx_grouped_gemm_ragged_wgrad(torch.empty((0, 64), dtype=BF16, device="cuda"),
                                         torch.empty((0, 32), dtype=BF16, device="cuda"), off, out_dtype=FP32)
    assert db.shape == (3, 64, 32) and db.dtype == FP32 and bool((db == 0).all())
    # rows, but none of them any expert's
    d = torch.full((40, 64), SENTINEL, dtype=BF16, device="cuda")
    mx.mx_grouped_gemm_ragged(normal((40, 32), BF16, 2), b, off + 40, d=d)
    assert bool((d == SENTINEL).all())
    db = mx.mx_grouped_gemm_ragged_wgrad(normal((40, 64), BF16, 3), normal((40, 32), BF16, 2), off + 40)
    assert bool((db == 0).all())


@pytest.mark.parametrize("cfg", [0, 1])
@pytest.mark.parametrize("bad", [[0, 50, 40, 100], [-1, 10, 20, 100], [0, 10, 20, 101], [5, 4, 100, 100]], ids=str)
def test_bad_offsets(mx, cfg, bad):
    with config(cfg):
        off = torch.tensor(bad, dtype=torch.int32, device="cuda")
        a, b, dd = normal((100, 64), BF16, 1), normal((3, 72, 64), BF16, 2), normal((100, 72), BF16, 3)
        for call, shape in ((lambda o, s: mx.mx_grouped_gemm_ragged(a, b, off, d=o, dev_status=s), (100, 72)),
                            (lambda o, s: mx.mx_grouped_gemm_ragged_dgrad(dd, b, off, da=o, dev_status=s), (100, 64)),
                            (lambda o, s: mx.mx_grouped_gemm_ragged_wgrad(dd, a, off, db=o, dev_status=s), (3, 72, 64))):
            out = torch.full(shape, SENTINEL, dtype=BF16, device="cuda")
            status = torch.zeros(1, dtype=torch.int32, device="cuda")
            call(out, status)
            torch.cuda.synchronize()
            assert int(status.item()) == mx.MX_DEV_BAD_OFFSETS and bool((out == SENTINEL).all())
        mx.read_internal_status()
        mx.mx_grouped_gemm_ragged(a, b, off)
        assert mx.read_internal_status() == mx.MX_DEV_BAD_OFFSETS


def test_gradients_against_differences(mx):
    """da and db against central differences of the 64-bit forward."""
    counts, n, k = [5, 0, 19, 8], 24, 40
    off = offsets_of(counts)
    m = sum(counts)
    a, b, c = normal((m, k), FP16, 1), normal((4, n, k), FP16, 2), normal((m, n), FP16, 3)
    da = mx.mx_grouped_gemm_ragged_dgrad(c, b, off)
    db = mx.mx_grouped_gemm_ragged_wgrad(c, a, off, out_dtype=FP32)
    expert = torch.repeat_interleave(torch.arange(4), torch.tensor(counts)).cuda()

    def value(ad, bd):
        return (c.double() * torch.einsum("mk,mnk->mn", ad, bd[expert])).sum().item()

    h = 1e-4
    for i, (t, got) in enumerate(((a, da), (b, db))):
        d = normal(t.shape, torch.float32, 10 + i).double()
        args = [a.double(), b.double()]
        args[i] = args[i] + h * d
        up = value(*args)
        args[i] = args[i] - 2 * h * d
        want = (up - value(*args)) / (2 * h)
        tol = (U[got.dtype] * got.double().abs() * d.abs()).sum().item() + 1e-4 * abs(want) + 1e-3
        assert abs((got.double() * d).sum().item() - want) <= tol


def test_captured_and_replayed(mx):
    """The group sizes are read on the device: a captured call follows new offsets."""
    m, n, k = 300, 136, 264
    a, b, dd = normal((m, k), BF16, 1), normal((4, n, k), BF16, 2), normal((m, n), BF16, 3)
    off = offsets_of([100, 50, 0, 150])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())

    def step():
        return (mx.mx_grouped_gemm_ragged(a, b, off), mx.mx_grouped_gemm_ragged_dgrad(dd, b, off),
                mx.mx_grouped_gemm_ragged_wgrad(dd, a, off))

    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for counts in ([1, 2, 3, 294], [0, 300, 0, 0], [77, 78, 79, 66]):
        off.copy_(offsets_of(counts))
        graph.replay()
        want = step()
        torch.cuda.synchronize()
        assert all(torch.equal(g, w) for g, w in zip(out, want))


def test_expert_layer_step(mx):
    """The calls in a row, as a step of a 16-bit expert layer makes them: the
    router's table to a plan without padding, rows gathered, gate-weighted expert
    products combined, the gradients of the experts' weights and the update of
    those weights, each stage against 64 bits on the stage's own inputs."""
    tokens, topk, experts, hidden, n = 150, 2, 6, 264, 136
    x = normal((tokens, hidden), BF16, 1)
    w = normal((experts, n, hidden), BF16, 2, 0.05)
    ids_np = mx_inputs.topk_ids(tokens, topk, experts, seed=3)
    ids = torch.from_numpy(ids_np.reshape(-1).copy()).cuda()
    gate = torch.from_numpy(mx_inputs.gate_weights(tokens, topk, seed=4)).cuda()
    counts, offsets, row, dropped = mx.mx_moe_route(ids, experts, pad=1)
    assert int(dropped.item()) == 0 and int(offsets[-1].item()) == tokens * topk
    # row[i] is where entry i goes: the source token of each grouped row
    source = torch.empty(tokens * topk, dtype=torch.int32, device="cuda")
    source[row.long()] = torch.arange(tokens * topk, dtype=torch.int32, device="cuda") // topk
    a = mx.mx_gather_rows(x, source)
    d = mx.mx_grouped_gemm_ragged(a, w, offsets)
    y = mx.mx_moe_combine(d, row, gate)
    expert = torch.empty(tokens * topk, dtype=torch.long, device="cuda")
    expert[row.long()] = ids.long()
    wd = w.double()[expert]
    ref = torch.einsum("mk,mnk->mn", x.double()[source.long()], wd)
    mass = torch.einsum("mk,mnk->mn", x.double()[source.long()].abs(), wd.abs())
    close(d, ref, product_tol(ref, mass, hidden, BF16), "expert rows")
    out = (gate.double()[..., None] * d.double()[row.long()].view(tokens, topk, n)).sum(1)
    scale = (gate.double()[..., None] * d.double().abs()[row.long()].view(tokens, topk, n)).sum(1)
    close(y, out, U[BF16] * out.abs() + 2.0 ** -20 * scale, "combined")
    # backward: each grouped row's gradient is its gate weight times the token's
    dy = normal((tokens, n), BF16, 5)
    dd = torch.empty((tokens * topk, n), dtype=BF16, device="cuda")
    dd[row.long()] = (gate[..., None] * dy.float()[:, None]).view(-1, n).to(BF16)
    dw = mx.mx_grouped_gemm_ragged_wgrad(dd, a, offsets)
    for e in range(experts):
        rows = expert == e
        ref = dd[rows].double().T @ a[rows].double()
        mass = dd[rows].double().abs().T @ a[rows].double().abs()
        close(dw[e], ref, product_tol(ref, mass, int(rows.sum()) + 1, BF16), f"dw of expert {e}")
    update = mx.mx_orthogonalize(dw)
    again = mx.mx_orthogonalize(dw[2].contiguous())
    assert update.shape == w.shape and torch.equal(update[2], again)
    # nearly orthogonal rows: with the usual coefficients five steps bring singular values of at
    # least 2e-3 of the norm into about [0.68, 1.14] (the bound [0.5, 1.3] leaves room for BF16)
    for e in range(experts):
        s = torch.linalg.svdvals(dw[e].double())
        got = torch.linalg.svdvals(update[e].double())
        large = int((s > 2e-3 * torch.linalg.vector_norm(s)).sum())
        assert bool((got[:large] > 0.5).all()) and bool((got < 1.3).all())


def test_more_elements_than_32_bits_count(mx):
    """Weights, their gradients and the grouped rows each of more than 2^31 elements."""
    groups, n, k = 66, 8192, 4096                       # 2.2e9 weights
    counts = [3] * groups
    counts[5] = 0
    off = offsets_of(counts)
    m = sum(counts)
    a, dd = normal((m, k), BF16, 1), normal((m, n), BF16, 2)
    b = torch.empty((groups, n, k), dtype=BF16, device="cuda").fill_(0.25)
    b[-1] = normal((n, k), BF16, 3, 0.02)
    d = mx.mx_grouped_gemm_ragged(a, b, off)
    da = mx.mx_grouped_gemm_ragged_dgrad(dd, b, off)
    for e in (0, 5, groups - 1):
        s = slice(int(off[e]), int(off[e + 1]))
        be = b[e].double()
        ref = a[s].double() @ be.T
        close(d[s], ref, product_tol(ref, a[s].double().abs() @ be.abs().T, k, BF16), f"d of expert {e}")
        ref = dd[s].double() @ be
        close(da[s], ref, product_tol(ref, dd[s].double().abs() @ be.abs(), n, BF16), f"da of expert {e}")
    del b, d, da
    db = mx.mx_grouped_gemm_ragged_wgrad(dd, a, off)
    for e in (0, 5, groups - 1):
        s = slice(int(off[e]), int(off[e + 1]))
        ref = dd[s].double().T @ a[s].double()
        close(db[e], ref, product_tol(ref, dd[s].double().abs().T @ a[s].double().abs(), 3, BF16), f"db of expert {e}")
    del db
    m = 600 * 1024                                      # 2.5e9 results in two experts
    off = offsets_of([m // 2 + 77, m - m // 2 - 77])
    a, b = normal((m, 64), BF16, 4), normal((2, 4096, 64), BF16, 5, 0.125)
    d = mx.mx_grouped_gemm_ragged(a, b, off)
    for row in (0, int(off[1]) - 1, int(off[1]), 524287, 524288, m - 1):
        e = int(row >= int(off[1]))
        ref = a[row].double() @ b[e].double().T
        close(d[row], ref, product_tol(ref, a[row].double().abs() @ b[e].double().abs().T, 64, BF16), f"row {row}")


def test_python_refusals(mx):
    a, b = normal((16, 64), BF16, 1), normal((2, 32, 64), BF16, 2)
    off = offsets_of([7, 9])
    with pytest.raises(TypeError):
        mx.mx_grouped_gemm_ragged(a.float(), b, off)
    with pytest.raises(TypeError):
        mx.mx_grouped_gemm_ragged(a, b.half(), off)
    with pytest.raises(TypeError):
        mx.mx_grouped_gemm_ragged(a, b, off.long())
    with pytest.raises(ValueError):
        mx.mx_grouped_gemm_ragged(a, b, off[:2].contiguous())
    with pytest.raises(ValueError):
        mx.mx_grouped_gemm_ragged(a, b, off.cpu())
    with pytest.raises(ValueError):
        mx.mx_grouped_gemm_ragged(a, b, off, d=torch.empty((16, 31), dtype=BF16, device="cuda"))
    with pytest.raises(TypeError):
        mx.mx_grouped_gemm_ragged_wgrad(normal((16, 32), BF16, 3), a, off, out_dtype=FP16)
    with pytest.raises(mx.MXError):
        mx.mx_grouped_gemm_ragged(normal((16, 60), BF16, 1), normal((2, 32, 60), BF16, 2), off)
