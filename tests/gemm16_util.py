"""Helpers of the tests of the 16-bit products: references in 64 bits and the
error a correct kernel may have.

A result rounded once to type T is off by at most u_T = eps_T / 2 relative to
its value.  The sum of K products (each exact in FP32) is formed 16 at a time
by the tensor core and added to an FP32 accumulator; counting one truncated
addition (2^-23 of the largest partial sum, itself at most sum |a b|) per step of 16
and 16 more inside it, doubled for the partial sums of a split K, the sum is off
by at most (K / 16 + 16) 2^-22 sum |a b|."""
import torch

U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
TINY = {torch.bfloat16: 2.0 ** -133, torch.float16: 2.0 ** -24, torch.float32: 2.0 ** -149}  # below the normal range
SENTINEL = -12.375  # what untouched memory is filled with; exact in every type


def sum_error(k: int) -> float:
    return (k / 16 + 16) * 2.0 ** -22


def normal(shape, dtype, seed, scale=1.0):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    return (torch.randn(shape, generator=gen, device="cuda") * scale).to(dtype)


def guarded(shape, dtype, guard=4096):
    """(tensor, check): a tensor inside a larger buffer of sentinels, and a
    function that tells whether the buffer's other elements still hold them."""
    n = 1
    for s in shape:
        n *= s
    pad = (n + 7) // 8 * 8 - n
    buf = torch.full((2 * guard + n + pad,), SENTINEL, dtype=dtype, device="cuda")
    t = buf[guard:guard + n].view(shape)

    def intact():
        return bool((buf[:guard] == SENTINEL).all()) and bool((buf[guard + n:] == SENTINEL).all())

    return t, intact


def close(got, ref, tol, what):
    """|got - ref| <= tol element by element (64-bit tensors on the GPU)."""
    got = got.double()
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    assert bool(torch.isfinite(got).all()), f"{what}: not finite"
    err = (got - ref).abs()
    bad = err > tol
    if bool(bad.any()):
        at = tuple(int(v) for v in bad.nonzero()[0])
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} off; at {at} got {got[at].item():.9g}, "
                             f"ref {ref[at].item():.9g}, tolerance {tol[at].item():.3g}")


def product_tol(ref, abs_sum, k, dtype):
    return U[dtype] * ref.abs() + sum_error(k) * abs_sum * (1 + U[dtype]) + TINY[dtype]


def act_ref(z, name):
    """act(z) and act'(z) in 64 bits."""
    import math
    if name == "relu":
        return z.clamp(min=0), (z > 0).double()
    if name == "silu":
        p = torch.sigmoid(z)
        return z * p, p * (1 + z * (1 - p))
    if name == "gelu":
        cdf = 0.5 * torch.erfc(-z / math.sqrt(2))
        return z * cdf, cdf + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    if name == "gelu_tanh":
        c = 2 * math.sqrt(2 / math.pi)
        p = torch.sigmoid(c * (z + 0.044715 * z ** 3))
        return z * p, p + z * p * (1 - p) * c * (1 + 0.134145 * z * z)
    return z, torch.ones_like(z)
