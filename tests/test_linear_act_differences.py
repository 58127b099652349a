"""The gradients of mx_linear_act against central differences of its 64-bit forward
pass, each along the direction in which a wrong gradient shows most: the signs of
the gradient itself, so that what is compared is the sum of its elements'
magnitudes, while the tolerance is a sum of roundings, some hundredths of that.
That this rejects gradients that are wrong is shown on the CPU.

L = sum(c * y); z is the 64-bit pre-activation rounded to FP16, as the forward
pass keeps it: 2^-11 |z| off, which moves act' by at most 1.2 times as much (the
largest |act''| of the smooth activations).  Each dz is rounded to FP16 once,
each gradient once more.  relu's kink is kept away from: c is zero where |z| < 2^-6."""
import pytest
import torch

from gemm16_util import act_ref

FP16 = torch.float16
ACTS = ["none", "relu", "silu", "gelu", "gelu_tanh"]
M, N, K = 24, 40, 48
NAMES = ("dx", "dw", "dbias")


def inputs(act):
    """x, w, b, c in FP16 and z in 64 bits, on the CPU."""
    gen = torch.Generator().manual_seed(5)
    x, w, b, c = (torch.randn(shape, generator=gen).mul(scale).to(FP16)
                  for shape, scale in (((M, K), 1.0), ((N, K), 0.2), ((N,), 0.3), ((M, N), 1.0)))
    z = x.double() @ w.double().T + b.double()
    if act == "relu":
        c = torch.where(z.abs() >= 2.0 ** -6, c, torch.zeros_like(c))
    return x, w, b, c, z


def from_slope(c, slope, x, w):
    """The three gradients from act'."""
    dz = c.double() * slope
    return dz @ w.double(), dz.T @ x.double(), dz.sum(0)


def compare(act, gradients):
    """For dx, dw and dbias: how far the gradient's sum along its direction is from the difference's, and the tolerance."""
    x, w, b, c, z = inputs(act)
    slope = act_ref(z, act)[1]
    true = from_slope(c, slope, x, w)

    def value(args):
        return (c.double() * act_ref(args[0] @ args[1].T + args[2], act)[0]).sum().item()

    h = 1e-6
    # dz: its rounding and, through z's, act's
    per = c.double().abs() * (2.0 ** -11 * slope.abs() + (1.2 * 2.0 ** -11 * (z.abs() + 2.0 ** -11) if act not in ("none", "relu") else 0.0))
    spread = (per @ w.double().abs(), per.T @ x.double().abs(), per.sum(0))
    out = []
    for i, got in enumerate(gradients):
        d = torch.sign(true[i])
        args = [x.double(), w.double(), b.double()]
        up = value([a + h * d if j == i else a for j, a in enumerate(args)])
        down = value([a - h * d if j == i else a for j, a in enumerate(args)])
        want = (up - down) / (2 * h)
        have = (got.double().cpu() * d).sum().item()
        tol = (1.01 * spread[i] + 2.0 ** -11 * true[i].abs() + 2.0 ** -24).sum().item() + 1e-4 * abs(want)
        out.append((abs(have - want), tol, abs(want)))
    return out


@pytest.mark.parametrize("act", ACTS)
def test_wrong_gradients_are_rejected(act):
    """The formula's gradients pass; zeros, gradients three hundredths too large and, for the smooth
    activations, a slope act(z) / z without its second term fail, for each of dx, dw and dbias."""
    x, w, b, c, z = inputs(act)
    y, slope = act_ref(z, act)
    right = from_slope(c, slope, x, w)
    for name, (off, tol, size) in zip(NAMES, compare(act, right)):
        assert off <= tol and tol < 0.03 * size, (act, name, off, tol, size)
    wrong = [[torch.zeros_like(g) for g in right], [1.03 * g for g in right]]
    if act in ("silu", "gelu", "gelu_tanh"):
        wrong.append(from_slope(c, y / z, x, w))
    for i, gradients in enumerate(wrong):
        for name, (off, tol, _) in zip(NAMES, compare(act, gradients)):
            assert off > tol, (act, name, i, off, tol)


@pytest.mark.gpu
@pytest.mark.parametrize("act", ACTS)
def test_gradients(act):
    import moe_grouped_gemm_mx_b200 as mx
    x, w, b, c, z = inputs(act)
    got = mx.mx_linear_act_backward(c.cuda(), x.cuda(), w.cuda(), z=z.to(FP16).cuda(), activation=act, bias_grad=True)
    for name, (off, tol, _) in zip(NAMES, compare(act, got)):
        assert off <= tol, (act, name, off, tol)
