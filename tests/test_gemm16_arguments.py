"""Arguments of a wrong kind are refused by the 16-bit calls as by the others: a TypeError that names the argument."""
import pytest
import torch

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


@pytest.fixture(scope="module")
def mx():
    import moe_grouped_gemm_mx_b200 as m
    return m


def test_outputs_and_workspaces_that_are_no_tensors(mx):
    x, w = torch.ones(16, 64, dtype=BF16, device="cuda"), torch.ones(32, 64, dtype=BF16, device="cuda")
    dy = torch.ones(16, 32, dtype=BF16, device="cuda")
    off = torch.tensor([0, 16], dtype=torch.int32, device="cuda")
    calls = {
        "workspace": [lambda v: mx.mx_orthogonalize(x, workspace=v),
                      lambda v: mx.mx_linear_act_backward(dy, x, w, bias_grad=True, workspace=v)],
        "out": [lambda v: mx.mx_orthogonalize(x, out=v)],
        "db": [lambda v: mx.mx_grouped_gemm_ragged_wgrad(dy, x, off, db=v),
               lambda v: mx.mx_grouped_gemm_ragged_wgrad(dy, x, off, db=v, out_dtype=torch.float32)],
        "dbias": [lambda v: mx.mx_linear_act_backward(dy, x, w, dbias=v)],
        "d": [lambda v: mx.mx_grouped_gemm_ragged(x, w[None], off, d=v)],
        "da": [lambda v: mx.mx_grouped_gemm_ragged_dgrad(dy, w[None], off, da=v)],
        "y": [lambda v: mx.mx_linear_act(x, w, y=v)],
        "bias": [lambda v: mx.mx_linear_act(x, w, bias=v)],
        "dev_status": [lambda v: mx.mx_linear_act(x, w, dev_status=v)],
    }
    for name, fs in calls.items():
        for f in fs:
            for value in ([0] * 64, 4096):
                with pytest.raises(TypeError, match=name):
                    f(value)


def test_workspace_of_another_type_or_shape(mx):
    g = torch.ones(136, 264, dtype=BF16, device="cuda")
    need = mx.mx_orthogonalize_workspace_bytes(1, 136, 264)
    with pytest.raises(TypeError):
        mx.mx_orthogonalize(g, workspace=torch.empty(need, dtype=torch.int8, device="cuda"))
    with pytest.raises(ValueError):
        mx.mx_orthogonalize(g, workspace=torch.empty(need, dtype=torch.uint8))
    with pytest.raises(ValueError):
        mx.mx_orthogonalize(g, workspace=torch.empty(2, need, dtype=torch.uint8, device="cuda"))
