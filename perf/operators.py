"""The library's products of 16-bit operands, as cases that can be timed and compared.

Three operators of a mixture-of-experts training step and of its serving form:

* ``linear``: y = act(x w^T + bias) + residual, and its backward pass
  (mx_linear_act, mx_linear_act_backward);
* ``experts``: products grouped by expert over ragged row ranges, with both
  gradients (mx_grouped_gemm_ragged, _dgrad, _wgrad);
* ``muon``: the Newton-Schulz orthogonalisation of a batch of weight updates
  (mx_orthogonalize).

``run`` computes the plain form (elementary torch operations in 32 bits,
rounded once) or, with ``own`` set, calls the library.  ``exact`` gives the
definition in 64 bits.
"""
import math

import torch

own = False

DEVICE = "cuda"
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
ACTIVATIONS = ("none", "relu", "silu", "gelu", "gelu_tanh")
NS_COEFFS = (3.4445, -4.7750, 2.0315)  # the quintic of Newton-Schulz orthogonalisation in common use
NS_EPS = 1e-7


# ---------------------------------------------------------------- cases

def listed():
    return [
        # a decode step's projection of 64 tokens into a latent of 2112: weights are read once, latency counts
        {"name": "linear decode 64x2112x7168", "op": "linear", "m": 64, "n": 2112, "k": 7168, "dtype": "bf16",
         "act": "none", "bias": True, "residual": False, "z": False},
        # a training step's first projection of a dense MLP (8192 tokens): GELU, pre-activation kept for backward
        {"name": "linear train 8192x4096x7168", "op": "linear", "m": 8192, "n": 4096, "k": 7168, "dtype": "bf16",
         "act": "gelu", "bias": True, "residual": False, "z": True},
        # an output projection added to the residual stream, an odd number of tokens of a packed batch
        {"name": "linear residual 1037x7168x2048", "op": "linear", "m": 1037, "n": 7168, "k": 2048, "dtype": "fp16",
         "act": "silu", "bias": True, "residual": True, "z": False},
        # the backward pass of the training step's projection: dx, dw, dbias
        {"name": "linear backward 8192x4096x7168", "op": "linear_backward", "m": 8192, "n": 4096, "k": 7168,
         "dtype": "bf16", "act": "gelu_tanh", "bias": True},
        # the same for a small adapter, all sizes odd multiples of eight
        {"name": "linear backward 333x1000x776", "op": "linear_backward", "m": 333, "n": 1000, "k": 776,
         "dtype": "fp16", "act": "relu", "bias": True},
        # the experts' gate/up product of a training step: 8192 tokens x top-8 over 32 experts, as routed
        {"name": "experts train 65536 rows", "op": "experts", "tokens": 8192, "topk": 8, "experts": 32, "n": 4096,
         "k": 7168, "dtype": "bf16"},
        # the same experts on a decode step of 64 tokens: about 16 rows an expert, the weights' bytes bound it
        {"name": "experts decode 512 rows", "op": "experts", "tokens": 64, "topk": 8, "experts": 32, "n": 4096,
         "k": 7168, "dtype": "bf16"},
        # the input gradient of the down projection
        {"name": "experts dgrad 65536 rows", "op": "experts_dgrad", "tokens": 8192, "topk": 8, "experts": 32,
         "n": 7168, "k": 2048, "dtype": "bf16"},
        # the weight gradient of the down projection, into 32-bit main gradients
        {"name": "experts wgrad 65536 rows", "op": "experts_wgrad", "tokens": 8192, "topk": 8, "experts": 32,
         "n": 7168, "k": 2048, "dtype": "bf16", "out": "fp32"},
        # the optimiser's update of 8 experts' gate/up weights held by one rank
        {"name": "muon 8x4096x7168", "op": "muon", "batch": 8, "m": 4096, "n": 7168, "dtype": "bf16", "steps": 5},
        # of 4 experts' down weights: tall matrices, from 32-bit momentum
        {"name": "muon 4x7168x2048", "op": "muon", "batch": 4, "m": 7168, "n": 2048, "dtype": "fp32", "steps": 5},
        # of a router's weight: one small matrix, launches count
        {"name": "muon 1x32x7168", "op": "muon", "batch": 1, "m": 32, "n": 7168, "dtype": "bf16", "steps": 5},
    ]


def _log_uniform(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def _dim(rng, low, high):
    """A row length the operands can have (whole 16-byte pieces): any multiple of eight."""
    return 8 * _log_uniform(rng, low // 8, high // 8)


def draw(rng):
    op = rng.choice(("linear", "linear_backward", "experts", "experts_dgrad", "experts_wgrad", "muon"))
    dtype = rng.choice(("bf16", "bf16", "fp16"))
    if op in ("linear", "linear_backward"):
        case = {"op": op, "m": _log_uniform(rng, 1, 8192), "n": _dim(rng, 64, 7168), "k": _dim(rng, 64, 7168),
                "dtype": dtype, "act": rng.choice(ACTIVATIONS), "bias": rng.random() < 0.7}
        if op == "linear":
            case["residual"] = rng.random() < 0.5
            case["z"] = rng.random() < 0.5
        return case
    if op == "muon":
        return {"op": op, "batch": rng.choice((1, 1, 2, 3, 4)), "m": _log_uniform(rng, 16, 4096),
                "n": _log_uniform(rng, 16, 7168), "dtype": rng.choice(("bf16", "fp32")),
                "steps": rng.choice((4, 5, 5, 6))}
    experts = _log_uniform(rng, 2, 64)
    case = {"op": op, "tokens": _log_uniform(rng, 1, 4096), "topk": rng.randint(1, min(8, experts)),
            "experts": experts, "n": _dim(rng, 128, 4096), "k": _dim(rng, 128, 4096), "dtype": dtype}
    if op == "experts_wgrad":
        case["out"] = rng.choice((dtype, "fp32"))
    return case


# ---------------------------------------------------------------- inputs

def _normal(gen, shape, scale, dtype):
    """Normal values of the given type, made in pieces so that no 32-bit copy of a large tensor is held."""
    out = torch.empty(shape, dtype=dtype, device=DEVICE)
    flat = out.view(-1)
    piece = 1 << 26
    for i in range(0, flat.numel(), piece):
        part = flat[i:i + piece]
        part.copy_(torch.randn(part.numel(), generator=gen, device=DEVICE).mul_(scale))
    return out


def _routing(gen, tokens, topk, experts):
    """Row ranges of the experts as a top-k router gives them: some experts are asked for more often than others."""
    liking = torch.randn(experts, generator=gen, device=DEVICE) * 0.4
    noise = -torch.log(-torch.log(torch.rand(tokens, experts, generator=gen, device=DEVICE).clamp_(1e-7, 1 - 1e-7)))
    chosen = (liking + noise).topk(topk, dim=1).indices.reshape(-1)
    counts = torch.bincount(chosen, minlength=experts)
    offsets = torch.zeros(experts + 1, dtype=torch.int32, device=DEVICE)
    offsets[1:] = torch.cumsum(counts, 0).to(torch.int32)
    return offsets, int(counts.max())


def prepare(case, seed):
    gen = torch.Generator(device=DEVICE)
    gen.manual_seed(seed)
    op = case["op"]
    dtype = DTYPES[case["dtype"]]
    s = {"case": dict(case)}
    if op in ("linear", "linear_backward"):
        m, n, k = case["m"], case["n"], case["k"]
        s["x"] = _normal(gen, (m, k), 1.0, dtype)
        s["w"] = _normal(gen, (n, k), k ** -0.5, dtype)
        s["bias"] = _normal(gen, (n,), 0.2, dtype) if case["bias"] else None
        if op == "linear":
            s["residual"] = _normal(gen, (m, n), 1.0, dtype) if case["residual"] else None
        else:  # the forward pass kept its pre-activation; the gradient comes from the layers above
            z = (s["x"] @ s["w"].t()).float()
            s["z"] = (z + s["bias"].float() if case["bias"] else z).to(dtype)
            s["dy"] = _normal(gen, (m, n), 0.05, dtype)
        return s
    if op == "muon":
        batch, m, n = case["batch"], case["m"], case["n"]
        # a momentum of gradients: a few strong directions over a floor of noise
        rank = max(1, min(m, n) // 16)
        left = torch.randn(batch, m, rank, generator=gen, device=DEVICE)
        right = torch.randn(batch, rank, n, generator=gen, device=DEVICE)
        g = torch.randn(batch, m, n, generator=gen, device=DEVICE)
        s["g"] = torch.baddbmm(g, left, right, beta=0.2, alpha=rank ** -0.5).mul_(1e-3).to(dtype)
        return s
    n, k = case["n"], case["k"]
    rows = case["tokens"] * case["topk"]
    s["offsets"], s["most"] = _routing(gen, case["tokens"], case["topk"], case["experts"])
    if op == "experts_wgrad":
        s["dd"] = _normal(gen, (rows, n), 0.05, dtype)
        s["a"] = _normal(gen, (rows, k), 1.0, dtype)
        return s
    s["b"] = _normal(gen, (case["experts"], n, k), k ** -0.5, dtype)
    if op == "experts":
        s["a"] = _normal(gen, (rows, k), 1.0, dtype)
    else:
        s["dd"] = _normal(gen, (rows, n), 0.05, dtype)
    return s


# ---------------------------------------------------------------- the plain forms

def _act(z, name):
    if name == "relu":
        return torch.clamp_min(z, 0.0)
    if name == "silu":
        return z / (1.0 + torch.exp(-z))
    if name == "gelu":
        return 0.5 * z * (1.0 + torch.erf(z * math.sqrt(0.5)))
    if name == "gelu_tanh":
        return 0.5 * z * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (z + 0.044715 * z * z * z)))
    return z


def _act_grad(z, name):
    if name == "relu":
        return (z > 0).to(z.dtype)
    if name == "silu":
        p = 1.0 / (1.0 + torch.exp(-z))
        return p * (1.0 + z * (1.0 - p))
    if name == "gelu":
        return 0.5 * (1.0 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) / math.sqrt(2.0 * math.pi)
    if name == "gelu_tanh":
        c = math.sqrt(2.0 / math.pi)
        t = torch.tanh(c * (z + 0.044715 * z * z * z))
        return 0.5 * (1.0 + t) + 0.5 * z * (1.0 - t * t) * c * (1.0 + 3 * 0.044715 * z * z)
    return torch.ones_like(z)


def _plain_linear(s):
    case, dtype = s["case"], s["x"].dtype
    z = s["x"].float() @ s["w"].float().t()
    if s["bias"] is not None:
        z = z + s["bias"].float()
    y = _act(z, case["act"])
    if s["residual"] is not None:
        y = y + s["residual"].float()
    return [y.to(dtype), z.to(dtype)] if case["z"] else [y.to(dtype)]


def _plain_linear_backward(s):
    case, dtype = s["case"], s["x"].dtype
    dz = s["dy"].float()
    if case["act"] != "none":
        dz = dz * _act_grad(s["z"].float(), case["act"])
    out = [(dz @ s["w"].float()).to(dtype), (dz.t() @ s["x"].float()).to(dtype)]
    if case["bias"]:
        out.append(dz.sum(0).to(dtype))
    return out


def _padded(rows, offsets, most):
    """The experts' rows as a [experts, most, columns] batch of 32-bit values, with zeros behind each expert's last."""
    at = offsets[:-1, None].long() + torch.arange(most, device=rows.device)
    inside = at < offsets[1:, None]
    return torch.where(inside[..., None], rows[at.clamp_max(rows.shape[0] - 1)].float(), 0.0), at[inside], inside


def _plain_experts(s, rows, b):
    padded, at, inside = _padded(rows, s["offsets"], s["most"])
    d = torch.bmm(padded, b.float())
    out = torch.empty(rows.shape[0], b.shape[2], dtype=rows.dtype, device=rows.device)
    out[at] = d[inside].to(rows.dtype)
    return [out]


def _plain_experts_wgrad(s):
    dd = _padded(s["dd"], s["offsets"], s["most"])[0]
    a = _padded(s["a"], s["offsets"], s["most"])[0]
    return [torch.bmm(dd.transpose(1, 2), a).to(DTYPES[s["case"]["out"]])]


def _plain_muon(s):
    g = s["g"]
    a, b, c = NS_COEFFS
    x = g.float()
    x = x / (torch.sqrt((x * x).sum(dim=(1, 2), keepdim=True)) + NS_EPS)
    tall = g.shape[1] > g.shape[2]
    if tall:
        x = x.transpose(1, 2)
    for _ in range(s["case"]["steps"]):  # the iteration itself: each step needs the one before
        p = torch.bmm(x, x.transpose(1, 2))
        x = a * x + torch.bmm(b * p + c * torch.bmm(p, p), x)
    if tall:
        x = x.transpose(1, 2)
    return [x.contiguous().to(torch.bfloat16)]


# ---------------------------------------------------------------- one pass

def run(state):
    case = state["case"]
    op = case["op"]
    if own:
        return _own(state, op, case)
    if op == "linear":
        return _plain_linear(state)
    if op == "linear_backward":
        return _plain_linear_backward(state)
    if op == "experts":
        return _plain_experts(state, state["a"], state["b"].transpose(1, 2))
    if op == "experts_dgrad":
        return _plain_experts(state, state["dd"], state["b"])
    if op == "experts_wgrad":
        return _plain_experts_wgrad(state)
    return _plain_muon(state)


def _own(s, op, case):
    import moe_grouped_gemm_mx_b200 as mx
    if op == "linear":
        got = mx.mx_linear_act(s["x"], s["w"], bias=s["bias"], residual=s["residual"], activation=case["act"],
                               return_z=case["z"])
        return list(got) if case["z"] else [got]
    if op == "linear_backward":
        got = mx.mx_linear_act_backward(s["dy"], s["x"], s["w"], z=s["z"], activation=case["act"],
                                        bias_grad=case["bias"])
        return [t for t in got if t is not None]
    if op == "experts":
        return [mx.mx_grouped_gemm_ragged(s["a"], s["b"], s["offsets"])]
    if op == "experts_dgrad":
        return [mx.mx_grouped_gemm_ragged_dgrad(s["dd"], s["b"], s["offsets"])]
    if op == "experts_wgrad":
        return [mx.mx_grouped_gemm_ragged_wgrad(s["dd"], s["a"], s["offsets"], out_dtype=DTYPES[case["out"]])]
    return [mx.mx_orthogonalize(s["g"], steps=case["steps"], coeffs=NS_COEFFS, eps=NS_EPS)]


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    op = case["op"]
    if op in ("linear", "linear_backward"):
        m, n, k = case["m"], case["n"], case["k"]
        bias = n if case["bias"] else 0
        if op == "linear":
            values = m * k + n * k + bias + m * n * (1 + case["residual"] + case["z"])
            return {"bytes": 2 * values, "flops": 2.0 * m * n * k}
        values = m * n * (2 if case["act"] != "none" else 1) + 2 * (m * k + n * k) + bias
        return {"bytes": 2 * values, "flops": 4.0 * m * n * k}
    if op == "muon":
        small, large = sorted((case["m"], case["n"]))
        size = 4 if case["dtype"] == "fp32" else 2
        # the two symmetric products need one triangle each
        step = small * (small + 1.0) * large + small * (small + 1.0) * small + 2.0 * small * small * large
        return {"bytes": case["batch"] * small * large * (size + 2), "flops": case["batch"] * case["steps"] * step}
    n, k, rows = case["n"], case["k"], case["tokens"] * case["topk"]
    # an expert without rows need not be read: with fewer rows than experts some have none
    weights = min(case["experts"], rows) * n * k
    if op == "experts_wgrad":
        size = DTYPES[case["out"]].itemsize
        return {"bytes": 2 * rows * (n + k) + size * case["experts"] * n * k, "flops": 2.0 * rows * n * k}
    return {"bytes": 2 * (rows * (n + k) + weights), "flops": 2.0 * rows * n * k}


# ---------------------------------------------------------------- the definitions in 64 bits

def _exact_act(z, name):
    """act(z) and its derivative."""
    if name == "relu":
        return z.clamp(min=0), (z > 0).double()
    if name == "silu":
        p = torch.sigmoid(z)
        return z * p, p + z * p * (1 - p)
    if name == "gelu":
        cdf = 0.5 * torch.erfc(-z / 2.0 ** 0.5)
        return z * cdf, cdf + z * torch.exp(-z * z / 2) / (2 * math.pi) ** 0.5
    if name == "gelu_tanh":
        # 0.5 (1 + tanh u) is the logistic function of 2u
        u2 = 2 * (2 / math.pi) ** 0.5 * (z + 0.044715 * z ** 3)
        p = torch.sigmoid(u2)
        return z * p, p + z * p * (1 - p) * 2 * (2 / math.pi) ** 0.5 * (1 + 0.134145 * z ** 2)
    return z, torch.ones_like(z)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "linear":
        z = torch.matmul(s["x"].double(), s["w"].double().T)
        if s["bias"] is not None:
            z += s["bias"].double()
        y = _exact_act(z, case["act"])[0]
        if s["residual"] is not None:
            y = y + s["residual"].double()
        return [y, z] if case["z"] else [y]
    if op == "linear_backward":
        dz = s["dy"].double() * _exact_act(s["z"].double(), case["act"])[1]
        out = [torch.matmul(dz, s["w"].double()), torch.matmul(dz.T, s["x"].double())]
        return out + [dz.sum(dim=0)] if case["bias"] else out
    if op == "muon":
        a, b, c = NS_COEFFS
        out = torch.empty(s["g"].shape, dtype=torch.float64, device=DEVICE)
        for i in range(case["batch"]):
            x = s["g"][i].double()
            x = x / (torch.linalg.vector_norm(x) + NS_EPS)
            flip = x.shape[0] > x.shape[1]
            x = x.T if flip else x
            for _ in range(case["steps"]):
                gram = x @ x.T
                gx = gram @ x
                x = a * x + b * gx + c * (gram @ gx)
            out[i] = x.T if flip else x
        return [out]
    bounds = s["offsets"].tolist()
    if op == "experts_wgrad":
        return [torch.stack([s["dd"][i:j].double().T @ s["a"][i:j].double() for i, j in zip(bounds, bounds[1:])])]
    rows = s["a"] if op == "experts" else s["dd"]
    parts = []
    for e, (i, j) in enumerate(zip(bounds, bounds[1:])):
        b = s["b"][e].double()
        parts.append(rows[i:j].double() @ (b.T if op == "experts" else b))
    return [torch.cat(parts)]
