"""What is measured of the dense linear layer and the gated MLP for blocks of tokens.

Three operators of ``sparse_input_gemv_threshold_b200``, each with its plain form in
elementary torch operations (32 bits, rounded once at the end) and its value in 64 bits:

  linear        Y = act(X WT + bias) + residual                       ``linear_act``
  gated         g = X WgT, u = X WuT, Y = (act(g) . u) WdT + residual   ``gated_mlp``
  gated_grad    dX, dWgT, dWuT, dWdT of ``gated`` from dY, X, g, u      ``gated_mlp_backward``

Weights are transposed as everywhere in this library (row i multiplies input i) and drawn
N(0, 1/d_in), so that projections have entries of order one whatever the size; tokens are
N(0, 1), as in the gated-MLP workload of the benchmark.
"""
import math

import torch

own = False

DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16}


def listed():
    return [
        # the attention output projection of one decoded token, added to the residual stream
        {"name": "linear 1x4096x4096 fp16", "op": "linear", "rows": 1, "K": 4096, "N": 4096, "dtype": "fp16",
         "act": "none", "bias": False, "residual": True},
        # sixteen sequences decoding together through a wide biased projection
        {"name": "linear 16x4096x11008 bf16", "op": "linear", "rows": 16, "K": 4096, "N": 11008, "dtype": "bf16",
         "act": "gelu", "bias": True, "residual": False},
        # a short prompt of odd length
        {"name": "linear 333x4096x4096 fp16", "op": "linear", "rows": 333, "K": 4096, "N": 4096, "dtype": "fp16",
         "act": "none", "bias": True, "residual": True},
        # the batched-token layer of the benchmark, with a biased activation
        {"name": "linear 4096x1024x1024 fp16", "op": "linear", "rows": 4096, "K": 1024, "N": 1024, "dtype": "fp16",
         "act": "relu", "bias": True, "residual": False},
        # the down projection of a long prompt, added to the residual stream
        {"name": "linear 4096x11008x4096 bf16", "op": "linear", "rows": 4096, "K": 11008, "N": 4096, "dtype": "bf16",
         "act": "none", "bias": False, "residual": True},
        # the MLP of one decoded token
        {"name": "gated 1x4096x11008 fp16", "op": "gated", "rows": 1, "d_model": 4096, "d_ff": 11008, "dtype": "fp16",
         "act": "silu", "residual": False, "save": False},
        # sixteen sequences decoding together at the largest MLP of the benchmark
        {"name": "gated 16x8192x28672 bf16", "op": "gated", "rows": 16, "d_model": 8192, "d_ff": 28672, "dtype": "bf16",
         "act": "silu", "residual": True, "save": False},
        # a prompt of odd length
        {"name": "gated 777x4096x11008 fp16", "op": "gated", "rows": 777, "d_model": 4096, "d_ff": 11008,
         "dtype": "fp16", "act": "silu", "residual": True, "save": False},
        # a training block of tokens, gate and up kept for the backward pass
        {"name": "gated 4096x4096x11008 bf16", "op": "gated", "rows": 4096, "d_model": 4096, "d_ff": 11008,
         "dtype": "bf16", "act": "silu", "residual": False, "save": True},
        # gradients of a few tokens: the weights and their gradients are nearly all of it
        {"name": "grad 16x4096x11008 fp16", "op": "gated_grad", "rows": 16, "d_model": 4096, "d_ff": 11008,
         "dtype": "fp16", "act": "silu"},
        # a small block of odd length through a small MLP
        {"name": "grad 515x1024x2816 bf16", "op": "gated_grad", "rows": 515, "d_model": 1024, "d_ff": 2816,
         "dtype": "bf16", "act": "gelu_tanh"},
        # a training block of tokens
        {"name": "grad 2048x4096x11008 bf16", "op": "gated_grad", "rows": 2048, "d_model": 4096, "d_ff": 11008,
         "dtype": "bf16", "act": "silu"},
    ]


def draw(rng):
    """One more case: token counts and widths spread over their logarithm, widths in steps of 8."""
    most = [max(work(c)[k] for c in listed()) for k in ("bytes", "flops")]
    while True:
        rows = int(round(math.exp(rng.uniform(0.0, math.log(4096)))))
        a = 8 * int(round(math.exp(rng.uniform(math.log(8), math.log(1024)))))
        b = 8 * int(round(math.exp(rng.uniform(math.log(8), math.log(3584)))))
        case = {"op": rng.choice(["linear", "gated", "gated_grad"]), "rows": rows,
                "dtype": rng.choice(["fp16", "bf16"])}
        if case["op"] == "linear":
            case["K"], case["N"] = (a, b) if rng.random() < 0.5 else (b, a)
            case.update(act=rng.choice(["none", "relu", "gelu", "gelu_tanh", "silu"]),
                        bias=rng.random() < 0.5, residual=rng.random() < 0.5)
        else:
            case.update(d_model=a, d_ff=b, act=rng.choice(["silu", "gelu", "gelu_tanh", "relu"]))
            if case["op"] == "gated":
                case.update(residual=rng.random() < 0.5, save=rng.random() < 0.5)
        w = work(case)
        if w["bytes"] <= most[0] and w["flops"] <= most[1]:
            return case


def work(case):
    """Bytes (two to a value; every input once, every output once) and flops of the products."""
    r = case["rows"]
    if case["op"] == "linear":
        K, N = case["K"], case["N"]
        values = r * K + K * N + r * N + (N if case["bias"] else 0) + (r * N if case["residual"] else 0)
        return {"bytes": 2 * values, "flops": 2 * r * K * N}
    m, f = case["d_model"], case["d_ff"]
    if case["op"] == "gated":
        values = 2 * r * m + 3 * m * f + (r * m if case["residual"] else 0) + (2 * r * f if case["save"] else 0)
        return {"bytes": 2 * values, "flops": 6 * r * m * f}
    return {"bytes": 2 * (3 * r * m + 2 * r * f + 6 * m * f), "flops": 12 * r * m * f}


def prepare(case, seed):
    dev = "cuda"
    gen = torch.Generator(device=dev).manual_seed(seed)
    t = DTYPES[case["dtype"]]

    def normal(*shape, scale=1.0):
        return (torch.randn(*shape, generator=gen, device=dev) * scale).to(t)

    s = {"case": dict(case)}
    r = case["rows"]
    if case["op"] == "linear":
        K, N = case["K"], case["N"]
        s.update(X=normal(r, K), WT=normal(K, N, scale=K ** -0.5),
                 bias=normal(N, scale=0.5) if case["bias"] else None,
                 residual=normal(r, N) if case["residual"] else None)
        return s
    m, f = case["d_model"], case["d_ff"]
    s.update(X=normal(r, m), WgT=normal(m, f, scale=m ** -0.5), WuT=normal(m, f, scale=m ** -0.5),
             WdT=normal(f, m, scale=f ** -0.5))
    if case["op"] == "gated":
        s.update(residual=normal(r, m) if case["residual"] else None)
    else:   # what the forward pass kept, and the gradient that comes in
        s.update(g=s["X"] @ s["WgT"], u=s["X"] @ s["WuT"], dY=normal(r, m))
    return s


def _act(name, z):
    """The activation and its slope, from sums, products, exponentials and comparisons."""
    if name == "none":
        return z, torch.ones_like(z)
    if name == "relu":
        on = (z > 0).to(z.dtype)
        return z * on, on
    if name == "silu":
        p = 1.0 / (1.0 + torch.exp(-z))
        return z * p, p * (1.0 + z * (1.0 - p))
    if name == "gelu":
        p = 0.5 * (1.0 + torch.erf(z * 0.5 ** 0.5))
        return z * p, p + z * torch.exp(-0.5 * z * z) * (2.0 * math.pi) ** -0.5
    c = (2.0 / math.pi) ** 0.5          # gelu_tanh: 0.5 (1 + tanh v) = 1 / (1 + exp(-2 v))
    p = 1.0 / (1.0 + torch.exp(-2.0 * c * (z + 0.044715 * z * z * z)))
    return z * p, p + z * p * (1.0 - p) * 2.0 * c * (1.0 + 3.0 * 0.044715 * z * z)


def run(s):
    c = s["case"]
    if own:
        import sparse_input_gemv_threshold_b200 as sig
        act = {"none": sig.ACT_NONE, "relu": sig.ACT_RELU, "gelu": sig.ACT_GELU,
               "gelu_tanh": sig.ACT_GELU_TANH, "silu": sig.ACT_SILU}[c["act"]]
        if c["op"] == "linear":
            return sig.linear_act(s["X"], s["WT"], bias=s["bias"], act=act, residual=s["residual"])
        if c["op"] == "gated":
            if not c["save"]:
                return sig.gated_mlp(s["X"], s["WgT"], s["WuT"], s["WdT"], act=act, residual=s["residual"])
            g = torch.empty((c["rows"], c["d_ff"]), dtype=s["X"].dtype, device=s["X"].device)
            u = torch.empty_like(g)
            Y = sig.gated_mlp(s["X"], s["WgT"], s["WuT"], s["WdT"], act=act, residual=s["residual"],
                              g_out=g, u_out=u)
            return {"Y": Y, "g": g, "u": u}
        dX, dWg, dWu, dWd = sig.gated_mlp_backward(s["dY"], s["X"], s["g"], s["u"], s["WgT"], s["WuT"],
                                                   s["WdT"], act=act)
        return {"dX": dX, "dWgT": dWg, "dWuT": dWu, "dWdT": dWd}
    t = s["X"].dtype
    X = s["X"].float()
    if c["op"] == "linear":
        z = X @ s["WT"].float()
        if s["bias"] is not None:
            z = z + s["bias"].float()
        y = _act(c["act"], z)[0]
        if s["residual"] is not None:
            y = y + s["residual"].float()
        return y.to(t)
    Wg, Wu, Wd = s["WgT"].float(), s["WuT"].float(), s["WdT"].float()
    if c["op"] == "gated":
        g, u = X @ Wg, X @ Wu
        Y = (_act(c["act"], g)[0] * u) @ Wd
        if s["residual"] is not None:
            Y = Y + s["residual"].float()
        return {"Y": Y.to(t), "g": g.to(t), "u": u.to(t)} if c["save"] else Y.to(t)
    g, u, dY = s["g"].float(), s["u"].float(), s["dY"].float()
    a, slope = _act(c["act"], g)
    dh = dY @ Wd.T
    dg, du = dh * u * slope, dh * a
    return {"dX": (dg @ Wg.T + du @ Wu.T).to(t), "dWgT": (X.T @ dg).to(t), "dWuT": (X.T @ du).to(t),
            "dWdT": ((a * u).T @ dY).to(t)}


def exact(case, seed):
    """The same outputs in 64 bits, from the definitions."""
    s = {k: v.double() if isinstance(v, torch.Tensor) else v for k, v in prepare(case, seed).items()}

    def phi(z):
        name = case["act"]
        if name == "relu":
            return z.clamp(min=0.0)
        if name == "silu":
            return z * torch.special.expit(z)
        if name == "gelu":
            return z * torch.special.ndtr(z)
        if name == "gelu_tanh":
            return 0.5 * z * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (z + 0.044715 * z ** 3)))
        return z

    if case["op"] == "linear":
        z = torch.einsum("rk,kn->rn", s["X"], s["WT"])
        y = phi(z if s["bias"] is None else z + s["bias"])
        return y if s["residual"] is None else y + s["residual"]
    if case["op"] == "gated":
        g = torch.einsum("rm,mf->rf", s["X"], s["WgT"])
        u = torch.einsum("rm,mf->rf", s["X"], s["WuT"])
        Y = torch.einsum("rf,fm->rm", phi(g) * u, s["WdT"])
        Y = Y if s["residual"] is None else Y + s["residual"]
        return {"Y": Y, "g": g, "u": u} if case["save"] else Y
    # the gradient of <Y, dY> in g and u by automatic differentiation, then the products
    g, u = s["g"].requires_grad_(), s["u"].requires_grad_()
    h = phi(g) * u
    dh = torch.einsum("rm,fm->rf", s["dY"], s["WdT"])
    dg, du = torch.autograd.grad((h * dh).sum(), (g, u))
    return {"dX": torch.einsum("rf,mf->rm", dg, s["WgT"]) + torch.einsum("rf,mf->rm", du, s["WuT"]),
            "dWgT": torch.einsum("rm,rf->mf", s["X"], dg), "dWuT": torch.einsum("rm,rf->mf", s["X"], du),
            "dWdT": torch.einsum("rf,rm->fm", h.detach(), s["dY"])}
