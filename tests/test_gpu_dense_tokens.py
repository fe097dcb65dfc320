"""GPU parity of the dense products for blocks of tokens (linear_act, gated_mlp,
gated_mlp_backward) with their definitions in float64.

Tolerances, derived per output before any run:
  products   every 16-bit x 16-bit product is exact in float32; each of the K
             additions of the tensor core errs by at most 2^-23 of the running
             sum's bound, so |z - z64| <= K 2^-23 sum|x w|.
  activation slope at most 1.13 (GELU), so an error e in z becomes at most
             1.13 e; evaluating act or its slope in float32 adds at most 2^-20
             in units of max(1, |z|): exp's relative error grows as |z| 2^-23,
             where act's sensitivity |z^2 p (1 - p)| stays below 1/2.
  rounding   at most half a step of the 16-bit type, relative to the value
             (fp16 2^-11, bf16 2^-8) or half the smallest fp16 subnormal.
"""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

TYPES = ["fp16", "bf16"]
ACTS = ["none", "relu", "gelu", "gelu_tanh", "silu"]
U = 2.0 ** -23


def dt(name):
    import torch
    return {"fp16": torch.float16, "bf16": torch.bfloat16}[name]


def code(sig, act):
    return {"none": sig.ACT_NONE, "relu": sig.ACT_RELU, "gelu": sig.ACT_GELU,
            "gelu_tanh": sig.ACT_GELU_TANH, "silu": sig.ACT_SILU}[act]


def normal(seed, *shape, dtype="fp16", scale=1.0):
    import torch
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(*shape, generator=gen, device="cuda") * scale).to(dt(dtype))


def act64(name, z):
    """(act(z), act'(z)) in float64."""
    import math
    import torch
    if name == "none":
        return z, torch.ones_like(z)
    if name == "relu":
        return z.clamp(min=0.0), (z > 0).double()
    if name == "silu":
        p = torch.special.expit(z)
        return z * p, p * (1 + z * (1 - p))
    if name == "gelu":
        p = torch.special.ndtr(z)
        return z * p, p + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    c = math.sqrt(2 / math.pi)
    th = torch.tanh(c * (z + 0.044715 * z ** 3))
    return 0.5 * z * (1 + th), 0.5 * (1 + th) + 0.5 * z * (1 - th * th) * c * (1 + 3 * 0.044715 * z * z)


def rounding(y64, err, dtype):
    """Half a step of the type at |y| + err, and half the smallest fp16 step."""
    import torch
    half = torch.finfo(dt(dtype)).eps / 2
    return err + half * (y64.abs() + err) + (2.0 ** -25 if dtype == "fp16" else 0.0)


def within(got, want, tol, what):
    import torch
    err = (got.double() - want).abs()
    bad = ~(err <= tol)
    if bool(bad.any()):
        at = torch.nonzero(bad)[0].tolist()
        i = tuple(at)
        raise AssertionError(f"{what}: {int(bad.sum())}/{bad.numel()} outputs out of tolerance; first {at} "
                             f"got {got[i].item()} want {want[i].item()} tol {tol[i].item()}")


def product(x, w):
    """x @ w in float64 and its error bound in float32."""
    x, w = x.double(), w.double()
    return x @ w, x.shape[1] * U * (x.abs() @ w.abs())


def act_err(act, z, ez):
    if act == "none":
        return ez
    return 1.13 * ez + 2.0 ** -20 * z.abs().clamp(min=1.0)


def check_linear(sig, rows, K, N, dtype, act, bias, residual, seed=0, **kw):
    X = normal(seed, rows, K, dtype=dtype)
    W = normal(seed + 1, K, N, dtype=dtype, scale=K ** -0.5)
    b = normal(seed + 2, N, dtype=dtype) if bias else None
    R = normal(seed + 3, rows, N, dtype=dtype) if residual else None
    Y = sig.linear_act(X, W, bias=b, act=code(sig, act), residual=R, **kw)
    z, ez = product(X, W)
    if bias:
        z = z + b.double()
        ez = ez + U * z.abs()
    y, e = act64(act, z)[0], act_err(act, z, ez)
    if residual:
        y = y + R.double()
        e = e + U * y.abs()
    within(Y, y, rounding(y, e, dtype), f"linear {rows}x{K}x{N} {dtype} {act}")
    return X, W, b, R, Y


# one token, a few, blocks around the 128- and 256-row tiles; widths around the
# 64-, 128- and 256-column tiles; depths from one value to many stages
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,K,N", [
    (1, 1, 8), (1, 8, 8), (1, 4096, 4096), (2, 63, 24), (3, 65, 136), (7, 128, 264), (16, 4096, 11008),
    (33, 200, 1000), (64, 1024, 120), (127, 72, 248), (128, 512, 256), (129, 64, 128), (255, 1000, 520),
    (256, 256, 2048), (257, 96, 512), (333, 4096, 4096), (1000, 136, 4104), (2048, 1024, 1024),
    (4096, 64, 8), (20000, 40, 72)])
def test_linear_shapes(sig, dtype, rows, K, N):
    ld = -(-K // 8) * 8
    X = normal(1, rows, ld, dtype=dtype)[:, :K]      # a stride of whole 16-byte groups for any K
    W = normal(2, K, N, dtype=dtype, scale=K ** -0.5)
    b, R = normal(3, N, dtype=dtype), normal(4, rows, N, dtype=dtype)
    y, e = product(X, W)
    within(sig.linear_act(X, W), y, rounding(y, e, dtype), f"{rows}x{K}x{N}")
    z = y + b.double()
    y, e = act64("silu", z)[0] + R.double(), act_err("silu", z, e + U * z.abs())
    Y = sig.linear_act(X, W, bias=b, act=sig.ACT_SILU, residual=R)
    within(Y, y, rounding(y, e + U * y.abs(), dtype), f"{rows}x{K}x{N} silu")


@pytest.mark.parametrize("rows", [5, 300])
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("bias,residual", [(False, False), (True, False), (False, True), (True, True)])
def test_linear_epilogues(sig, rows, act, bias, residual):
    for dtype in TYPES:
        check_linear(sig, rows, 256, 2312, dtype, act, bias, residual)


@pytest.mark.parametrize("rows", [3, 128, 200, 700])
def test_linear_row_strides_and_untouched_gaps(sig, rows):
    import torch
    K, N = 136, 264
    Xs = normal(5, rows, K + 24)
    Rs = normal(6, rows, N + 40)
    W = normal(7, K, N, scale=K ** -0.5)
    Ys = torch.full((rows + 1, N + 56), 7.0, dtype=torch.float16, device="cuda")
    X, R, Y = Xs[:, :K], Rs[:, 8:8 + N], Ys[:rows, 16:16 + N]
    out = sig.linear_act(X, W, residual=R, Y=Y)
    assert out.data_ptr() == Y.data_ptr()
    y, e = product(X, W)
    y = y + R.double()
    within(Y, y, rounding(y, e + U * y.abs(), "fp16"), "strided")
    assert bool((Ys[:, :16] == 7).all()) and bool((Ys[:, 16 + N:] == 7).all()) and bool((Ys[rows] == 7).all())
    # the contiguous call gives the same bits
    assert torch.equal(Y, sig.linear_act(X.contiguous(), W, residual=R.contiguous()))


@pytest.mark.parametrize("rows", [1, 100, 513])
def test_linear_adds_into_the_residual_in_place(sig, rows):
    import torch
    X, W, R = normal(8, rows, 320), normal(9, 320, 520, scale=0.05), normal(10, rows, 520)
    want = sig.linear_act(X, W, act=sig.ACT_GELU, residual=R)
    S = R.clone()
    sig.linear_act(X, W, act=sig.ACT_GELU, residual=S, Y=S)
    assert torch.equal(S, want)


@pytest.mark.parametrize("rows", [4, 400])
def test_special_values_stay_in_their_rows_and_columns(sig, rows):
    import torch
    K, N = 192, 512
    X, W = normal(11, rows, K), normal(12, K, N, scale=0.1)
    clean = sig.linear_act(X, W)
    X2, W2 = X.clone(), W.clone()
    X2[1, 5] = float("nan")
    X2[2, 7] = float("inf")
    Y = sig.linear_act(X2, W2)
    assert bool(Y[1].isnan().all())
    ref = X2[2].double() @ W2.double()
    assert torch.equal(torch.sign(Y[2]), torch.sign(ref).half()) and bool(Y[2].isinf().all())
    keep = [r for r in range(rows) if r not in (1, 2)]
    assert torch.equal(Y[keep], clean[keep])
    W2[:, 300] = float("inf")
    Y = sig.linear_act(X, W2)
    cols = [c for c in range(N) if c != 300]
    assert torch.equal(Y[:, cols], clean[:, cols])
    # activations at the ends: relu and the others pass +inf, NaN stays NaN
    b = torch.tensor([float("inf"), float("nan"), -float("inf"), 0.0] * (N // 4), dtype=torch.float16,
                     device="cuda")
    for act in ACTS[1:]:
        Y = sig.linear_act(X, W, bias=b, act=code(sig, act))
        assert bool((Y[:, 0::4] == float("inf")).all()) and bool(Y[:, 1::4].isnan().all()), act
    assert bool((sig.linear_act(X, W, bias=b, act=sig.ACT_RELU)[:, 2::4] == 0).all())
    # large arguments: act(z) is z or 0 there, with no overflow on the way
    b = torch.tensor([3e4, -3e4] * (N // 2), dtype=torch.float16, device="cuda")
    for act in ACTS[1:]:
        Y = sig.linear_act(X, W, bias=b, act=code(sig, act))
        assert bool((Y[:, 1::2] == 0).all()) and bool((Y[:, 0::2] > 2.9e4).all()), act


def test_overflow_of_the_output_type_rounds_to_infinity(sig):
    import torch
    X = torch.full((2, 64), 100.0, dtype=torch.float16, device="cuda")
    W = torch.full((64, 16), 100.0, dtype=torch.float16, device="cuda")
    assert bool((sig.linear_act(X, W) == float("inf")).all())       # 640000 > 65504


def gated_reference(X, Wg, Wu, act, dtype):
    g, eg = product(X, Wg)
    u, eu = product(X, Wu)
    a = act64(act, g)[0]
    ea = act_err(act, g, eg)
    h = a * u
    eh = u.abs() * ea + a.abs() * eu + ea * eu + U * h.abs()
    return g, eg, u, eu, h, eh


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,m,f,act", [
    (1, 8, 8, "silu"), (1, 4096, 11008, "silu"), (2, 72, 40, "gelu"), (9, 1024, 2816, "gelu_tanh"),
    (64, 264, 1000, "relu"), (128, 512, 1024, "silu"), (129, 136, 264, "none"), (300, 1000, 520, "silu"),
    (777, 1024, 2816, "gelu"), (2500, 256, 384, "silu")])
def test_gated_mlp(sig, dtype, rows, m, f, act):
    import torch
    X = normal(20, rows, m, dtype=dtype)
    Wg, Wu = (normal(21 + i, m, f, dtype=dtype, scale=m ** -0.5) for i in range(2))
    Wd = normal(23, f, m, dtype=dtype, scale=f ** -0.5)
    R = normal(24, rows, m, dtype=dtype)
    h, g, u = (torch.empty((rows, f), dtype=dt(dtype), device="cuda") for _ in range(3))
    Y = sig.gated_mlp(X, Wg, Wu, Wd, act=code(sig, act), residual=R, h_out=h, g_out=g, u_out=u)
    g64, eg, u64, eu, h64, eh = gated_reference(X, Wg, Wu, act, dtype)
    within(g, g64, rounding(g64, eg, dtype), "g")
    within(u, u64, rounding(u64, eu, dtype), "u")
    within(h, h64, rounding(h64, eh, dtype), "h")
    # strict: the down projection of the h that the call formed
    y, e = product(h, Wd)
    y = y + R.double()
    within(Y, y, rounding(y, e + U * y.abs(), dtype), "Y of h")
    # end to end: the error of h carried through the projection
    y2 = h64 @ Wd.double() + R.double()
    e2 = e + rounding(h64, eh, dtype) @ Wd.double().abs() + U * y2.abs()
    within(Y, y2, rounding(y2, e2, dtype), "Y")
    # the other ways to call it give the same bits
    assert torch.equal(Y, sig.gated_mlp(X, Wg, Wu, Wd, act=code(sig, act), residual=R))
    S = R.clone()
    sig.gated_mlp(X, Wg, Wu, Wd, act=code(sig, act), residual=S, Y=S)
    assert torch.equal(Y, S)


def backward_reference(dY, X, g, u, Wg, Wu, Wd, act, dtype):
    """Gradients in float64 and their tolerances."""
    g64, u64 = g.double(), u.double()
    a, s = act64(act, g64)
    ev = 2.0 ** -20 * g64.abs().clamp(min=1.0)        # act and its slope, evaluated in float32
    dh, edh = product(dY, Wd.T)
    dg, du, h = dh * u64 * s, dh * a, a * u64

    def kept(v, e):
        return rounding(v, e + 2 * U * v.abs(), dtype)
    edg = kept(dg, (u64 * s).abs() * edh + (dh * u64).abs() * ev + (u64.abs() * ev) * edh)
    edu = kept(du, a.abs() * edh + dh.abs() * ev + ev * edh)
    eh = kept(h, u64.abs() * ev)

    def prod(x, ex, w):
        w = w.double()
        y = x @ w
        return y, ex @ w.abs() + x.shape[1] * U * ((x.abs() + ex) @ w.abs())
    xg, exg = prod(dg, edg, Wg.T)
    xu, exu = prod(du, edu, Wu.T)
    f = dg.shape[1]
    both = (dg.abs() + edg) @ Wg.double().T.abs() + (du.abs() + edu) @ Wu.double().T.abs()
    out = {"dX": (xg + xu, edg @ Wg.double().T.abs() + edu @ Wu.double().T.abs() + 2 * f * U * both)}
    for name, v, e, x in (("dWgT", dg, edg, X), ("dWuT", du, edu, X)):
        y, t = prod(v.T.contiguous(), e.T.contiguous(), x)
        out[name] = (y.T, t.T)
    out["dWdT"] = prod(h.T.contiguous(), eh.T.contiguous(), dY)
    return {k: (y, rounding(y, t, dtype)) for k, (y, t) in out.items()}


def backward_inputs(rows, m, f, dtype, seed=30):
    X, dY = normal(seed, rows, m, dtype=dtype), normal(seed + 1, rows, m, dtype=dtype)
    g, u = normal(seed + 2, rows, f, dtype=dtype), normal(seed + 3, rows, f, dtype=dtype)
    Wg, Wu = (normal(seed + 4 + i, m, f, dtype=dtype, scale=m ** -0.5) for i in range(2))
    return dY, X, g, u, Wg, Wu, normal(seed + 6, f, m, dtype=dtype, scale=f ** -0.5)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,m,f,act", [
    (1, 8, 8, "silu"), (1, 1024, 2816, "silu"), (3, 72, 40, "gelu"), (16, 1024, 2816, "gelu_tanh"),
    (64, 264, 1000, "relu"), (65, 512, 1024, "silu"), (130, 136, 264, "none"), (300, 1000, 520, "gelu"),
    (777, 512, 1408, "silu"), (2500, 256, 384, "gelu_tanh")])
def test_gated_mlp_backward(sig, dtype, rows, m, f, act):
    import torch
    args = backward_inputs(rows, m, f, dtype)
    got = sig.gated_mlp_backward(*args, act=code(sig, act))
    ref = backward_reference(*args, act, dtype)
    for v, (k, (y, tol)) in zip(got, ref.items()):
        within(v, y, tol, f"{k} {rows}x{m}x{f} {act}")
    # a part of the gradients alone gives the same bits
    dX, *none = sig.gated_mlp_backward(*args, act=code(sig, act), want_weights=False)
    assert torch.equal(dX, got[0]) and none == [None] * 3
    none, *dW = sig.gated_mlp_backward(*args, act=code(sig, act), want_x=False)
    assert none is None and all(torch.equal(a, b) for a, b in zip(dW, got[1:]))


def test_gradients_against_differences(sig):
    """The formulas against central differences of the float64 forward pass, and
    the kernel against the differences at random directions."""
    import torch
    rows, m, f = 5, 24, 40
    X = normal(40, rows, m, dtype="fp16")
    Wg, Wu = normal(41, m, f, scale=m ** -0.5), normal(42, m, f, scale=m ** -0.5)
    Wd, dY = normal(43, f, m, scale=f ** -0.5), normal(44, rows, m)
    for act in ACTS:
        def loss(x, a, b, c):
            return ((act64(act, x @ a)[0] * (x @ b)) @ c * dY.double()).sum()
        p = [t.double() for t in (X, Wg, Wu, Wd)]
        g, u = p[0] @ p[1], p[0] @ p[2]
        got = sig.gated_mlp_backward(dY, X, g.half(), u.half(), Wg, Wu, Wd, act=code(sig, act))
        for i in range(4):
            d = torch.randn(p[i].shape, generator=torch.Generator().manual_seed(i), dtype=torch.float64).cuda()
            if act == "relu":   # keep the step away from the kink
                eps = min(1e-6, 1e-3 * g.abs().min().item())
            else:
                eps = 1e-5
            q1, q2 = list(p), list(p)
            q1[i], q2[i] = p[i] + eps * d, p[i] - eps * d
            diff = ((loss(*q1) - loss(*q2)) / (2 * eps)).item()
            # g and u, h, dg and du and the result are each rounded to fp16 (2^-11
            # relative): six roundings of terms whose magnitudes sum to at most this
            ref = backward_reference(dY, X, g.half(), u.half(), Wg, Wu, Wd, act, "fp16")
            tol = list(ref.values())[i][1]
            s = act64(act, g)[1].abs() + 1.13
            spread = (g.abs() + u.abs() + 1) * 2.0 ** -11 * 4 * (1 + s)
            dh = dY.double().abs() @ p[3].T.abs()
            lim = [(dh * spread) @ p[1].T.abs() + (dh * spread) @ p[2].T.abs(), p[0].T.abs() @ (dh * spread),
                   p[0].T.abs() @ (dh * spread), (spread * (1 + u.abs())).T @ dY.double().abs()][i]
            assert abs((got[i].double() * d).sum().item() - diff) <= ((tol + lim) * d.abs()).sum().item(), (act, i)


@pytest.mark.parametrize("rows", [5, 90, 300])
def test_nothing_between_the_rows_is_read(sig, rows):
    """NaN in the gaps of strided inputs, behind the last row and around the
    weights reaches no output."""
    import torch
    K, N = 100, 264

    def gapped(seed, r, c, ld, scale=1.0):
        buf = torch.full((r + 2, ld), float("nan"), dtype=torch.float16, device="cuda")
        buf[1:r + 1, 8:8 + c] = normal(seed, r, c, scale=scale)
        return buf[1:r + 1, 8:8 + c]

    X, R = gapped(100, rows, K, 136), gapped(101, rows, N, 304)
    flat = torch.full((K * N + 128,), float("nan"), dtype=torch.float16, device="cuda")
    flat[64:64 + K * N] = normal(102, K, N, scale=0.1).reshape(-1)
    W = flat[64:64 + K * N].view(K, N)
    y, e = product(X, W)
    y = y + R.double()
    within(sig.linear_act(X, W, residual=R), y, rounding(y, e + U * y.abs(), "fp16"), "gaps")
    m, f = 104, 136
    X, dY = gapped(103, rows, m, 120), gapped(104, rows, m, 144)
    g, u = normal(105, rows, f), normal(106, rows, f)
    Wg, Wu, Wd = normal(107, m, f, scale=0.1), normal(108, m, f, scale=0.1), normal(109, f, m, scale=0.1)
    got = sig.gated_mlp_backward(dY, X, g, u, Wg, Wu, Wd)
    want = sig.gated_mlp_backward(dY.contiguous(), X.contiguous(), g, u, Wg, Wu, Wd)
    assert all(torch.equal(a, b) for a, b in zip(got, want)) and all(bool(v.isfinite().all()) for v in got)


@pytest.mark.parametrize("rows", [3, 200])
def test_outputs_in_the_place_of_inputs(sig, rows):
    """The places that the documentation allows give the same bits; the others are refused."""
    import torch
    args = backward_inputs(rows, 264, 520, "fp16", seed=110)
    dY, X, g, u, Wg, Wu, Wd = args
    want = sig.gated_mlp(X, Wg, Wu, Wd, residual=X)
    S = X.clone()
    sig.gated_mlp(S, Wg, Wu, Wd, residual=S, Y=S)
    assert torch.equal(S, want)
    dX = sig.gated_mlp_backward(*args, want_weights=False)[0]
    for i in (0, 1):
        moved = [t.clone() for t in args]
        sig.gated_mlp_backward(*moved, dX=moved[i], want_weights=False)
        assert torch.equal(moved[i], dX)
        with pytest.raises(sig.SigError):
            sig.gated_mlp_backward(*moved, dX=moved[i])
    sq = normal(117, 264, 264)
    with pytest.raises(sig.SigError):
        sig.linear_act(X, sq, Y=X)


def test_two_threads(sig):
    """Two host threads, each on its own stream."""
    import threading
    import torch
    sets = [backward_inputs(100 + 200 * i, 264, 520, "fp16", seed=150 + 10 * i) for i in range(2)]
    want = [(sig.gated_mlp(s[1], *s[4:]), *sig.gated_mlp_backward(*s)) for s in sets]
    torch.cuda.synchronize()
    wrong = []

    def work(i):
        with torch.cuda.stream(torch.cuda.Stream()):
            for _ in range(20):
                got = (sig.gated_mlp(sets[i][1], *sets[i][4:]), *sig.gated_mlp_backward(*sets[i]))
            torch.cuda.current_stream().synchronize()
            wrong.extend(k for k, (a, b) in enumerate(zip(got, want[i])) if not torch.equal(a, b))
    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert wrong == []


def test_the_first_call_may_be_captured():
    """In a process that has called nothing of the library, the first calls go
    straight into a graph; its replay gives the eager bits."""
    import os
    import subprocess
    import sys
    code = """
import torch, sparse_input_gemv_threshold_b200 as sig
X = torch.randn(300, 256, device='cuda').half(); W = torch.randn(256, 512, device='cuda').half() * 0.1
D = torch.randn(512, 256, device='cuda').half() * 0.1
s = torch.cuda.Stream(); g = torch.cuda.CUDAGraph()
torch.cuda.synchronize()
with torch.cuda.graph(g, stream=s):
    a = sig.gated_mlp(X, W, W, D); b = sig.gated_mlp(X[:3], W, W, D)
g.replay(); torch.cuda.synchronize()
assert torch.equal(a, sig.gated_mlp(X, W, W, D)) and torch.equal(b, sig.gated_mlp(X[:3], W, W, D))
assert sig.take_device_error() == 0 and bool(a.isfinite().all())
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]


def test_beside_the_other_tensor_core_kernels(sig):
    """Blocks of tokens on one stream and the N:M GEMMs on another, and in turn on
    one: kernels that ask for tensor memory side by side."""
    import torch
    import oracle
    import workloads
    WT, Xn = workloads.nm_tokens(7, rows=512, d=512, d_out=512)
    dW, dXn = torch.from_numpy(WT).cuda(), torch.from_numpy(Xn).cuda()
    Y64, B = oracle.nm_gemm(Xn, WT, oracle.nm_mask(Xn, 2, 4))
    X, W = normal(160, 40, 512), normal(161, 512, 1096, scale=0.05)
    Xb = normal(162, 700, 512)
    want = sig.linear_act(X, W), sig.linear_act(Xb, W)
    wantn = sig.nm_act_gemm(dXn, dW, 2, 4)
    assert np.all(np.abs(wantn.cpu().numpy().astype(np.float64) - Y64) <= 2e-3 * B + 2.0 ** -24)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(30):
        a = sig.linear_act(X, W, stream=s1), sig.linear_act(Xb, W, stream=s1)
        n2 = sig.nm_act_gemm(dXn, dW, 2, 4, stream=s2)
        n1 = sig.nm_act_gemm(dXn, dW, 2, 4, stream=s1)
        b = sig.linear_act(X, W, stream=s2)
    torch.cuda.synchronize()
    assert torch.equal(a[0], want[0]) and torch.equal(a[1], want[1]) and torch.equal(b, want[0])
    assert torch.equal(n1, wantn) and torch.equal(n2, wantn)


def test_empty_blocks(sig):
    import torch
    X, W = normal(50, 0, 64), normal(51, 64, 32)
    assert sig.linear_act(X, W).shape == (0, 32)
    assert sig.gated_mlp(X, W, W, W.T.contiguous()).shape == (0, 64)
    e = torch.empty((0, 32), dtype=torch.float16, device="cuda")
    dX, *dW = sig.gated_mlp_backward(X, X, e, e, W, W, W.T.contiguous())
    assert dX.shape == (0, 64) and all(bool((w == 0).all()) for w in dW)


@pytest.mark.parametrize("dtype", TYPES)
def test_empty_block_with_a_part_of_the_gradients(sig, dtype):
    """No tokens reached the block (frozen weights, or weight gradients alone)."""
    X, W = normal(50, 0, 64, dtype=dtype), normal(51, 64, 32, dtype=dtype)
    e, Wd = normal(52, 0, 32, dtype=dtype), W.T.contiguous()
    dX, *none = sig.gated_mlp_backward(X, X, e, e, W, W, Wd, want_weights=False)
    assert dX.shape == (0, 64) and none == [None] * 3
    none, *dW = sig.gated_mlp_backward(X, X, e, e, W, W, Wd, want_x=False)
    assert none is None and all(bool((w == 0).all()) for w in dW)
    assert [w.shape for w in dW] == [(64, 32), (64, 32), (32, 64)]


def test_refusals_of_the_binding(sig):
    import torch
    X, W = normal(52, 4, 64), normal(53, 64, 32)
    Wd = W.T.contiguous()
    with pytest.raises(ValueError):
        sig.linear_act(X, W.T)                                   # shape
    with pytest.raises(ValueError):
        sig.linear_act(X, normal(1, 32, 64).T)                   # a weight that is not contiguous
    with pytest.raises(ValueError):
        sig.linear_act(normal(1, 64, 4).T, W)                    # tokens without contiguous rows
    with pytest.raises(TypeError):
        sig.linear_act(X, W.bfloat16())
    with pytest.raises(ValueError):
        sig.linear_act(X, W, bias=normal(1, 31))
    with pytest.raises(ValueError):
        sig.linear_act(X, W, residual=normal(1, 4, 64))
    with pytest.raises(sig.SigError):
        sig.linear_act(X, W, act=9)
    with pytest.raises(sig.SigError):
        sig.linear_act(normal(1, 4, 68)[:, :64], W)              # a stride of 68 entries
    with pytest.raises(sig.SigError):
        sig.linear_act(X, W, residual=normal(1, 1, 32).expand(4, 32))
    with pytest.raises(sig.SigError):
        sig.linear_act(X, normal(1, 64, 12))                     # N % 8
    with pytest.raises(sig.SigError):
        sig.gated_mlp(X, W, W, Wd, g_out=normal(1, 4, 32))       # g without u
    with pytest.raises(ValueError):
        sig.gated_mlp(X, W, W, W)
    with pytest.raises(sig.SigError):
        sig.gated_mlp_backward(X, X, normal(1, 4, 32), normal(1, 4, 32), W, W, Wd, want_x=False,
                               want_weights=False)
    torch.cuda.synchronize()


@pytest.mark.parametrize("rows", [3, 500])
def test_runs_give_the_same_bits(sig, rows):
    import torch
    args = backward_inputs(rows, 520, 1096, "bf16")
    first = sig.gated_mlp_backward(*args)
    y = sig.gated_mlp(args[1], *args[4:])
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(first, sig.gated_mlp_backward(*args)))
        assert torch.equal(y, sig.gated_mlp(args[1], *args[4:]))


def test_streams_at_once(sig):
    """Two streams run the block at the same time; each call's outputs and
    workspace belong to its stream."""
    import torch
    sets = [backward_inputs(200, 512, 1408, "fp16", seed=60 + 10 * i) for i in range(2)]
    want = [(sig.gated_mlp(s[1], *s[4:]), *sig.gated_mlp_backward(*s)) for s in sets]
    streams = [torch.cuda.Stream() for _ in sets]
    torch.cuda.synchronize()
    got = [None, None]
    for _ in range(5):
        for i, s in enumerate(sets):
            got[i] = (sig.gated_mlp(s[1], *s[4:], stream=streams[i]),
                      *sig.gated_mlp_backward(*s, stream=streams[i]))
    torch.cuda.synchronize()
    for w, g in zip(want, got):
        assert all(torch.equal(a, b) for a, b in zip(w, g))


def test_two_captured_graphs_share_nothing(sig):
    """Forward and backward captured twice on one stream, replayed at the same
    time on two streams."""
    import torch
    sets = [backward_inputs(130, 512, 1096, "bf16", seed=90 + 10 * i) for i in range(2)]
    want = [(sig.gated_mlp(s[1], *s[4:]), *sig.gated_mlp_backward(*s)) for s in sets]
    st = torch.cuda.Stream()
    graphs, outs = [], []
    torch.cuda.synchronize()
    for s in sets:
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr, stream=st):
            outs.append((sig.gated_mlp(s[1], *s[4:]), *sig.gated_mlp_backward(*s)))
        graphs.append(gr)
    streams = [torch.cuda.Stream() for _ in sets]
    for _ in range(4):
        for gr, s2 in zip(graphs, streams):
            with torch.cuda.stream(s2):
                gr.replay()
    torch.cuda.synchronize()
    for w, g in zip(want, outs):
        assert all(torch.equal(a, b) for a, b in zip(w, g))
    # new inputs in the captured buffers
    sets[0][1].copy_(sets[1][1])
    graphs[0].replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0][0], sig.gated_mlp(sets[0][1], *sets[0][4:]))


def test_block_and_single_token_agree(sig):
    """The dense MLP of this library for one token (every neuron kept) and the
    block form give the same hidden vector and output up to their roundings."""
    import torch
    m, f = 1024, 2816
    X = normal(70, 5, m)
    Wg, Wu, Wd = normal(71, m, f, scale=0.02), normal(72, m, f, scale=0.02), normal(73, f, m, scale=0.02)
    h = torch.empty((5, f), dtype=torch.float16, device="cuda")
    Y = sig.gated_mlp(X, Wg, Wu, Wd, h_out=h)
    norms = sig.row_norms(Wd)
    _, _, _, _, h64, eh = gated_reference(X, Wg, Wu, "silu", "fp16")
    for r in range(5):
        h1 = torch.empty(f, dtype=torch.float16, device="cuda")
        y1 = sig.gated_mlp_sparse(X[r].contiguous(), Wg, Wu, Wd, norms, 0.0, h_out=h1)
        tol_h = 2 * rounding(h64[r], eh[r], "fp16")
        within(h[r], h1.double(), tol_h, "h")
        y64, e = product(h1[None], Wd)
        tol = 2 * rounding(y64[0], e[0], "fp16") + tol_h @ Wd.double().abs()
        within(Y[r], y1.double(), tol, "y")


def test_a_training_step_through_the_block(sig):
    """Attention output projection into the residual stream, the gated MLP on it,
    its gradients, and the projection's own gradients' operands: the calls of a
    step in order on one stream, each against the float64 value of its inputs."""
    import torch
    rows, m, f, dtype = 260, 512, 1408, "bf16"
    ctx = normal(80, rows, m, dtype=dtype)
    Wo = normal(81, m, m, dtype=dtype, scale=m ** -0.5)
    stream0 = normal(82, rows, m, dtype=dtype)
    Wg, Wu = (normal(83 + i, m, f, dtype=dtype, scale=m ** -0.5) for i in range(2))
    Wd = normal(85, f, m, dtype=dtype, scale=f ** -0.5)
    X = sig.linear_act(ctx, Wo, residual=stream0)
    g, u = (torch.empty((rows, f), dtype=dt(dtype), device="cuda") for _ in range(2))
    Y = sig.gated_mlp(X, Wg, Wu, Wd, residual=X, g_out=g, u_out=u)
    dY = normal(86, rows, m, dtype=dtype)
    grads = sig.gated_mlp_backward(dY, X, g, u, Wg, Wu, Wd)
    y, e = product(ctx, Wo)
    y = y + stream0.double()
    within(X, y, rounding(y, e + U * y.abs(), dtype), "X")
    g64, eg, u64, eu, h64, eh = gated_reference(X, Wg, Wu, "silu", dtype)
    within(g, g64, rounding(g64, eg, dtype), "g")
    y2 = h64 @ Wd.double() + X.double()
    e2 = rounding(h64, eh, dtype) @ Wd.double().abs() + f * U * (h64.abs() @ Wd.double().abs()) + U * y2.abs()
    within(Y, y2, rounding(y2, e2, dtype), "Y")
    for v, (k, (w, tol)) in zip(grads, backward_reference(dY, X, g, u, Wg, Wu, Wd, "silu", dtype).items()):
        within(v, w, tol, k)


def test_outputs_beyond_32_bit_offsets(sig):
    """More than 2^31 outputs: 270 000 tokens to 8192 columns, the last rows and
    a sample of the others against float64."""
    import torch
    rows, K, N = 270_000, 40, 8192
    X, W = normal(120, rows, K), normal(121, K, N, scale=K ** -0.5)
    b = normal(122, N)
    Y = sig.linear_act(X, W, bias=b, act=sig.ACT_RELU)
    at = torch.cat([torch.randint(0, rows, (400,), generator=torch.Generator().manual_seed(5)),
                    torch.tensor([0, 262143, 262144, rows - 1])]).cuda()
    z, e = product(X[at], W)
    z = z + b.double()
    y, e = z.clamp(min=0.0), e + U * z.abs()
    within(Y[at], y, rounding(y, e, "fp16"), "270000 x 40 x 8192")


# the listed kernels' borders: one block of tokens and several in the few-token
# kernel, its join in its own place (to 96 tokens) and in the ring's, odd numbers
# of parts along K, whole and half tiles of the pair kernel, one and many waves
@pytest.mark.parametrize("rows,K,N", [
    (15, 64, 4096), (17, 640, 128), (48, 1024, 384), (63, 4096, 1000), (65, 1024, 136), (66, 11008, 136),
    (112, 2048, 2816), (176, 5632, 512), (257, 4096, 256), (515, 5632, 1024), (640, 1024, 2816),
    (1024, 520, 1024), (1025, 64, 9728), (1281, 320, 5000), (9473, 128, 520)])
def test_linear_kernel_borders(sig, rows, K, N):
    for dtype in TYPES:
        check_linear(sig, rows, K, N, dtype, "gelu", True, True, seed=rows)
        check_linear(sig, rows, K, N, dtype, "none", False, False, seed=rows + 7)


# blocks of 16 to 256 tokens joined from 1 to 8 parts: shares of a part that end
# within a group of 16 tokens, a last block of a few tokens (fewer than there are
# parts), one and two CTAs an SM, the join beside the ring and in its place
@pytest.mark.parametrize("rows,K,N", [
    (5, 520, 8), (16, 11008, 4096), (17, 136, 264), (31, 520, 1000), (33, 520, 136), (49, 11008, 520),
    (81, 11008, 1000), (127, 4096, 2816), (129, 520, 520), (129, 4096, 2816), (177, 11008, 1000),
    (193, 11008, 264), (209, 11008, 1000), (241, 11008, 2816), (255, 64, 8200), (257, 11008, 520),
    (257, 4096, 2816), (333, 4096, 520), (333, 4096, 2816), (400, 4096, 520), (500, 11008, 1000),
    (641, 4096, 136), (641, 11008, 264), (777, 520, 136), (777, 11008, 520)])
def test_join_of_the_parts(sig, rows, K, N):
    for dtype in TYPES:
        check_linear(sig, rows, K, N, dtype, "silu", True, True, seed=rows + 3)
        check_linear(sig, rows, K, N, dtype, "none", False, False, seed=rows + 4)


@pytest.mark.parametrize("rows,m,f,act", [
    (17, 520, 264, "gelu"), (33, 2048, 1000, "silu"), (65, 264, 2056, "gelu_tanh"), (95, 4096, 392, "relu"),
    (130, 1024, 136, "none"), (255, 72, 2104, "silu"), (401, 1024, 520, "silu")])
def test_joins_of_the_gated_block(sig, rows, m, f, act):
    for dtype in TYPES:
        test_gated_mlp(sig, dtype, rows, m, f, act)
        test_gated_mlp_backward(sig, dtype, rows, m, f, act)


# the pairs with the tokens as N: tiles of 64 to 256 tokens, one wave and many, more
# token tiles than are walked together, last tiles of a few tokens and columns
@pytest.mark.parametrize("rows,K,N", [
    (333, 2048, 5000), (515, 520, 8200), (777, 1000, 8200), (900, 2048, 8200), (1025, 520, 1000),
    (1281, 1000, 1000), (1300, 1000, 8200), (1500, 2048, 8200), (2100, 1000, 1000), (6000, 2048, 2056),
    (1100, 520, 8200), (1300, 1000, 5000), (5000, 520, 1000)])
def test_tall_tiles(sig, rows, K, N):
    for dtype in TYPES:
        check_linear(sig, rows, K, N, dtype, "gelu", True, True, seed=rows + 5)
        check_linear(sig, rows, K, N, dtype, "none", False, False, seed=rows + 6)


@pytest.mark.parametrize("rows,m,f,act", [
    (520, 1000, 2120, "silu"), (777, 1024, 2816, "gelu_tanh"), (1025, 520, 520, "relu"), (1281, 1000, 1000, "gelu"),
    (2101, 1000, 1000, "silu"), (777, 1000, 8200, "silu"), (1300, 1000, 5000, "gelu"),
    (1300, 4104, 1000, "gelu_tanh")])
def test_tall_tiles_of_the_gated_block(sig, rows, m, f, act):
    for dtype in TYPES:
        test_gated_mlp(sig, dtype, rows, m, f, act)
        test_gated_mlp_backward(sig, dtype, rows, m, f, act)


@pytest.mark.parametrize("rows,K,N", [(1281, 1000, 1000), (1300, 1000, 5000)])
def test_tall_tiles_strided_in_place_and_beside_nan(sig, rows, K, N):
    import torch
    buf = torch.full((rows + 2, K + 40), float("nan"), dtype=torch.float16, device="cuda")
    X = buf[1:rows + 1, 16:16 + K]
    X.copy_(normal(150, rows, K))
    W = normal(151, K, N, scale=K ** -0.5)
    out = torch.full((rows + 1, N + 56), 7.0, dtype=torch.float16, device="cuda")
    Y = out[:rows, 24:24 + N]
    Y.copy_(normal(152, rows, N))
    y, e = product(X, W)
    y = y + Y.double()
    sig.linear_act(X, W, residual=Y, Y=Y)
    within(Y, y, rounding(y, e + U * y.abs(), "fp16"), "in place, strided")
    assert bool((out[:, :24] == 7).all()) and bool((out[:, 24 + N:] == 7).all()) and bool((out[rows] == 7).all())
    # NaN and infinity stay in their rows and columns
    X = X.contiguous()
    clean = sig.linear_act(X, W)
    X[700, 3], W[5, N - 1] = float("nan"), float("inf")
    Y = sig.linear_act(X, W)
    assert bool(Y[700].isnan().all()) and not bool(Y[:, N - 1].isfinite().any())
    keep = [r for r in range(rows) if r != 700]
    assert torch.equal(Y[keep, :N - 1], clean[keep, :N - 1])


def test_tall_tiles_on_two_streams_and_in_graphs(sig):
    """Two captured gated blocks replayed at once on two streams, beside eager
    calls on a third, give the bits of calls made alone."""
    import torch
    rows, m, f = 777, 1000, 8200
    blocks = [backward_inputs(rows, m, f, "fp16", seed=180 + 10 * i) for i in range(3)]

    def run(b):
        return [sig.gated_mlp(b[1], *b[4:]), *sig.gated_mlp_backward(*b)]
    want = [run(b) for b in blocks]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    graphs, got = [], []
    for b, s in zip(blocks[:2], streams):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            got.append(run(b))
        graphs.append(g)
    for _ in range(5):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        with torch.cuda.stream(streams[2]):
            eager = run(blocks[2])
    torch.cuda.synchronize()
    for a, b in zip(want, got + [eager]):
        assert all(torch.equal(x, y) for x, y in zip(a, b))
    assert sig.take_device_error() == 0


@pytest.mark.parametrize("rows,m,f", [(1281, 1000, 1000), (1300, 1000, 5000), (1300, 4104, 1000)])
def test_tall_tiles_give_up_and_recover(sig, rows, m, f):
    """Waits that give up at once, in the producer, the issuer and the epilogues,
    end the launch with an error, and the calls after it are right."""
    import torch
    args = backward_inputs(rows, m, f, "bf16", seed=160)
    R = normal(170, rows, f, dtype="bf16")

    def run():
        return [sig.linear_act(args[1], args[4], residual=R), sig.gated_mlp(args[1], *args[4:]),
                *sig.gated_mlp_backward(*args)]
    want = run()
    assert sig.take_device_error() == 0
    for limit in (1, 64, 20000):
        try:
            sig.set_wait_limit(limit)
            run()
            torch.cuda.synchronize()
            assert limit > 64 or sig.take_device_error() != 0
        finally:
            sig.set_wait_limit(0)
            sig.take_device_error()
        assert all(torch.equal(a, b) for a, b in zip(want, run()))
        assert sig.take_device_error() == 0


@pytest.mark.parametrize("rows", [600, 1500])
def test_a_wait_that_gives_up_lets_the_epilogues_reads_land(sig, rows):
    """The same for the epilogues that read while they wait: the residual, and g
    and u of the backward pass."""
    import torch
    args = backward_inputs(rows, 256, 1096, "fp16", seed=130)
    R = normal(140, rows, 1096)
    W = args[4]
    want = [sig.linear_act(args[1], W, residual=R), *sig.gated_mlp_backward(*args)]
    assert sig.take_device_error() == 0
    try:
        sig.set_wait_limit(64)
        sig.linear_act(args[1], W, residual=R)
        sig.gated_mlp_backward(*args)
        torch.cuda.synchronize()
        assert sig.take_device_error() != 0
    finally:
        sig.set_wait_limit(0)
    got = [sig.linear_act(args[1], W, residual=R), *sig.gated_mlp_backward(*args)]
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    assert sig.take_device_error() == 0


@pytest.mark.parametrize("act", ["gelu", "gelu_tanh", "silu", "relu"])
def test_activations_and_slopes_over_their_range(sig, act):
    """Every activation and its slope at values from deep in one tail to the
    other: an identity weight, so that the kernel's sum is the argument itself."""
    import torch
    n = 1024
    for dtype in TYPES:
        z = torch.linspace(-12.0, 12.0, 512 * n, dtype=torch.float64, device="cuda").reshape(512, n).to(dt(dtype))
        eye = torch.eye(n, dtype=dt(dtype), device="cuda")
        a, slope = act64(act, z.double())
        err = 2.0 ** -20 * z.double().abs().clamp(min=1.0)
        within(sig.linear_act(z, eye, act=code(sig, act)), a, rounding(a, err, dtype), "act")
        within(sig.linear_act(z[:7], eye, act=code(sig, act)), a[:7], rounding(a, err, dtype)[:7], "act, few")
        # dX with dh = 1 (WdT = I, dY = 1), u = 1 and unit gate weights is act'(g) + act(g) u'
        one, zero = torch.ones_like(z), torch.zeros(n, n, dtype=dt(dtype), device="cuda")
        dX = sig.gated_mlp_backward(one, z, z, one, eye, zero, eye, act=code(sig, act), want_weights=False)[0]
        e1 = rounding(slope, err, dtype)             # dg rounded to the type, then dX = dg
        within(dX, slope, rounding(slope, e1, dtype), "slope")


@pytest.mark.parametrize("rows", [4, 600])
def test_a_wait_that_gives_up_is_reported(sig, rows):
    """With the wait limit at a few cycles the first wait for data gives up; the
    error word says so, and with the limit restored the next call is right."""
    import ctypes
    import torch
    X, W = normal(87, rows, 1024), normal(88, 1024, 2048, scale=0.03)
    want = sig.linear_act(X, W)
    assert sig.take_device_error() == 0
    try:
        sig.set_wait_limit(64)
        sig.linear_act(X, W)
        torch.cuda.synchronize()
        word = ctypes.c_uint(0)
        st = sig._lib.sig_take_device_error(ctypes.byref(word), None)
    finally:
        sig.set_wait_limit(0)
    assert st == 6 and word.value != 0
    assert torch.equal(sig.linear_act(X, W), want)
    assert sig.take_device_error() == 0
    assert np.isfinite(want.float().cpu().numpy()).all()


def test_calls_are_outside_autograd(sig):
    """As documented: outputs carry no gradient, and no .grad is touched."""
    import torch
    args = [t.requires_grad_() for t in backward_inputs(5, 64, 136, "bf16", seed=300)]
    Y = sig.gated_mlp(args[1], *args[4:])
    outs = [Y, sig.linear_act(args[1], args[4]), *sig.gated_mlp_backward(*args)]
    assert not any(t.requires_grad for t in outs) and all(t.grad is None for t in args)
    with torch.no_grad():
        assert torch.equal(Y, sig.gated_mlp(args[1], *args[4:]))
