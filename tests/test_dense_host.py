"""Host-side checks of linear_act, gated_mlp and gated_mlp_backward: every call
here fails argument validation (or is an empty block), so nothing is launched
and no address is dereferenced."""
import ctypes
import os

import pytest

from tests.conftest import ROOT, load_builder

OK, NULL, SHAPE, ALIGN, WORKSPACE, CUDA, TIMEOUT, ARG = range(8)
P = 1 << 40                # an aligned, never dereferenced "device" address
ODD = P + 2
OUT = P + (1 << 32)        # another, for outputs
F16, BF16 = 0, 1
BIG = 1 << 60


@pytest.fixture(scope="module")
def lib():
    path = load_builder().build()
    lib = ctypes.CDLL(path)
    import sparse_input_gemv_threshold_b200 as sig
    for name, (res, args) in sig._SIGNATURES.items():
        fn = getattr(lib, name)
        fn.restype, fn.argtypes = res, args
    return lib


def linear(lib, **kw):
    a = dict(X=P, rows=4, K=64, ldx=64, WT=P, N=64, bias=None, act=0, residual=None, ldr=0, Y=OUT, ldy=64,
             dtype=F16)
    a.update(kw)
    return lib.linear_act(*a.values(), None)


def gated(lib, **kw):
    a = dict(X=P, rows=4, ldx=64, WgT=P, WuT=P, WdT=P, d_model=64, d_ff=128, act=4, residual=None, ldr=0,
             Y=OUT, ldy=64, h_out=None, g_out=None, u_out=None, dtype=F16, ws=P, ws_bytes=BIG)
    a.update(kw)
    return lib.gated_mlp(*a.values(), None)


def backward(lib, **kw):
    a = dict(dY=P, lddy=64, X=P, ldx=64, rows=4, g=P, u=P, WgT=P, WuT=P, WdT=P, d_model=64, d_ff=128,
             act=4, dX=OUT, lddx=64, dWgT=P, dWuT=P, dWdT=P, dtype=F16, ws=P, ws_bytes=BIG)
    a.update(kw)
    return lib.gated_mlp_backward(*a.values(), None)


def test_linear_act_validation(lib):
    for name in ("X", "WT", "Y"):
        assert linear(lib, **{name: None}) == NULL, name
        assert linear(lib, **{name: ODD}) == ALIGN, name
    assert linear(lib, bias=ODD) == ALIGN
    assert linear(lib, residual=ODD, ldr=64) == ALIGN
    for kw in (dict(rows=-1), dict(rows=(1 << 24) + 1), dict(K=0), dict(K=(1 << 20) + 1), dict(N=0),
               dict(N=60), dict(N=(1 << 20) + 8), dict(ldx=56), dict(ldy=56), dict(ldx=(1 << 30) + 8),
               dict(residual=P, ldr=0), dict(residual=P, ldr=56)):
        assert linear(lib, **kw) == SHAPE, kw
    for kw in (dict(ldx=65), dict(ldy=68), dict(residual=P, ldr=66), dict(K=65, ldx=65)):
        assert linear(lib, **kw) == ALIGN, kw
    for kw in (dict(dtype=2), dict(dtype=-1), dict(act=5), dict(act=-1)):
        assert linear(lib, **kw) == ARG, kw
    # an empty block touches no pointer
    assert linear(lib, rows=0, X=None, WT=None, Y=None) == OK
    # outputs in the place of what is still read
    Q = P + (1 << 30)
    assert linear(lib, X=Q, Y=Q) == ARG
    assert linear(lib, residual=Q, ldr=72, Y=Q, X=P) == ARG


def test_gated_mlp_validation(lib):
    for name in ("X", "WgT", "WuT", "WdT", "Y"):
        assert gated(lib, **{name: None}) == NULL, name
        assert gated(lib, **{name: ODD}) == ALIGN, name
    assert gated(lib, g_out=P) == NULL and gated(lib, u_out=P) == NULL
    for kw in (dict(h_out=ODD), dict(g_out=ODD, u_out=P), dict(g_out=P, u_out=ODD), dict(ws=P + 16),
               dict(ldx=68), dict(residual=P, ldr=68), dict(ldy=68)):
        assert gated(lib, **kw) == ALIGN, kw
    for kw in (dict(rows=-1), dict(d_model=60), dict(d_model=0), dict(d_ff=12), dict(d_ff=1 << 21),
               dict(ldx=56), dict(ldy=8), dict(residual=P, ldr=56)):
        assert gated(lib, **kw) == SHAPE, kw
    assert gated(lib, dtype=7) == ARG and gated(lib, act=9) == ARG
    need = lib.sig_workspace_bytes(10, 64, 128, 4)
    assert need == 4 * 128 * 2
    assert gated(lib, ws=None) == WORKSPACE and gated(lib, ws_bytes=need - 1) == WORKSPACE
    assert gated(lib, rows=0, X=None, Y=None, ws=None, ws_bytes=0) == OK
    assert gated(lib, residual=OUT, ldr=72) == ARG                  # Y with the residual's rows elsewhere


def test_gated_mlp_backward_validation(lib):
    for name in ("dY", "X", "g", "u", "WgT", "WuT", "WdT"):
        assert backward(lib, **{name: None}) == NULL, name
        assert backward(lib, **{name: ODD}) == ALIGN, name
    assert backward(lib, dWgT=None) == NULL and backward(lib, dWuT=None) == NULL
    assert backward(lib, dX=None, dWgT=None, dWuT=None, dWdT=None) == NULL
    for kw in (dict(dX=ODD), dict(dWgT=ODD), dict(dWuT=ODD), dict(dWdT=ODD), dict(lddy=68), dict(ldx=68),
               dict(lddx=68), dict(ws=P + 128)):
        assert backward(lib, **kw) == ALIGN, kw
    for kw in (dict(rows=-1), dict(d_model=20), dict(d_ff=4), dict(lddy=8), dict(ldx=8), dict(lddx=8)):
        assert backward(lib, **kw) == SHAPE, kw
    assert backward(lib, dtype=3) == ARG and backward(lib, act=5) == ARG
    Q = P + (1 << 30)
    for kw in (dict(dX=Q, dY=Q), dict(dX=Q, X=Q), dict(dX=Q, X=Q, dWdT=None), dict(dX=Q, dY=Q, dWgT=None, dWuT=None)):
        assert backward(lib, **kw) == ARG, kw
    need = lib.sig_workspace_bytes(11, 64, 128, 4)
    assert need == 3 * 4 * 128 * 2
    assert backward(lib, ws=None) == WORKSPACE and backward(lib, ws_bytes=need - 1) == WORKSPACE


def test_gated_mlp_backward_of_an_empty_block(lib):
    """No tokens: whatever gradient is wanted, no pointer is looked at.  The gradient in
    X of an empty tensor is a NULL pointer, so it cannot count as one that is missing."""
    none = dict(rows=0, dY=None, X=None, g=None, u=None, dWgT=None, dWuT=None, dWdT=None, ws=None, ws_bytes=0)
    assert backward(lib, dX=None, **none) == OK
    assert backward(lib, **none) == OK
    # one of the two projections' gradients alone stays an error, and so do bad sizes
    assert backward(lib, **{**none, "dWgT": P}) == NULL and backward(lib, **{**none, "dWuT": P}) == NULL
    assert backward(lib, **{**none, "d_model": 20}) == SHAPE and backward(lib, **{**none, "act": 5}) == ARG


def test_workspace_sizes(lib):
    ws = lib.sig_workspace_bytes
    assert ws(10, 64, 8, 3) == 256 and ws(11, 64, 8, 3) == 3 * 256      # whole 256-byte parts
    assert ws(10, 1 << 20, 1 << 20, 1 << 24) == 1 << 45                  # no 32-bit product
    for bad in ((0, 128, 4), (64, 12, 4), (64, 128, 0), (64, 128, -1), (64, 128, (1 << 24) + 1)):
        assert ws(10, *bad) == 0 and ws(11, *bad) == 0, bad


def test_binding_refuses_before_any_launch():
    import torch
    import sparse_input_gemv_threshold_b200 as sig
    X = torch.zeros(2, 64, dtype=torch.float16)
    W = torch.zeros(64, 64, dtype=torch.float16)
    with pytest.raises(ValueError, match="CUDA device"):
        sig.linear_act(X, W)
    with pytest.raises(TypeError, match="float16 or torch.bfloat16"):
        sig.linear_act(X.float(), W.float())
    with pytest.raises(ValueError, match="2-D"):
        sig.gated_mlp(X[0], W, W, W)
    with pytest.raises(ValueError, match="CUDA device"):
        sig.gated_mlp_backward(X, X, X, X, W, W, W)


def test_header_and_binding_agree_on_codes():
    import sparse_input_gemv_threshold_b200 as sig
    src = open(os.path.join(ROOT, "include", "sig.h")).read()
    for name, value in (("SIG_ACT_NONE", sig.ACT_NONE), ("SIG_ACT_RELU", sig.ACT_RELU),
                        ("SIG_ACT_GELU", sig.ACT_GELU), ("SIG_ACT_GELU_TANH", sig.ACT_GELU_TANH),
                        ("SIG_ACT_SILU", sig.ACT_SILU), ("SIG_OP_GATED_TOKENS", sig.OP_GATED_TOKENS),
                        ("SIG_OP_GATED_BACKWARD", sig.OP_GATED_BACKWARD)):
        assert f"{name} = {value}" in src, name
