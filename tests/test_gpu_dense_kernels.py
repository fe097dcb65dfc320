"""GPU parity of the dense products, kernel by kernel: the shapes of dense_shapes, at
which the plan gives every kernel and every form of its walk or join to every product
that can have it, and the uses whose tests at other shapes reach one kernel only.
Tolerances as in test_gpu_dense_tokens, whose checks these are.
"""
import numpy as np
import pytest

from tests import test_gpu_dense_tokens as tokens
from tests.dense_shapes import PRODUCTS, cases, form
from tests.test_gpu_dense_give_up import under_limit
from tests.test_gpu_dense_tokens import TYPES, backward_inputs, check_linear, normal

pytestmark = pytest.mark.gpu


def plan_form(sig, product, rows, d_in, d_out):
    return form(sig.dense_plan(getattr(sig, "PRODUCT_" + product), rows, d_in, d_out))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,K,N,f", cases("LINEAR"))
def test_linear(sig, dtype, rows, K, N, f):
    assert plan_form(sig, "LINEAR", rows, K, N) == f
    check_linear(sig, rows, K, N, dtype, "none", False, False, seed=rows)
    check_linear(sig, rows, K, N, dtype, "gelu", True, True, seed=rows + 1)
    check_linear(sig, rows, K, N, dtype, "silu", False, True, seed=rows + 2)
    check_linear(sig, rows, K, N, dtype, "relu", True, False, seed=rows + 3)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,m,ff,f", cases("GATED"))
def test_gated(sig, dtype, rows, m, ff, f):
    assert plan_form(sig, "GATED", rows, m, ff) == f
    tokens.test_gated_mlp(sig, dtype, rows, m, ff, "silu")
    tokens.test_gated_mlp(sig, dtype, rows, m, ff, "gelu")


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,m,ff,f", cases("HIDDEN_GRAD", "INPUT_GRAD", "WEIGHT_GRADS"))
def test_backward(sig, dtype, rows, m, ff, f):
    assert f in [plan_form(sig, p, rows, m, ff) for p in ("HIDDEN_GRAD", "INPUT_GRAD", "WEIGHT_GRADS")]
    tokens.test_gated_mlp_backward(sig, dtype, rows, m, ff, "silu")
    tokens.test_gated_mlp_backward(sig, dtype, rows, m, ff, "gelu_tanh")


@pytest.mark.parametrize("rows,m,ff", [(300, 136, 264), (407, 520, 1096), (371, 8216, 200)])
def test_weight_gradients_by_themselves(sig, rows, m, ff):
    """The library gives dWgT and dWuT without dWdT, and dWdT without them: the same bits
    as all three in one launch."""
    import torch
    dY, X, g, u, Wg, Wu, Wd = backward_inputs(rows, m, ff, "bf16", seed=210)
    want = sig.gated_mlp_backward(dY, X, g, u, Wg, Wu, Wd)[1:]
    n = sig.workspace_bytes(sig.OP_GATED_BACKWARD, m, ff, rows)
    for keep in ((True, True, False), (False, False, True)):
        got = [torch.full_like(w, 7.0) if k else None for w, k in zip(want, keep)]
        ws = torch.empty(n, dtype=torch.uint8, device="cuda")
        st = sig._lib.gated_mlp_backward(
            dY.data_ptr(), m, X.data_ptr(), m, rows, g.data_ptr(), u.data_ptr(), Wg.data_ptr(), Wu.data_ptr(),
            Wd.data_ptr(), m, ff, sig.ACT_SILU, None, m, *[None if t is None else t.data_ptr() for t in got], 1,
            ws.data_ptr(), n, torch.cuda.current_stream().cuda_stream)
        torch.cuda.synchronize()
        assert st == 0
        assert all(torch.equal(a, b) for a, b in zip(got, want) if a is not None)


# ---------------------------------------------------------------------------
# The pair kernel's epilogues that read (residual; g and u) and its strided stores
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("rows,K,N", PRODUCTS["LINEAR"]["pair, whole"][:1] + PRODUCTS["LINEAR"]["pair, both"][:2]
                         + PRODUCTS["LINEAR"]["tall, many items"][1:])
def test_strided_in_place_and_beside_nan(sig, rows, K, N):
    tokens.test_tall_tiles_strided_in_place_and_beside_nan(sig, rows, K, N)


def test_pair_kernel_with_few_columns(sig):
    """4300 tokens through narrow layers, where the tests of strides, gaps, places and
    special values use the pair kernel."""
    rows = 4300
    for product, d_in, d_out in (("LINEAR", 136, 264), ("LINEAR", 320, 520), ("LINEAR", 192, 512),
                                 ("LINEAR", 100, 264), ("HIDDEN_GRAD", 104, 136), ("INPUT_GRAD", 104, 136),
                                 ("HIDDEN_GRAD", 264, 520), ("INPUT_GRAD", 264, 520), ("GATED", 264, 520)):
        assert plan_form(sig, product, rows, d_in, d_out).startswith("pair"), (product, d_in, d_out)
    tokens.test_linear_row_strides_and_untouched_gaps(sig, rows)
    tokens.test_linear_adds_into_the_residual_in_place(sig, rows)
    tokens.test_special_values_stay_in_their_rows_and_columns(sig, rows)
    tokens.test_nothing_between_the_rows_is_read(sig, rows)
    tokens.test_outputs_in_the_place_of_inputs(sig, rows)


@pytest.mark.parametrize("rows,m,ff", [(4300, 264, 520), (843, 400, 9488)])
def test_pair_kernel_gives_the_same_bits_in_graphs_and_on_streams(sig, rows, m, ff):
    """Two captured steps replayed at once, beside eager calls on a third stream."""
    import torch
    assert plan_form(sig, "HIDDEN_GRAD", rows, m, ff).startswith("pair")
    blocks = [backward_inputs(rows, m, ff, "bf16", seed=220 + 10 * i) for i in range(3)]
    R = normal(250, rows, ff, dtype="bf16")

    def run(b):
        return [sig.linear_act(b[1], b[4], act=sig.ACT_GELU, residual=R), sig.gated_mlp(b[1], *b[4:], residual=b[1]),
                *sig.gated_mlp_backward(*b)]
    want = [run(b) for b in blocks]
    streams = [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    graphs, got = [], []
    for b, s in zip(blocks[:2], streams):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            got.append(run(b))
        graphs.append(g)
    for _ in range(3):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        with torch.cuda.stream(streams[2]):
            eager = run(blocks[2])
    torch.cuda.synchronize()
    for a, b in zip(want, got + [eager]):
        assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_kernels_that_take_all_tensor_memory_beside_the_others(sig):
    """A pair and a tall walk on one stream, the N:M GEMMs and a few-token product on
    another, and in turn on one."""
    import torch
    import oracle
    import workloads
    WT, Xn = workloads.nm_tokens(7, rows=512, d=512, d_out=512)
    dW, dXn = torch.from_numpy(WT).cuda(), torch.from_numpy(Xn).cuda()
    Y64, B = oracle.nm_gemm(Xn, WT, oracle.nm_mask(Xn, 2, 4))
    shapes = [(1281, 320, 5000), (1300, 1000, 8200), (40, 512, 1096)]
    assert [sig.dense_plan(sig.PRODUCT_LINEAR, *s).kernel for s in shapes] == ["pair", "tall", "few"]
    args = [(normal(260 + i, r, K), normal(270 + i, K, N, scale=K ** -0.5)) for i, (r, K, N) in enumerate(shapes)]
    want = [sig.linear_act(*a) for a in args]
    wantn = sig.nm_act_gemm(dXn, dW, 2, 4)
    assert np.all(np.abs(wantn.cpu().numpy().astype(np.float64) - Y64) <= 2e-3 * B + 2.0 ** -24)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(20):
        got = [sig.linear_act(*args[0], stream=s1), sig.linear_act(*args[1], stream=s1)]
        n2 = sig.nm_act_gemm(dXn, dW, 2, 4, stream=s2)
        got.append(sig.linear_act(*args[2], stream=s2))
        n1 = sig.nm_act_gemm(dXn, dW, 2, 4, stream=s1)
        more = [sig.linear_act(*args[1], stream=s2), sig.linear_act(*args[0], stream=s2)]
        last = sig.linear_act(*args[2], stream=s1)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want)) and torch.equal(last, want[2])
    assert torch.equal(more[0], want[1]) and torch.equal(more[1], want[0])
    assert torch.equal(n1, wantn) and torch.equal(n2, wantn)


# ---------------------------------------------------------------------------
# Give-ups, in the kernels that the uses without a plan's check no longer reach
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("rows,m,ff,kernels", [
    (1061, 952, 3232, {"HIDDEN_GRAD": "pair"}), (4300, 256, 1096, {"HIDDEN_GRAD": "pair", "GATED": "pair"}),
    (4210, 416, 40, {"HIDDEN_GRAD": "pair", "GATED": "pair"}), (9722, 792, 200, {"INPUT_GRAD": "pair"}),
    (1300, 1000, 5000, {"HIDDEN_GRAD": "tall", "GATED": "tall"})])
def test_a_give_up_in_every_epilogue_and_the_calls_after_it(sig, rows, m, ff, kernels):
    """Waits that give up while the epilogue's reads of g, u or the residual are under
    way: the launch ends with an error, what it had in flight lands, and the next calls
    are right."""
    import torch
    for product, kernel in kernels.items():
        assert sig.dense_plan(getattr(sig, "PRODUCT_" + product), rows, m, ff).kernel == kernel
    args = backward_inputs(rows, m, ff, "bf16", seed=280)
    R = normal(290, rows, ff, dtype="bf16")

    def run():
        return [sig.linear_act(args[1], args[4], act=sig.ACT_SILU, residual=R),
                sig.gated_mlp(args[1], *args[4:], residual=args[1]), *sig.gated_mlp_backward(*args)]
    want = run()
    assert sig.take_device_error() == 0
    for limit in (1, 64, 600, 1200, 2000, 3000, 5000, 8000):
        _, code = under_limit(sig, limit, run)
        assert limit > 64 or code != 0
        assert all(torch.equal(a, b) for a, b in zip(want, run())), limit
        assert sig.take_device_error() == 0


def test_a_wait_that_gives_up_is_reported_by_every_kernel(sig):
    import torch
    for (rows, K, N), kernel in (((600, 1024, 2048), "few"), ((1300, 1000, 8200), "tall"), ((1281, 320, 5000), "pair")):
        assert sig.dense_plan(sig.PRODUCT_LINEAR, rows, K, N).kernel == kernel
        X, W = normal(300, rows, K), normal(301, K, N, scale=K ** -0.5)
        want = sig.linear_act(X, W)
        _, code = under_limit(sig, 64, lambda: sig.linear_act(X, W))
        assert code == 1, kernel
        assert torch.equal(sig.linear_act(X, W), want) and sig.take_device_error() == 0


# ---------------------------------------------------------------------------
# The limits of the sizes
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("rows,K,N", [(1, 1 << 20, 8), (300, 1 << 20, 8), (3, 8, 1 << 20), (1300, 8, 1 << 20),
                                      (1 << 24, 8, 8), ((1 << 24) - 5, 72, 8)])
def test_largest_sizes(sig, rows, K, N):
    import torch
    X, W = normal(310, rows, K), normal(311, K, N, scale=K ** -0.5)
    b = normal(312, N)
    Y = sig.linear_act(X, W, bias=b, act=sig.ACT_RELU)
    at = torch.unique(torch.cat([torch.randint(0, rows, (300,), generator=torch.Generator().manual_seed(3)),
                                 torch.tensor([0, rows - 1])])).cuda()
    z, e = tokens.product(X[at], W)
    z = z + b.double()
    y, e = z.clamp(min=0.0), e + tokens.U * z.abs()
    tokens.within(Y[at], y, tokens.rounding(y, e, "fp16"), f"{rows}x{K}x{N}")


def test_largest_sizes_of_the_gated_block(sig):
    """2^24 tokens forward, and weight gradients that sum over 2^20 + 3 of them."""
    import torch
    rows = 1 << 24
    X, Wg, Wu, Wd = normal(320, rows, 8), normal(321, 8, 8), normal(322, 8, 8), normal(323, 8, 8)
    Y = sig.gated_mlp(X, Wg, Wu, Wd, residual=X)
    for at in (slice(0, 300), slice(rows - 300, rows), slice(1 << 23, (1 << 23) + 300)):
        assert torch.equal(Y[at], sig.gated_mlp(X[at].contiguous(), Wg, Wu, Wd, residual=X[at].contiguous()))
    rows = (1 << 20) + 3
    tokens.test_gated_mlp_backward(sig, "fp16", rows, 8, 16, "silu")


def test_largest_stride(sig):
    """Two rows 2^30 entries apart: X, the residual and Y, whose gap stays as it was."""
    import torch
    ld, K, N = 1 << 30, 72, 136
    buf = [torch.empty(ld + N, dtype=torch.float16, device="cuda") for _ in range(2)]
    X, R = (b.as_strided((2, c), (ld, 1)) for b, c in zip(buf, (K, N)))
    X.copy_(normal(330, 2, K))
    R.copy_(normal(331, 2, N))
    buf[1][N:ld] = 7.0
    W = normal(332, K, N, scale=0.1)
    want = sig.linear_act(X.contiguous(), W, residual=R.contiguous())
    sig.linear_act(X, W, residual=R, Y=R)
    assert torch.equal(R, want) and bool((buf[1][N:ld] == 7).all())
