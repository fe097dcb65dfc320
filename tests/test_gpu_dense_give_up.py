"""What the dense products leave behind when a pipeline wait gives up: every output
is either the right one or as it was, never a sum with a missing part, and the
give-up is reported.  No GPU fault is involved: the wait limit is shortened
(sig_set_wait_limit) and restored."""
import pytest

from tests.test_gpu_dense_tokens import normal

pytestmark = pytest.mark.gpu

MARK = 7.0   # what the output holds before a call


def under_limit(sig, limit, run):
    """The output of run() and the device error word with the waits' limit at `limit` cycles."""
    import torch
    try:
        sig.set_wait_limit(limit)
        Y = run()
        torch.cuda.synchronize()
        return Y, sig.take_device_error()
    finally:
        sig.set_wait_limit(0)


# the few-token kernel with a join of several parts beside the ring and in its place,
# the tall kernel and the pair kernel, each with a residual that its epilogue reads.
# The limits go from before the first load's arrival to past the whole product, so that
# the CTAs of a cluster come to different verdicts in some of the calls.
@pytest.mark.parametrize("rows,K,N", [
    (5, 4096, 1000), (16, 11008, 4096), (48, 4096, 1000), (200, 4096, 520), (333, 4096, 1000),
    (1300, 1000, 8200), (1281, 320, 5000)])
def test_no_sum_with_a_missing_part_is_stored(sig, rows, K, N):
    import torch
    X, W, R = normal(1, rows, K), normal(2, K, N, scale=K ** -0.5), normal(3, rows, N)
    want = sig.linear_act(X, W, act=sig.ACT_SILU, residual=R)
    gave_up = 0
    for limit in [1, 64, 300, 600, 900] + list(range(1000, 6000, 250)) + [8000, 12000, 20000, 40000]:
        for _ in range(3):
            Y, code = under_limit(sig, limit, lambda: sig.linear_act(
                X, W, act=sig.ACT_SILU, residual=R, Y=torch.full_like(R, MARK)))
            right, before = Y == want, Y == MARK
            assert bool((right | before).all()), (limit, code, int((~(right | before)).sum()))
            assert code != 0 or bool(right.all()), limit
            gave_up += code != 0
    assert gave_up > 0
    assert torch.equal(sig.linear_act(X, W, act=sig.ACT_SILU, residual=R), want)


def test_a_sum_of_many_stages_outlasts_a_stages_limit(sig):
    """256 stages a CTA take some 40 us and no wait for one of them lasts 16 us: the
    few-token kernel's wait for its sums has the default limit at least, and a limit
    above the default holds for it too."""
    import torch
    K = 131072
    X, W = normal(4, 3, K), normal(5, K, 8, scale=K ** -0.5)
    want = sig.linear_act(X, W)
    for limit in (30000, 20_000_000, 1 << 33):
        Y, code = under_limit(sig, limit, lambda: sig.linear_act(X, W))
        assert code == 0 and torch.equal(Y, want), limit


@pytest.mark.parametrize("rows,K,N", [(1300, 1000, 8200), (1281, 320, 5000)])
def test_a_pair_that_gives_up_waits_for_no_copy_that_was_not_issued(sig, rows, K, N):
    """When one CTA of a pair stops a stage before the other, the stage's barrier never
    completes; a wait for it would last for the default limit, 2 s."""
    import time
    X, W, R = normal(6, rows, K), normal(7, K, N, scale=K ** -0.5), normal(8, rows, N)
    want = sig.linear_act(X, W, residual=R)
    for limit in (600, 1500, 3000, 5000):
        t0 = time.perf_counter()
        _, code = under_limit(sig, limit, lambda: sig.linear_act(X, W, residual=R))
        assert code != 0 and time.perf_counter() - t0 < 0.5, limit
    assert bool((sig.linear_act(X, W, residual=R) == want).all())
