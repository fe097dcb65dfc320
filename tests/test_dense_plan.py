"""The plan of the dense products, on the CPU: every kernel and every form of its walk
or join has a shape among those that the GPU tests run, so that a change of the plan's
estimates cannot leave one of them without a test."""
import ctypes
import random

import pytest

from tests.conftest import load_builder
from tests.dense_shapes import LINEAR_FORMS, PRODUCTS, cases, form

load_builder().build()   # the import below loads the library
import sparse_input_gemv_threshold_b200 as sig  # noqa: E402

OK, NULL, SHAPE, ALIGN, WORKSPACE, CUDA, TIMEOUT, ARG = range(8)


@pytest.mark.parametrize("product", PRODUCTS)
def test_every_shape_has_the_form_that_it_is_listed_for(product):
    for rows, d_in, d_out, f in cases(product):
        plan = sig.dense_plan(getattr(sig, "PRODUCT_" + product), rows, d_in, d_out)
        assert form(plan) == f, (rows, d_in, d_out, plan)


@pytest.mark.parametrize("product", PRODUCTS)
def test_every_form_that_a_product_takes_has_a_shape(product):
    """A sweep of sizes meets the listed forms and no other."""
    rng = random.Random(1)
    met = set()
    for _ in range(40000):
        rows = int(2 ** rng.uniform(0, 13.5))
        d_in, d_out = (8 * int(2 ** rng.uniform(0, 10.5)) for _ in range(2))
        met.add(form(sig.dense_plan(getattr(sig, "PRODUCT_" + product), rows, d_in, d_out)))
    assert met == set(PRODUCTS[product])
    if product != "WEIGHT_GRADS":
        assert set(PRODUCTS[product]) == set(LINEAR_FORMS)


def test_the_parts_of_the_weight_gradients_are_the_pair_kernels():
    for rows, d_in, d_out, _ in cases("WEIGHT_GRADS"):
        both = [sig.dense_plan(p, rows, d_in, d_out) for p in (sig.PRODUCT_UP_GRADS, sig.PRODUCT_DOWN_GRAD)]
        tiles = -(-d_in // 256) * -(-d_out // 256)
        assert [p.kernel for p in both] == ["pair"] * 2
        assert [p.tiles + p.halves / 2 for p in both] == [2 * tiles, tiles]


def test_refusals():
    f = sig._lib.sig_dense_plan
    out = (ctypes.c_int * 6)()
    assert f(0, 1, 1, 8, out) == OK and f(0, 1, 1, 8, None) == NULL
    for product in (-1, 7):
        assert f(product, 1, 64, 64, out) == ARG
    for bad in ((0, 64, 64), ((1 << 24) + 1, 64, 64), (1, 64, 12), (1, 64, (1 << 20) + 8), (1, 0, 64)):
        for product in range(7):
            assert f(product, *bad, out) == SHAPE, (product, bad)
    assert f(0, 1, 63, 8, out) == OK and f(1, 1, 63, 8, out) == SHAPE    # only K of a linear product is free
    with pytest.raises(sig.SigError):
        sig.dense_plan(sig.PRODUCT_GATED, 4, 12, 64)


def test_the_largest_sizes_stay_in_range():
    """Tile counts fit 32 bits at the limits of the sizes."""
    for product in range(7):
        plan = sig.dense_plan(product, 1 << 24, 1 << 20, 1 << 20)
        assert min(plan.tokens, plan.parts, plan.per_sm) > 0 and plan.tiles >= 0 and plan.halves >= 0
        assert plan.tiles + plan.halves > 0
