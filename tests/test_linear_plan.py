"""What the feed-forward products launch, without a GPU: every plan keeps to what the kernels
take (tile widths, shared memory, TMEM, k-blocks for every CTA of a cluster)."""
import random

import pytest

from bf16_gemm_skinny_gb300 import _native as bsk
from bf16_gemm_skinny_gb300 import build as bsk_build


@pytest.fixture(scope="module", autouse=True)
def lib():
    bsk_build.build()
    yield bsk.load()
    for k in ("linear_kernel", "linear_tile", "split_k"):
        bsk.set_option(k, 0)


def blocks(v, unit):
    return -(-v // unit)


def check(p, M, K, n, gated, dx, dW):
    grad = dx or dW
    unit = (128 if p["pair"] else 64) if grad else 32 if p["pair"] or gated else 16
    assert p["tile"] % unit == 0 and unit <= p["tile"] <= 256, p
    assert p["split"] in (1, 2, 4, 8) and not (p["pair"] and p["split"] > 1), p
    if p["split"] > 1:
        parts = 2 if gated else 1
        k = max(blocks(M, 64) * parts if dx else 0, blocks(n, 64) if dW else 0) if grad else blocks(K, 64)
        assert k >= 2 * p["split"], p
        if dx and dW:   # the clusters of the longer k loops are on the device at once
            longer_w = blocks(n, 64) > blocks(M, 64) * parts
            tiles = (blocks(M, 128) * parts if longer_w else blocks(n, 128)) * blocks(K, p["tile"])
            assert tiles * p["split"] <= 152, p


@pytest.mark.parametrize("seed", range(8))
def test_plans_keep_to_the_kernels_limits(seed):
    rng = random.Random(seed)
    for _ in range(300):
        M, K, n = (int(2 ** rng.uniform(0, 15)) for _ in range(3))
        gated = rng.random() < 0.5
        dx, dW = rng.choice(((False, False), (True, False), (False, True), (True, True)))
        check(bsk.plan_linear(M, K, n, gated, dx, dW), M, K, n, gated, dx, dW)


@pytest.mark.parametrize("kernel,tile,split", [(1, 64, 0), (1, 256, 4), (2, 256, 0), (2, 128, 0), (1, 48, 2), (0, 96, 8)])
def test_options_choose_where_they_can(kernel, tile, split):
    for name, value in (("linear_kernel", kernel), ("linear_tile", tile), ("split_k", split)):
        bsk.set_option(name, value)
    try:
        for M, K, n in ((1000, 4096, 200), (64, 64, 1), (5000, 1024, 3000)):
            for gated in (False, True):
                p = bsk.plan_linear(M, K, n, gated)
                check(p, M, K, n, gated, False, False)
                assert kernel == 0 or p["pair"] == (kernel == 2)
                if tile % 32 == 0:
                    assert p["tile"] == tile
                if split > 1 and not p["pair"] and blocks(K, 64) >= 2 * split:
                    assert p["split"] == split
    finally:
        for name in ("linear_kernel", "linear_tile", "split_k"):
            bsk.set_option(name, 0)


def test_long_loops_of_few_tiles_are_split_and_large_products_take_pairs():
    assert bsk.plan_linear(5120, 17408, 1)["split"] > 1
    assert bsk.plan_linear(1024, 8192, 512)["split"] > 1
    assert bsk.plan_linear(17408, 5120, 4096, gated=True)["pair"] == 1
    assert bsk.plan_linear(17408, 5120, 4096, gated=True, dx=True, dW=True) == {"pair": 1, "tile": 256, "split": 1}
    assert bsk.plan_linear(10112, 64, 71, dx=True, dW=True)["split"] > 1


def test_bad_queries():
    for bad in (dict(M=0, K=1, n=1), dict(M=1, K=0, n=1), dict(M=1, K=1, n=0), dict(M=1, K=1, n=1, sms=1)):
        with pytest.raises(bsk.BskError):
            bsk.plan_linear(**bad)


A = 1 << 24   # stands for a device address; nothing is read from it


def gated(g, u, gu_stride, h=6 * A, h_stride=100):
    bsk.gated_linear_enqueue(0, A, 2 * A, 64, 3 * A, 64, None, None, h, h_stride, g, u, gu_stride, 100, 64, 7, bsk.ACT_SILU, 0)


@pytest.mark.parametrize("args,fits", [
    (dict(g=7 * A, u=7 * A + 200, gu_stride=200), True),        # two halves of the same rows
    (dict(g=7 * A + 200, u=7 * A, gu_stride=200), True),
    (dict(g=7 * A, u=7 * A + 200, gu_stride=199), False),       # u's last column is g's first of the next row
    (dict(g=7 * A, u=7 * A + 198, gu_stride=200), False),       # one column shared
    (dict(g=7 * A, u=7 * A + 600 + 200, gu_stride=300), True),  # other rows of the same buffer
    (dict(g=7 * A, u=7 * A + 600 + 402, gu_stride=300), False),
    (dict(g=7 * A, u=7 * A + 200, gu_stride=300, h=7 * A + 400, h_stride=300), True),
    (dict(g=7 * A, u=7 * A + 200, gu_stride=300, h=7 * A + 400, h_stride=301), False),   # not the same rows
])
def test_parts_of_the_same_rows(args, fits):
    import torch

    if fits and torch.cuda.is_available():
        pytest.skip("would launch on made-up addresses")
    with pytest.raises(bsk.BskError) as exc:
        gated(**args)
    assert (exc.value.status != 1) == fits, str(exc.value)   # what fits ends at the missing device


def test_gradients_of_another_size_beside_each_other():
    """FP32 weight gradients within rows that hold 16-bit values too: the same number of bytes apart."""
    import torch

    if torch.cuda.is_available():
        pytest.skip("would launch on made-up addresses")
    for dx, fits in ((8 * A + 256, True), (8 * A + 254, False)):   # dW: rows of 64 FP32 values, 512 bytes apart
        with pytest.raises(bsk.BskError) as exc:
            bsk.linear_act_backward_enqueue(0, A, 64, 2 * A, 64, None, 100, 4 * A, 100, dx, 256, 8 * A, 128, None, 0, 0, 100, 64, 7, 0, 0)
        assert (exc.value.status != 1) == fits, str(exc.value)
