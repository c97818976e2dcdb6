"""Gradients that are sums over very many tokens or features: the accuracy of their FP32 sums does not go with the length.

Operands of one sign, so that what an accumulation cuts off adds up.  Bounds: within a segment the forward pass's, two
errors of 2^-23 of the sum of magnitudes for every 16 terms; the segments' sums are added in FP32, at most 2^-23 of that sum
each; 32 more for what is around (sums of split k loops, the old gradient).  One rounding to the type: half a step.
"""
import pytest
import torch

import linear_reference as ref
from bf16_gemm_skinny_gb300 import _native as bsk
from bf16_gemm_skinny_gb300 import build as bsk_build
from test_gpu_linear import KIND, check

pytestmark = pytest.mark.gpu

SEGMENT_32, SEGMENT_16 = 12 * 64, 64 * 64   # terms in a segment: FP32 weight gradients, 16-bit results
KERNELS = [(0, 0), (1, 1), (1, 4), (2, 0)]   # the plan's choice, one CTA per tile, split over four, CTA pairs


@pytest.fixture(scope="module", autouse=True)
def lib():
    bsk_build.build()
    torch.cuda.init()
    yield bsk.load()


@pytest.fixture(autouse=True)
def options(request):
    kernel, split = request.getfixturevalue("kernel")
    bsk.set_option("linear_kernel", kernel)
    bsk.set_option("split_k", split)
    yield
    bsk.set_option("linear_kernel", 0)
    bsk.set_option("split_k", 0)


def positive(seed, *shape, t):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return ((torch.rand(*shape, generator=g, device="cuda") * 0.5 + 0.5) / 16).to(t)


def error(terms, segment):
    return (segment / 8 + terms / segment + 32) * 2.0 ** -23


@pytest.mark.parametrize("kernel", KERNELS, ids=str)
def test_weight_gradients_in_fp32(kernel):
    n, m, k, t = 33_000, 200, 136, torch.float16
    x, dy, w = positive(1, n, k, t=t), positive(2, n, m, t=t), positive(3, m, k, t=t)
    dw = torch.full((m, k), float("nan"), device="cuda")
    bsk.linear_act_backward(KIND["f16"], w, k, x, k, None, m, dy, m, None, k, dw, k, None, bsk.GRAD_F32, 0, m, k, n, bsk.ACT_NONE)
    want = dy.double().T @ x.double()
    check(dw, want, error(n, SEGMENT_32) * want, torch.float32, "dW")


@pytest.mark.parametrize("type_", ["bf16", "f16"])
@pytest.mark.parametrize("kernel", KERNELS, ids=str)
def test_weight_gradients_in_16_bits(kernel, type_):
    """Added to the rounded gradient's negative, which leaves the sum's error and what the rounding took."""
    n, m, k, t = 400_003, 200, 136, ref.TYPES[type_]
    x, dy, w = positive(1, n, k, t=t), positive(2, n, m, t=t), positive(3, m, k, t=t)
    want = dy.double().T @ x.double()
    dw = (-want).to(t)
    old = dw.double()
    bsk.linear_act_backward(KIND[type_], w, k, x, k, None, m, dy, m, None, k, dw, k, None, bsk.GRAD_16, 1, m, k, n, bsk.ACT_NONE)
    check(dw, want + old, error(n, SEGMENT_16) * want, t, "dW")


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("kernel", KERNELS, ids=str)
def test_input_gradients(kernel, gated):
    n, m, k, t = 70, 400_003, 72, torch.float16
    dy, w, x = positive(4, n, m, t=t), positive(5, m, k, t=t), positive(6, n, k, t=t)
    dx = torch.full((n, k), float("nan"), dtype=t, device="cuda")
    if gated:   # g = u = 1: dg and du are dh
        w2, one = positive(7, m, k, t=t), torch.ones(n, m, dtype=t, device="cuda")
        bsk.gated_linear_backward(KIND["f16"], w, w2, k, x, k, one, one, m, dy, m, dx, k, None, None, k, None, None, bsk.GRAD_F32, 0,
                                  m, k, n, bsk.ACT_NONE)
        want = dy.double() @ w.double() + dy.double() @ w2.double()
    else:
        bsk.linear_act_backward(KIND["f16"], w, k, x, k, None, m, dy, m, dx, k, None, k, None, bsk.GRAD_F32, 0, m, k, n, bsk.ACT_NONE)
        want = dy.double() @ w.double()
    check(dx, want, error(m * (2 if gated else 1), SEGMENT_16) * want, t, "dx")
