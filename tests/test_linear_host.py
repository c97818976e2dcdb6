"""Refusals of the feed-forward layer calls: every bad argument is turned down with
BSK_ERR_INVALID_ARG before a device is touched (no GPU needed)."""
import pytest

from bf16_gemm_skinny_gb300 import _native as bsk
from bf16_gemm_skinny_gb300 import build as bsk_build

A = 1 << 24   # stands for a device address; nothing is read from it


@pytest.fixture(scope="module", autouse=True)
def lib():
    bsk_build.build()
    return bsk.load()


LINEAR = dict(type=0, W=A, w_stride=64, x=2 * A, x_stride=64, bias=3 * A, residual=4 * A, residual_stride=100, y=5 * A,
              y_stride=100, z=6 * A, z_stride=100, M=100, K=64, n=7, activation=4)
GATED = dict(type=1, Wg=A, Wu=2 * A, w_stride=64, x=3 * A, x_stride=64, bias_g=4 * A, bias_u=5 * A, h=6 * A, h_stride=100,
             g=7 * A, u=8 * A, gu_stride=100, M=100, K=64, n=7, activation=3)
LINEAR_B = dict(type=0, W=A, w_stride=64, x=2 * A, x_stride=64, z=3 * A, z_stride=100, dy=4 * A, dy_stride=100, dx=5 * A,
                dx_stride=64, dW=6 * A, dw_stride=64, dbias=7 * A, grad_type=0, accumulate=0, M=100, K=64, n=7, activation=4)
GATED_B = dict(type=0, Wg=A, Wu=2 * A, w_stride=64, x=3 * A, x_stride=64, g=4 * A, u=5 * A, gu_stride=100, dh=6 * A,
               dh_stride=100, dx=7 * A, dx_stride=64, dWg=8 * A, dWu=9 * A, dw_stride=64, dbias_g=10 * A, dbias_u=11 * A,
               grad_type=0, accumulate=0, M=100, K=64, n=7, activation=4)
BASES = {"linear_act": LINEAR, "gated_linear": GATED, "linear_act_backward": LINEAR_B, "gated_linear_backward": GATED_B}

COMMON = [dict(type=2), dict(type=-1), dict(activation=5), dict(activation=-1), dict(M=-1), dict(K=-1), dict(n=-1),
          dict(x=None), dict(x_stride=63), dict(w_stride=63), dict(x_stride=-64), dict(M=2 ** 31 - 1), dict(x=2 * A + 1)]
CASES = {
    "linear_act": COMMON + [dict(W=None), dict(y=None), dict(y_stride=99), dict(z_stride=99), dict(residual_stride=99),
                            dict(y=2 * A), dict(y=A + 2), dict(z=5 * A + 2), dict(residual=5 * A + 2), dict(z=4 * A),
                            dict(residual=5 * A, residual_stride=101), dict(bias=3 * A + 1), dict(y=3 * A + 198),
                            dict(z=2 * A)],
    "gated_linear": COMMON + [dict(Wg=None), dict(Wu=None), dict(h=None), dict(h_stride=99), dict(gu_stride=99), dict(g=None),
                              dict(u=None), dict(h=3 * A), dict(u=7 * A), dict(g=6 * A + 4), dict(h=2 * A + 64 * 100 * 2 - 2),
                              dict(bias_u=5 * A + 1)],
    "linear_act_backward": COMMON + [dict(W=None), dict(dy=None), dict(z=None), dict(grad_type=2), dict(accumulate=2),
                                     dict(accumulate=-1), dict(dx=2 * A), dict(dW=A), dict(dx=4 * A), dict(dW=5 * A),
                                     dict(dbias=6 * A), dict(dw_stride=63), dict(dx_stride=63), dict(dW=6 * A + 2),
                                     dict(dbias=7 * A + 2), dict(dy_stride=99), dict(z_stride=99)],
    "gated_linear_backward": COMMON + [dict(Wg=None), dict(Wu=None), dict(g=None), dict(u=None), dict(dh=None), dict(dWg=None),
                                       dict(dWu=None), dict(dWu=8 * A), dict(dx=6 * A), dict(dbias_u=10 * A), dict(grad_type=-1),
                                       dict(dx=4 * A), dict(dh_stride=99), dict(gu_stride=99)],
}


@pytest.mark.parametrize("name,change", [(n, c) for n in CASES for c in CASES[n]], ids=lambda v: str(v).replace(" ", ""))
@pytest.mark.parametrize("form", ["", "_enqueue"])
def test_refused(name, change, form):
    with pytest.raises(bsk.BskError) as exc:
        getattr(bsk, name + form)(**{**BASES[name], **change}, stream=0)
    assert exc.value.status == 1, str(exc.value)
    assert bsk.last_error()


@pytest.mark.parametrize("name", BASES)
def test_what_is_accepted_reaches_the_device(name):
    """The unchanged arguments pass every check: without a device the call ends at it."""
    import torch

    if torch.cuda.is_available():
        pytest.skip("would launch on made-up addresses")
    for change in ({}, dict(type=1), dict(activation=0), dict(x_stride=65)):
        with pytest.raises(bsk.BskError) as exc:
            getattr(bsk, name)(**{**BASES[name], **change}, stream=0)
        assert exc.value.status != 1, str(exc.value)


def test_the_residual_may_be_the_output():
    import torch

    if torch.cuda.is_available():
        pytest.skip("would launch on made-up addresses")
    with pytest.raises(bsk.BskError) as exc:
        bsk.linear_act(**{**LINEAR, "residual": 5 * A}, stream=0)
    assert exc.value.status != 1, str(exc.value)


@pytest.mark.parametrize("change", [
    dict(x=5 * A, x_stride=100),                                  # y += act(y W^T): tiles would store over rows still read
    dict(x=5 * A, x_stride=100, K=100, w_stride=100),             # the same of a square layer
    dict(W=5 * A, w_stride=100), dict(W=5 * A, w_stride=100, n=100),
    dict(bias=5 * A), dict(bias=5 * A, M=99, residual_stride=100),   # a vector of M, its "stride" M + 1 that of y's rows
    dict(x=5 * A, x_stride=100, n=1), dict(z=5 * A), dict(x=5 * A, x_stride=100, residual_stride=101)], ids=str)
@pytest.mark.parametrize("form", ["", "_enqueue"])
def test_no_other_operand_may_be_the_output_beside_the_residual(change, form):
    with pytest.raises(bsk.BskError) as exc:
        getattr(bsk, "linear_act" + form)(**{**LINEAR, "residual": 5 * A, **change}, stream=0)
    assert exc.value.status == 1 and "overlaps" in str(exc.value), str(exc.value)


def test_nothing_to_do_is_no_error():
    for change in (dict(M=0), dict(n=0)):
        bsk.linear_act(**{**LINEAR, "W": None, "x": None, "y": None, **change}, stream=0)
        bsk.gated_linear(**{**GATED, "Wg": None, "x": None, "h": None, "g": None, **change}, stream=0)
    none = dict(dx=None, dbias=None, dW=None)
    bsk.linear_act_backward(**{**LINEAR_B, **none}, stream=0)
    bsk.gated_linear_backward(**{**GATED_B, "dx": None, "dWg": None, "dWu": None, "dbias_g": None, "dbias_u": None}, stream=0)
    bsk.linear_act_backward(**{**LINEAR_B, "n": 0, "M": 0}, stream=0)


@pytest.mark.parametrize("name", BASES)
def test_python_side(name):
    with pytest.raises(OverflowError):
        getattr(bsk, name)(**{**BASES[name], "M": 2 ** 31}, stream=0)
    with pytest.raises(TypeError):
        getattr(bsk, name)(**{**BASES[name], "K": 1.5}, stream=0)
    with pytest.raises((TypeError, AttributeError)):
        getattr(bsk, name)(**{**BASES[name], "x": "here"}, stream=0)
