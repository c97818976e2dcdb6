"""linear_act and gated_linear against the formulas in 64 bits.

Bounds.  Products of two 16-bit values are exact in FP32.  A tensor-core instruction
adds 16 of them to an accumulator and may cut every term at 2^-23 of the largest
magnitude met, at most S = sum |x||w| + |b|: two such errors a group of 16, so K/8
of them, and 32 more for the additions around it (partial sums of split k loops, bias,
residual).  The activation passes the sum's error on times its slope (at most 1.13)
and adds 2^-15 of its value at most (e^v by the hardware's 2^x: 2 + 1.2|v| units in the
last place, |v| <= 88 where it counts).  One rounding to the type: half a step.
"""
import pytest
import torch

import linear_reference as ref
from bf16_gemm_skinny_gb300 import _native as bsk
from bf16_gemm_skinny_gb300 import build as bsk_build

pytestmark = pytest.mark.gpu

ACT = {"none": bsk.ACT_NONE, "relu": bsk.ACT_RELU, "gelu": bsk.ACT_GELU, "gelu_tanh": bsk.ACT_GELU_TANH, "silu": bsk.ACT_SILU}
KIND = {"bf16": bsk.TYPE_BF16, "f16": bsk.TYPE_F16}


@pytest.fixture(scope="module", autouse=True)
def lib():
    bsk_build.build()
    torch.cuda.init()
    yield bsk.load()
    for k in bsk.OPTIONS:
        bsk.set_option(k, 0)


@pytest.fixture(autouse=True)
def defaults():
    yield
    for k in ("linear_kernel", "linear_tile", "split_k", "pdl", "num_sms"):
        bsk.set_option(k, 0)


class Rows:
    """A matrix in wider rows, `first` elements into its buffer, with a pattern around it that must stay."""

    FILL = 0x7FFF   # a NaN in both 16-bit types

    def __init__(self, n, width, pad, first, dtype, values=None):
        self.n, self.width, self.stride = n, width, width + pad
        size = {2: torch.int16, 4: torch.int32}[torch.empty(0, dtype=dtype).element_size()]
        self.raw = torch.full((first + n * self.stride + 64,), self.FILL, dtype=size, device="cuda")
        self.all = self.raw[first:first + n * self.stride].view(n, self.stride)
        self.t = self.all[:, :width].view(dtype)
        self.first = first
        if values is None:
            self.t.fill_(float("nan"))
        else:
            self.t.copy_(values)

    def intact(self):
        end = self.first + self.n * self.stride
        return bool((self.raw[:self.first] == self.FILL).all() and (self.raw[end:] == self.FILL).all() and
                    (self.all[:, self.width:] == self.FILL).all())


def draw(seed, *shape, size=1.0, t=torch.bfloat16):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(*shape, generator=g, device="cuda") * size).to(t)


def accumulate(K):
    return (K / 8 + 32) * 2.0 ** -23


def check(got, want, err, t, what):
    bound = err + ref.half_step(t) * (want.abs() + err) + ref.tiny(t)
    off = (got.double() - want).abs() - bound
    assert not torch.isnan(off).any(), f"{what}: not a number"
    assert float(off.max()) <= 0, f"{what}: off by {float((got.double() - want).abs().max()):.3g}, over its bound by {float(off.max()):.3g}"


def forward(gated, n, M, K, type_="bf16", act="silu", bias=True, residual=False, keep=False, pads=(0, 0, 0, 0), first=0,
            seed=0, inplace=False, enqueue=False, scale=1.0):
    t = ref.TYPES[type_]
    parts = 2 if gated else 1
    x = Rows(n, K, pads[0], first, t, draw(seed, n, K, size=scale, t=t))
    ws = [Rows(M, K, pads[1], first, t, draw(seed + 1 + i, M, K, size=max(K, 1) ** -0.5, t=t)) for i in range(parts)]
    bs = [draw(seed + 5 + i, M, size=0.5, t=t) if bias else None for i in range(parts)]
    out = Rows(n, M, pads[2], first, t)
    kept = [Rows(n, M, pads[3], first, t) if keep else None for _ in range(parts)]
    r = None
    if residual:
        r = out if inplace else Rows(n, M, pads[3], first, t)
        r.t.copy_(draw(seed + 9, n, M, size=2.0, t=t))
    rd = r.t.double() if residual else None
    raw = [m.raw.clone() for m in (x, *ws)]
    kt = [k.t if keep else None for k in kept]
    suffix = "_enqueue" if enqueue else ""
    kept_stride = kept[0].stride if keep else M
    if gated:
        getattr(bsk, "gated_linear" + suffix)(KIND[type_], ws[0].t, ws[1].t, ws[0].stride, x.t, x.stride, bs[0], bs[1], out.t,
                                              out.stride, kt[0], kt[1], kept_stride, M, K, n, ACT[act])
    else:
        getattr(bsk, "linear_act" + suffix)(KIND[type_], ws[0].t, ws[0].stride, x.t, x.stride, bs[0], r.t if r else None,
                                            r.stride if r else 0, out.t, out.stride, kt[0], kept_stride, M, K, n, ACT[act])
    if enqueue:
        bsk.stream_check()
    for m, before in zip((x, *ws), raw):
        assert torch.equal(m.raw, before), "an input was written"
    for m in (out, *(k for k in kept if k)):
        assert m.intact(), "written outside the output's rows"
    xd, wd = x.t.double(), [w.t.double() for w in ws]
    bd = [None if b is None else b.double() for b in bs]
    sums = [xd.abs() @ w.abs().T + (0 if b is None else b.abs()) for w, b in zip(wd, bd)]
    errs = [accumulate(K) * s for s in sums]
    if gated:
        want, *z = ref.gated(act, xd, wd[0], wd[1], bd[0], bd[1])
        a = ref.act(act, z[0])[0]
        ea = ref.SLOPE * errs[0] + 2.0 ** -15 * a.abs()
        err = a.abs() * errs[1] + z[1].abs() * ea + ea * errs[1] + 2.0 ** -23 * want.abs()
    else:
        want, z0 = ref.linear(act, xd, wd[0], bd[0], rd)
        z = [z0]
        err = ref.SLOPE * errs[0] + 2.0 ** -15 * ref.act(act, z0)[0].abs() + (2.0 ** -23 * (want.abs() + rd.abs()) if residual else 0)
    check(out.t, want, err, t, f"out {n}x{M}x{K}")
    for k, zi, e in zip(kept, z, errs):
        if k:
            check(k.t, zi, e, t, f"kept {n}x{M}x{K}")
    return out.t.clone()


SIZES = [(1, 1, 1), (1, 8, 8), (1, 1000, 512), (2, 17, 33), (3, 130, 1000), (4, 64, 64), (5, 333, 129), (8, 100, 136), (16, 512, 256),
         (31, 129, 65), (33, 257, 300), (64, 96, 1024), (100, 60, 72), (127, 255, 200), (128, 128, 128), (129, 127, 64),
         (200, 1000, 1024), (257, 511, 100), (300, 517, 203), (512, 768, 640), (777, 1031, 515), (1000, 777, 1030)]


@pytest.mark.parametrize("n,M,K", SIZES)
@pytest.mark.parametrize("gated", [False, True])
def test_sizes(n, M, K, gated):
    forward(gated, n, M, K, residual=not gated, keep=True)
    forward(gated, n, M, K, "f16", "gelu_tanh", bias=False)


@pytest.mark.parametrize("act", ref.ACTS)
@pytest.mark.parametrize("type_", ["bf16", "f16"])
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("n", [2, 70, 300])
def test_activations(gated, type_, act, n):
    forward(gated, n, 200, 320, type_, act, keep=True, residual=not gated, scale=3.0)


@pytest.mark.parametrize("pads,first", [((8, 8, 8, 8), 0), ((3, 0, 0, 0), 0), ((0, 5, 0, 0), 0), ((0, 0, 1, 0), 0), ((0, 0, 0, 7), 0),
                                        ((1, 2, 3, 4), 0), ((0, 0, 0, 0), 1), ((8, 8, 8, 8), 3), ((64, 0, 128, 8), 8)])
@pytest.mark.parametrize("n", [1, 3, 9, 150])
@pytest.mark.parametrize("gated", [False, True])
def test_strides_and_alignment(pads, first, n, gated):
    forward(gated, n, 136, 264, pads=pads, first=first, residual=not gated, keep=True)


@pytest.mark.parametrize("kernel", [1, 2])
@pytest.mark.parametrize("tile", [16, 32, 48, 64, 96, 128, 160, 192, 224, 256])
@pytest.mark.parametrize("gated", [False, True])
def test_every_tile(kernel, tile, gated):
    bsk.set_option("linear_kernel", kernel)
    bsk.set_option("linear_tile", tile)
    for n, M, K in ((7, 300, 200), (130, 513, 136), (600, 700, 300)):
        forward(gated, n, M, K, residual=not gated, keep=True)


@pytest.mark.parametrize("split", [2, 4, 8])
@pytest.mark.parametrize("tile", [32, 64, 128, 256])
@pytest.mark.parametrize("gated", [False, True])
def test_split_k(split, tile, gated):
    bsk.set_option("linear_kernel", 1)
    bsk.set_option("split_k", split)
    bsk.set_option("linear_tile", tile)
    for n, M, K in ((1, 77, 1100), (8, 300, 1024), (130, 203, 2000), (40, 64, 1030)):
        forward(gated, n, M, K, residual=not gated, keep=True)


@pytest.mark.parametrize("kernel", [1, 2])
@pytest.mark.parametrize("sms", [2, 5])
def test_many_tiles_per_unit(kernel, sms):
    bsk.set_option("linear_kernel", kernel)
    bsk.set_option("num_sms", sms)
    forward(True, 700, 900, 200)
    forward(False, 700, 900, 200, residual=True)


@pytest.mark.parametrize("n", [1, 5, 200])
def test_residual_in_place(n):
    for type_ in ("bf16", "f16"):
        a = forward(False, n, 520, 136, type_, "gelu", residual=True, inplace=True)
        b = forward(False, n, 520, 136, type_, "gelu", residual=True)
        assert torch.equal(a, b)


@pytest.mark.parametrize("gated", [False, True])
def test_no_inputs_is_an_empty_sum(gated):
    """K = 0: the bias through the activation."""
    for bias in (True, False):
        forward(gated, 9, 130, 0, bias=bias, residual=not gated, keep=True)


def test_repeated_calls_give_equal_bits():
    for shape in ((3, 500, 512), (40, 500, 2048), (700, 900, 300)):
        a = forward(True, *shape)
        b = forward(True, *shape, enqueue=True)
        assert torch.equal(a, b)


def test_large_values_and_tails():
    """Activations far out: nothing turns into NaN, tails keep their relative accuracy."""
    z = torch.tensor([-3e38, -1e30, -200.0, -88.0, -30.0, -9.0, -5.0, -1.0, -0.0, 0.0, 1.0, 9.0, 88.0, 1e30, 3e38], device="cuda")
    for type_, t in ref.TYPES.items():
        v = z.clamp(-6e4, 6e4).to(t) if type_ == "f16" else z.to(t)
        v = torch.cat([v, v.new_zeros(1)])
        n = v.numel()
        x = torch.eye(n, 16, device="cuda", dtype=t)
        w = torch.zeros(8, 16, device="cuda", dtype=t)
        w[:, :] = v[:16]
        for name in ref.ACTS:
            y = torch.empty(n, 8, dtype=t, device="cuda")
            bsk.linear_act(KIND[type_], w, 16, x, 16, None, None, 0, y, 8, None, 8, 8, 16, n, ACT[name])
            want = ref.act(name, v.double())[0]
            got = y[:, 3].double()
            assert torch.isfinite(got).all(), (type_, name)
            # the tails of e^-v: the bound at the top, and nothing below the type's smallest numbers
            err = 2.0 ** -12 * want.abs() + ref.half_step(t) * want.abs() + max(ref.tiny(t), 2.0 ** -125)
            assert ((got - want).abs() <= err).all(), (type_, name, got, want)


def test_not_a_number_stays_in_its_row():
    t = torch.bfloat16
    for n in (2, 40, 300):
        x, w = draw(1, n, 128), draw(2, 64, 128)
        x[1, 5] = float("nan")
        for name in ref.ACTS:
            y = torch.empty(n, 64, dtype=t, device="cuda")
            bsk.linear_act(0, w, 128, x, 128, None, None, 0, y, 64, None, 64, 64, 128, n, ACT[name])
            assert torch.isnan(y[1]).all() and not torch.isnan(y[0]).any() and not torch.isnan(y[2:]).any(), (n, name)


@pytest.mark.slow
def test_outputs_past_32_bits():
    """More than 2^31 output values: rows far out come out right."""
    n, M, K = 33000, 66000, 64
    x, w = draw(3, n, K), draw(4, M, K, size=K ** -0.5)
    y = torch.empty(n, M, dtype=torch.bfloat16, device="cuda")
    bsk.linear_act(0, w, K, x, K, None, None, 0, y, M, None, M, M, K, n, bsk.ACT_SILU)
    for r in (0, 17000, 32990, n - 1):
        want, z = ref.linear("silu", x[r:r + 1].double(), w.double())
        err = ref.SLOPE * accumulate(K) * (x[r:r + 1].double().abs() @ w.double().abs().T) + 2.0 ** -15 * want.abs()
        check(y[r:r + 1], want, err, torch.bfloat16, f"row {r}")
