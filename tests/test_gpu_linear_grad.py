"""linear_act_backward and gated_linear_backward against the formulas in 64 bits and against differences.

Bounds.  dz is computed in FP32 (2^-14 of |dy| (|u|) for the derivative, whose terms may cancel), rounded to the
type (half a step) and multiplied: its error goes through the products with the other factor's magnitudes.  The products'
sums: as in the forward pass, two errors of 2^-23 of the sum of magnitudes for every 16 terms.
"""
import math

import pytest
import torch

import linear_reference as ref
from bf16_gemm_skinny_gb300 import _native as bsk
from bf16_gemm_skinny_gb300 import build as bsk_build
from test_gpu_linear import ACT, KIND, Rows, accumulate, check, draw

pytestmark = pytest.mark.gpu


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


def backward(gated, n, M, K, type_="bf16", act="silu", f32=True, accumulate_into=False, pads=(0, 0, 0, 0, 0, 0), first=0, seed=0,
             want=("dx", "dw", "db"), enqueue=False):
    t = ref.TYPES[type_]
    gt = torch.float32 if f32 else t
    parts = 2 if gated else 1
    x = Rows(n, K, pads[0], first, t, draw(seed, n, K, t=t))
    ws = [Rows(M, K, pads[1], first, t, draw(seed + 1 + i, M, K, size=K ** -0.5, t=t)) for i in range(parts)]
    zs = [Rows(n, M, pads[2], first, t, draw(seed + 3 + i, n, M, size=1.5, t=t)) for i in range(parts)]
    dy = Rows(n, M, pads[3], first, t, draw(seed + 6, n, M, size=0.3, t=t))
    dx = Rows(n, K, pads[4], first, t)
    dw = [Rows(M, K, pads[5], first, gt) for _ in range(parts)]
    db = [Rows(1, M, 0, first, gt) for _ in range(parts)]
    old = []
    for i, m in enumerate((*dw, *db)):
        if accumulate_into:
            m.t.copy_(draw(seed + 20 + i, m.n, m.width, size=3.0, t=gt))
        old.append(m.t.double() if accumulate_into else torch.zeros(m.n, m.width, dtype=torch.float64, device="cuda"))
    before = [m.raw.clone() for m in (x, *ws, *zs, dy)]
    skip = not gated and act == "none"
    g = (bsk.GRAD_F32 if f32 else bsk.GRAD_16, int(accumulate_into), M, K, n, ACT[act])
    dxt = dx.t if "dx" in want else None
    dwt = [m.t if "dw" in want else None for m in dw]
    dbt = [m.t if "db" in want else None for m in db]
    suffix = "_enqueue" if enqueue else ""
    if gated:
        getattr(bsk, "gated_linear_backward" + suffix)(
            KIND[type_], ws[0].t, ws[1].t, ws[0].stride, x.t, x.stride, zs[0].t, zs[1].t, zs[0].stride, dy.t, dy.stride, dxt,
            dx.stride, dwt[0], dwt[1], dw[0].stride, dbt[0], dbt[1], *g)
    else:
        getattr(bsk, "linear_act_backward" + suffix)(
            KIND[type_], ws[0].t, ws[0].stride, x.t, x.stride, None if skip else zs[0].t, zs[0].stride, dy.t, dy.stride, dxt,
            dx.stride, dwt[0], dw[0].stride, dbt[0], *g)
    if enqueue:
        bsk.stream_check()
    for m, b in zip((x, *ws, *zs, dy), before):
        assert torch.equal(m.raw, b), "an input was written"
    for m in (dx, *dw, *db):
        assert m.intact(), "written outside an output's rows"
    xd, wd, zd, dyd = x.t.double(), [w.t.double() for w in ws], [z.t.double() for z in zs], dy.t.double()
    if gated:
        rdx, rdw0, rdw1, rdb0, rdb1, dg, du = ref.gated_backward(act, xd, wd[0], wd[1], zd[0], zd[1], dyd)
        dz, rdw, rdb = [dg, du], [rdw0, rdw1], [rdb0, rdb1]
        raw = [2.0 ** -14 * (dyd * zd[1]).abs(), 2.0 ** -14 * du.abs()]
    else:
        rdx, rdw0, rdb0, d = ref.linear_backward(act, xd, wd[0], zd[0], dyd)
        dz, rdw, rdb = [d], [rdw0], [rdb0]
        raw = [torch.zeros_like(d) if skip else 2.0 ** -14 * dyd.abs()]
    edz = [r if skip else r + ref.half_step(t) * (d.abs() + r) + ref.tiny(t) for r, d in zip(raw, dz)]
    if "dx" in want:
        err = sum(e @ w.abs() for e, w in zip(edz, wd)) + accumulate(M * parts) * sum((d.abs() + e) @ w.abs() for d, e, w in zip(dz, edz, wd))
        check(dx.t, rdx, err, t, "dx")
    for i in range(parts):
        if "dw" in want:
            err = edz[i].T @ xd.abs() + accumulate(n) * ((dz[i].abs() + edz[i]).T @ xd.abs() + old[i].abs())
            check(dw[i].t, rdw[i] + old[i], err, gt, f"dw{i}")
        if "db" in want:
            err = (raw[i].sum(0) + accumulate(8 * n) * dz[i].abs().sum(0) + 2.0 ** -23 * old[parts + i].abs())
            check(db[i].t, (rdb[i] + old[parts + i]), err, gt, f"db{i}")
    return [m.t.clone() for m in (dx, *dw, *db)]


SIZES = [(1, 1, 1), (1, 8, 8), (2, 17, 33), (7, 100, 136), (31, 129, 65), (64, 64, 64), (65, 257, 300), (128, 128, 128), (130, 66, 200),
         (200, 1000, 1024), (300, 517, 203), (512, 768, 640), (1000, 777, 515), (3000, 100, 72)]


@pytest.mark.parametrize("n,M,K", SIZES)
@pytest.mark.parametrize("gated", [False, True])
def test_sizes(n, M, K, gated):
    backward(gated, n, M, K)
    backward(gated, n, M, K, "f16", "gelu_tanh", f32=False)
    backward(gated, n, M, K, act="none")


@pytest.mark.parametrize("act", ref.ACTS)
@pytest.mark.parametrize("type_", ["bf16", "f16"])
@pytest.mark.parametrize("gated", [False, True])
def test_activations(gated, type_, act):
    for f32 in (False, True):
        backward(gated, 150, 200, 320, type_, act, f32=f32)


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("n", [3, 200, 2000])
def test_accumulate(gated, f32, n):
    backward(gated, n, 136, 200, f32=f32, accumulate_into=True)
    backward(gated, n, 61, 67, f32=f32, accumulate_into=True, act="none")


@pytest.mark.parametrize("want", [("dx",), ("dw",), ("db",), ("dx", "db"), ("dw", "db")])
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("act", ["none", "gelu"])
def test_parts(want, gated, act):
    out = backward(gated, 77, 136, 200, want=want, act=act)
    parts = 2 if gated else 1
    for i, m in enumerate(out):
        name = "dx" if i == 0 else "dw" if i <= parts else "db"
        if name not in want:
            assert torch.isnan(m).all(), name


@pytest.mark.parametrize("pads,first", [((8,) * 6, 0), ((3, 0, 0, 0, 0, 0), 0), ((0, 5, 0, 0, 0, 0), 0), ((0, 0, 1, 0, 0, 0), 0),
                                        ((0, 0, 0, 7, 0, 0), 0), ((0, 0, 0, 0, 1, 0), 0), ((0, 0, 0, 0, 0, 3), 0), ((1, 2, 3, 4, 5, 6), 0),
                                        ((0,) * 6, 1), ((64, 0, 128, 8, 16, 24), 8)])
@pytest.mark.parametrize("gated", [False, True])
def test_strides_and_alignment(pads, first, gated):
    backward(gated, 90, 136, 264, pads=pads, first=first)
    backward(gated, 90, 136, 264, pads=pads, first=first, act="none", f32=False)


@pytest.mark.parametrize("kernel", [1, 2])
@pytest.mark.parametrize("tile", [64, 128, 192, 256])
@pytest.mark.parametrize("gated", [False, True])
def test_every_tile(kernel, tile, gated):
    bsk.set_option("linear_kernel", kernel)
    bsk.set_option("linear_tile", tile)
    for n, M, K in ((90, 300, 200), (600, 700, 300), (130, 129, 513)):
        backward(gated, n, M, K)


@pytest.mark.parametrize("split", [2, 4, 8])
@pytest.mark.parametrize("tile", [64, 256])
@pytest.mark.parametrize("gated", [False, True])
def test_split_k(split, tile, gated):
    bsk.set_option("linear_kernel", 1)
    bsk.set_option("split_k", split)
    bsk.set_option("linear_tile", tile)
    for n, M, K in ((1100, 77, 130), (2000, 1024, 60), (90, 1200, 300)):
        backward(gated, n, M, K, accumulate_into=True)


@pytest.mark.parametrize("gated", [False, True])
def test_no_tokens_and_no_features(gated):
    """Empty sums: zero gradients of the weights, or nothing added; a dx of zeros."""
    t = torch.bfloat16
    parts = 2 if gated else 1

    def call(n, M, K, acc, dx, dw, db):
        x, w, z = torch.ones(max(n, 1), K, dtype=t, device="cuda"), torch.ones(max(M, 1), K, dtype=t, device="cuda"), torch.ones(
            max(n, 1), max(M, 1), dtype=t, device="cuda")
        if gated:
            bsk.gated_linear_backward(0, w, w, K, x, K, z, z, max(M, 1), z, max(M, 1), dx, K, dw[0], dw[1], K, db[0], db[1], 0, acc, M,
                                      K, n, bsk.ACT_SILU)
        else:
            bsk.linear_act_backward(0, w, K, x, K, z, max(M, 1), z, max(M, 1), dx, K, dw[0], K, db[0], 0, acc, M, K, n, bsk.ACT_SILU)

    for acc in (0, 1):
        dw, db = [torch.full((5, 7), 3.0, device="cuda") for _ in range(parts)], [torch.full((5,), 2.0, device="cuda") for _ in range(parts)]
        call(0, 5, 7, acc, None, dw, db)
        assert all(bool((m == 3.0 * acc).all()) for m in dw) and all(bool((m == 2.0 * acc).all()) for m in db)
    dx = torch.full((4, 7), 3.0, dtype=t, device="cuda")
    call(4, 0, 7, 0, dx, [None] * parts, [None] * parts)
    assert bool((dx == 0).all())


def test_bias_gradient_without_inputs():
    """K = 0 leaves the bias's gradient."""
    dy, z = draw(1, 50, 33), draw(2, 50, 33)
    db = torch.empty(33, device="cuda")
    bsk.linear_act_backward(0, None, 1, None, 1, z, 33, dy, 33, None, 1, None, 1, db, 0, 0, 33, 0, 50, bsk.ACT_GELU)
    want = (dy.double() * ref.act("gelu", z.double())[1]).sum(0)
    assert (db.double() - want).abs().max() <= 50 * 2.0 ** -14 * dy.double().abs().max()


def test_repeated_calls_give_equal_bits():
    for shape in ((300, 500, 512), (2000, 130, 200)):
        for a, b in zip(backward(True, *shape), backward(True, *shape, enqueue=True)):
            assert torch.equal(a, b)


def test_derivatives_far_out():
    """Far out the derivatives are 0 or 1: no NaN from 0 times infinity."""
    z = torch.tensor([-3e38, -1e20, -1e10, -100.0, -20.0, 20.0, 100.0, 1e10, 1e20, 3e38, 0.0, -0.0], device="cuda").bfloat16()[:, None].repeat(1, 8)
    dy = torch.ones_like(z)
    for name in ref.ACTS:
        db = torch.empty(8, device="cuda")
        for r in range(z.shape[0]):
            bsk.linear_act_backward(0, None, 1, None, 1, z[r:r + 1], 8, dy, 8, None, 1, None, 1, db, 0, 0, 8, 0, 1, ACT[name])
            want = ref.act(name, z[r:r + 1].double())[1][0]
            if name == "gelu_tanh":   # the formula's own second term is 0 * infinity here
                want = torch.where(z[r].double().abs() >= 20, (z[r] > 0).double(), want)
            assert torch.isfinite(db).all(), (name, z[r, 0])
            assert (db.double() - want).abs().max() <= 2.0 ** -14, (name, z[r, 0], db, want)


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("act", ["gelu", "gelu_tanh", "silu", "none"])
def test_against_differences(gated, act):
    """The loss sum(dy * forward) moved along random directions of x, W and b, by central differences of the formula in
    64 bits (step 1e-5: an error of 1e-10 of the third derivative), against the gradients' products with them.  z comes in
    16 bits: the derivative is taken at that z, half a step (2^-11 relative, FP16) from the formula's, which moves each
    dz by 2^-11 |z| CURVE |dy u| at most, beside the gradients' own roundings (2^-11)."""
    n, M, K = 40, 72, 56
    t = torch.float16
    x, w, b = draw(1, n, K, t=t), [draw(2 + i, M, K, size=K ** -0.5, t=t) for i in range(2)], [draw(5 + i, M, size=0.3, t=t) for i in range(2)]
    dy = draw(8, n, M, t=t)
    g, u = (torch.empty(n, M, dtype=t, device="cuda") for _ in range(2))
    out = torch.empty(n, M, dtype=t, device="cuda")
    dx, dw, db = torch.empty(n, K, dtype=t, device="cuda"), [torch.empty(M, K, device="cuda") for _ in range(2)], [torch.empty(M, device="cuda") for _ in range(2)]
    if gated:
        bsk.gated_linear(1, w[0], w[1], K, x, K, b[0], b[1], out, M, g, u, M, M, K, n, ACT[act])
        bsk.gated_linear_backward(1, w[0], w[1], K, x, K, g, u, M, dy, M, dx, K, dw[0], dw[1], K, db[0], db[1], 0, 0, M, K, n, ACT[act])
    else:
        bsk.linear_act(1, w[0], K, x, K, b[0], None, 0, out, M, g, M, M, K, n, ACT[act])
        bsk.linear_act_backward(1, w[0], K, x, K, g, M, dy, M, dx, K, dw[0], K, db[0], 0, 0, M, K, n, ACT[act])

    def loss(x, w, b):
        y = ref.gated(act, x, w[0], w[1], b[0], b[1])[0] if gated else ref.linear(act, x, w[0], b[0])[0]
        return float((dy.double() * y).sum())

    xd, wd, bd = x.double(), [v.double() for v in w], [v.double() for v in b]
    parts = 2 if gated else 1
    for seed in range(3):
        vx = draw(30 + seed, n, K, t=torch.float64)
        vw = [draw(40 + 10 * i + seed, M, K, t=torch.float64) for i in range(2)]
        vb = [draw(60 + 10 * i + seed, M, t=torch.float64) for i in range(2)]
        s = 1e-5
        moved = [loss(xd + k * s * vx, [a + k * s * d for a, d in zip(wd, vw)], [a + k * s * d for a, d in zip(bd, vb)]) for k in (1, -1)]
        numeric = (moved[0] - moved[1]) / (2 * s)
        got = float((dx.double() * vx).sum() + sum((dw[i].double() * vw[i]).sum() + (db[i].double() * vb[i]).sum() for i in range(parts)))
        # the step along (vx, vw, vb) moves every z by at most `reach`; a dz wrong by e changes the product by e * reach
        reach = [vx.abs() @ a.abs().T + xd.abs() @ d.abs().T + e.abs() for a, d, e in zip(wd, vw, vb)]
        mags = [u.double().abs() + 1, g.double().abs() + 1] if gated else [torch.ones_like(reach[0])]
        z = g.double().abs()
        bound = sum((dy.double().abs() * m * (2.0 ** -10 * 1.13 + 2.0 ** -11 * (z + 1) * ref.CURVE) * r).sum() for m, r in zip(mags, reach))
        assert abs(got - numeric) <= float(bound) and math.isfinite(got), (got, numeric, float(bound))
        # and much closer than the worst case, which adds all signs: errors of random sign add up like a walk
        assert abs(got - numeric) <= 8 * float(bound) / math.sqrt(n * M) + 1e-6 * abs(numeric)
