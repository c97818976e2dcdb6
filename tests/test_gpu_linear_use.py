"""The feed-forward calls as a program uses them: a block's forward and backward pass together, in CUDA graphs,
on other streams and host threads, chained without synchronisation."""
import math
import random
import threading

import pytest
import torch

import linear_reference as ref
from bf16_gemm_skinny_gb300 import _native as bsk
from bf16_gemm_skinny_gb300 import build as bsk_build
from test_gpu_linear import accumulate, check, draw, forward
from test_gpu_linear_grad import backward

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def lib():
    bsk_build.build()
    torch.cuda.init()
    yield bsk.load()
    for k in bsk.OPTIONS:
        bsk.set_option(k, 0)


class Block:
    """y = r + Wd (silu(x Wg^T) * (x Wu^T)) + bd: a gated feed-forward block on a residual stream, with its buffers."""

    def __init__(self, n, hidden, width, t=torch.bfloat16, seed=0):
        self.n, self.hidden, self.width, self.t = n, hidden, width, t
        self.kind = bsk.TYPE_BF16 if t == torch.bfloat16 else bsk.TYPE_F16
        self.x, self.r = draw(seed, n, width, t=t), draw(seed + 1, n, width, t=t)
        self.wg, self.wu = (draw(seed + 2 + i, hidden, width, size=width ** -0.5, t=t) for i in range(2))
        self.wd, self.bd = draw(seed + 4, width, hidden, size=hidden ** -0.5, t=t), draw(seed + 5, width, size=0.1, t=t)
        self.dy = draw(seed + 6, n, width, size=0.1, t=t)
        e = lambda *s, d=t: torch.zeros(*s, dtype=d, device="cuda")  # noqa: E731
        self.h, self.g, self.u, self.y = e(n, hidden), e(n, hidden), e(n, hidden), e(n, width)
        self.dh, self.dx = e(n, hidden), e(n, width)
        self.dwd, self.dbd = e(width, hidden, d=torch.float32), e(width, d=torch.float32)
        self.dwg, self.dwu = e(hidden, width, d=torch.float32), e(hidden, width, d=torch.float32)

    def forward(self, stream=None):
        n, m, k = self.n, self.hidden, self.width
        bsk.gated_linear_enqueue(self.kind, self.wg, self.wu, k, self.x, k, None, None, self.h, m, self.g, self.u, m, m, k, n,
                                 bsk.ACT_SILU, stream)
        bsk.linear_act_enqueue(self.kind, self.wd, m, self.h, m, self.bd, self.r, k, self.y, k, None, k, k, m, n, bsk.ACT_NONE, stream)

    def backward(self, accumulate=0, stream=None):
        n, m, k = self.n, self.hidden, self.width
        bsk.linear_act_backward_enqueue(self.kind, self.wd, m, self.h, m, None, k, self.dy, k, self.dh, m, self.dwd, m, self.dbd,
                                        bsk.GRAD_F32, accumulate, k, m, n, bsk.ACT_NONE, stream)
        bsk.gated_linear_backward_enqueue(self.kind, self.wg, self.wu, k, self.x, k, self.g, self.u, m, self.dh, m, self.dx, k,
                                          self.dwg, self.dwu, k, None, None, bsk.GRAD_F32, accumulate, m, k, n, bsk.ACT_SILU, stream)

    def outputs(self):
        return [self.h, self.g, self.u, self.y, self.dh, self.dx, self.dwd, self.dbd, self.dwg, self.dwu]

    def clone(self):
        return [o.clone() for o in self.outputs()]

    def clear(self):
        for o in self.outputs():
            o.fill_(float("nan"))


@pytest.mark.parametrize("n,hidden,width", [(1, 256, 128), (5, 1000, 264), (150, 704, 520), (700, 1024, 512)])
@pytest.mark.parametrize("t", [torch.bfloat16, torch.float16])
def test_block(n, hidden, width, t):
    """Each call's outputs against the formula in 64 bits on what the call before it left."""
    b = Block(n, hidden, width, t)
    b.forward()
    b.backward()
    bsk.stream_check()
    d = lambda v: v.double()  # noqa: E731
    h, g, u = ref.gated("silu", d(b.x), d(b.wg), d(b.wu))
    eg = accumulate(width) * (d(b.x).abs() @ d(b.wg).abs().T)
    eu = accumulate(width) * (d(b.x).abs() @ d(b.wu).abs().T)
    a = ref.act("silu", g)[0]
    ea = ref.SLOPE * eg + 2.0 ** -15 * a.abs()
    check(b.h, h, a.abs() * eu + u.abs() * ea + ea * eu, t, "h")
    y, _ = ref.linear("none", d(b.h), d(b.wd), d(b.bd), d(b.r))
    ey = accumulate(hidden) * (d(b.h).abs() @ d(b.wd).abs().T + d(b.bd).abs() + d(b.r).abs())
    check(b.y, y, ey, t, "y")
    dh, dwd, dbd, _ = ref.linear_backward("none", d(b.h), d(b.wd), None, d(b.dy))
    check(b.dh, dh, accumulate(width) * (d(b.dy).abs() @ d(b.wd).abs()), t, "dh")
    check(b.dwd, dwd, accumulate(n) * (d(b.dy).abs().T @ d(b.h).abs()), torch.float32, "dWd")
    check(b.dbd, dbd, accumulate(8 * n) * d(b.dy).abs().sum(0), torch.float32, "dbd")
    dx, dwg, dwu, _, _, dg, du = ref.gated_backward("silu", d(b.x), d(b.wg), d(b.wu), d(b.g), d(b.u), d(b.dh))
    eg = 2.0 ** -14 * (d(b.dh) * d(b.u)).abs()
    eg = eg + ref.half_step(t) * (dg.abs() + eg) + ref.tiny(t)
    eu = 2.0 ** -14 * du.abs()
    eu = eu + ref.half_step(t) * (du.abs() + eu) + ref.tiny(t)
    ex = eg @ d(b.wg).abs() + eu @ d(b.wu).abs()
    check(b.dx, dx, ex + accumulate(2 * hidden) * ((dg.abs() + eg) @ d(b.wg).abs() + (du.abs() + eu) @ d(b.wu).abs()), t, "dx")
    for got, want, e, z in ((b.dwg, dwg, eg, dg), (b.dwu, dwu, eu, du)):
        check(got, want, e.T @ d(b.x).abs() + accumulate(n) * ((z.abs() + e).T @ d(b.x).abs()), torch.float32, "dW")


def test_block_accumulates():
    """Two backward passes with accumulate: twice the gradients (FP32 sums of equal values are exact)."""
    b = Block(300, 512, 256)
    b.forward()
    b.backward()
    once = [v.clone() for v in (b.dwd, b.dbd, b.dwg, b.dwu)]
    b.backward(accumulate=1)
    bsk.stream_check()
    for v, o in zip((b.dwd, b.dbd, b.dwg, b.dwu), once):
        assert torch.equal(v, 2 * o)


def test_graphs():
    """Two graphs of two blocks, with workspaces of their own (dz, sums, packed operands), replayed in turn
    and after each other on new inputs: the bits of the eager calls."""
    blocks = [Block(200, 520, 264), Block(90, 1003, 131, torch.float16, seed=50)]   # the second: unaligned rows
    graphs = []
    for b in blocks:
        b.forward()
        b.backward()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        side = torch.cuda.Stream()
        with torch.cuda.graph(g, stream=side):
            b.forward(side)
            b.backward(stream=side)
        graphs.append(g)
    for seed in (100, 200):
        want = []
        for b in blocks:
            for v, s in ((b.x, 1.0), (b.r, 1.0), (b.dy, 0.1)):
                v.copy_(draw(seed, *v.shape, size=s, t=v.dtype))
                seed += 1
            b.forward()
            b.backward()
            bsk.stream_check()
            want.append(b.clone())
            b.clear()
        for order in ((0, 1), (1, 0), (0, 0, 1, 1)):
            for i in order:
                graphs[i].replay()
            torch.cuda.synchronize()
            for b, w in zip(blocks, want):
                assert all(torch.equal(o, v) for o, v in zip(b.outputs(), w))
                b.clear()


def test_streams_side_by_side():
    """Blocks on two streams at once, another being the current one: the bits of one after the other."""
    blocks = [Block(120, 800, 256, seed=10), Block(60, 900, 320, seed=30)]
    want = []
    for b in blocks:
        b.forward()
        b.backward()
        bsk.stream_check()
        want.append(b.clone())
    streams = [torch.cuda.Stream() for _ in blocks]
    for _ in range(20):
        for b in blocks:
            b.clear()
        torch.cuda.synchronize()
        for b, s in zip(blocks, streams):
            b.forward(s)
            b.backward(stream=s)
        for s in streams:
            bsk.stream_check(s)
        for b, w in zip(blocks, want):
            assert all(torch.equal(o, v) for o, v in zip(b.outputs(), w))


def test_host_threads():
    blocks = [Block(40 + 30 * i, 300 + 64 * i, 128 + 8 * i, seed=7 * i) for i in range(4)]
    want = []
    for b in blocks:
        b.forward()
        b.backward()
        bsk.stream_check()
        want.append(b.clone())
        b.clear()
    torch.cuda.synchronize()
    failed = []

    def work(b, w):
        try:
            s = torch.cuda.Stream()
            for _ in range(30):
                b.forward(s)
                b.backward(stream=s)
            bsk.stream_check(s)
            assert all(torch.equal(o, v) for o, v in zip(b.outputs(), w))
        except Exception as e:   # noqa: BLE001
            failed.append(e)

    threads = [threading.Thread(target=work, args=a) for a in zip(blocks, want)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed, failed


@pytest.mark.parametrize("n", [1, 7, 130])
def test_chain_on_one_residual_stream(n):
    """Layer after layer without a synchronisation, each adding to the same residual stream in place: with and
    without programmatic launches the same bits, and those of calls that wait for each other."""
    t, hidden, width, layers = torch.bfloat16, 768, 256, 6
    ws = [[draw(100 + 10 * i + k, *((hidden, width) if k < 2 else (width, hidden)), size=(width if k < 2 else hidden) ** -0.5)
           for k in range(3)] for i in range(layers)]
    x = draw(1, n, width)

    def run(blocking):
        y, h = x.clone(), torch.empty(n, hidden, dtype=t, device="cuda")
        suffix = "" if blocking else "_enqueue"
        for wg, wu, wd in ws:
            getattr(bsk, "gated_linear" + suffix)(0, wg, wu, width, y, width, None, None, h, hidden, None, None, hidden, hidden, width,
                                                  n, bsk.ACT_SILU)
            getattr(bsk, "linear_act" + suffix)(0, wd, hidden, h, hidden, None, y, width, y, width, None, width, width, hidden, n,
                                                bsk.ACT_NONE)
        bsk.stream_check()
        return y

    want = run(True)
    for _ in range(10):
        assert torch.equal(run(False), want)
    bsk.set_option("pdl", 1)
    try:
        assert torch.equal(run(False), want)
    finally:
        bsk.set_option("pdl", 0)


def test_beside_the_other_calls():
    """Between a GEMV, a GEMM and a packed GEMM in one stream (kernels with other needs of shared memory and TMEM)."""
    b = Block(33, 640, 384)
    w, x = draw(71, 1000, 384), draw(72, 9, 384)
    y = torch.empty(9, 1000, dtype=torch.bfloat16, device="cuda")
    a16 = torch.randn(300, 200, device="cuda").half()
    c16 = torch.empty(300, 300, dtype=torch.half, device="cuda")

    def run(wait):
        for _ in range(3):
            bsk.gemv_bf16_enqueue(w, x, y, 1000, 384, 9)
            if wait:
                torch.cuda.synchronize()
            b.forward()
            if wait:
                torch.cuda.synchronize()
            bsk.gemm_f16_enqueue(bsk.ROW_MAJOR, 0, 1, a16, 200, a16, 200, c16, 300, 300, 300, 200)
            if wait:
                torch.cuda.synchronize()
            b.backward()
            if wait:
                torch.cuda.synchronize()
        bsk.stream_check()
        return b.clone() + [y.clone(), c16.clone()]

    want = run(True)
    for _ in range(5):
        b.clear()
        assert all(torch.equal(p, q) for p, q in zip(run(False), want))


@pytest.mark.parametrize("call", ["linear_act", "gated_linear", "linear_act_backward", "gemm_f16"])
def test_first_call_of_a_host_thread(call):
    """A host thread whose first CUDA call is one that needs no workspace."""
    n, m, k = 128, 256, 128
    w, x, dy = draw(1, m, k), draw(2, n, k), draw(3, n, m)
    y, dx = torch.empty(n, m, dtype=torch.bfloat16, device="cuda"), torch.empty(n, k, dtype=torch.bfloat16, device="cuda")
    h16, b16 = w.half(), x.half()
    c16 = torch.empty(n, m, dtype=torch.half, device="cuda")
    stream = torch.cuda.current_stream().cuda_stream
    out = {"linear_act": y, "gated_linear": y, "linear_act_backward": dx, "gemm_f16": c16}[call]

    def run():
        if call == "linear_act":
            bsk.linear_act_enqueue(0, w, k, x, k, None, None, m, y, m, None, m, m, k, n, bsk.ACT_RELU, stream)
        elif call == "gated_linear":
            bsk.gated_linear_enqueue(0, w, w, k, x, k, None, None, y, m, None, None, m, m, k, n, bsk.ACT_RELU, stream)
        elif call == "linear_act_backward":
            bsk.linear_act_backward_enqueue(0, w, k, x, k, None, m, dy, m, dx, k, None, k, None, 0, 0, m, k, n, bsk.ACT_NONE, stream)
        else:
            bsk.gemm_f16_enqueue(bsk.ROW_MAJOR, 0, 1, b16, k, h16, k, c16, m, n, m, k, stream=stream)

    run()
    bsk.stream_check()
    want = out.clone()
    out.zero_()
    torch.cuda.synchronize()
    failed = []

    def work():
        try:
            run()
        except Exception as e:   # noqa: BLE001
            failed.append(e)

    t = threading.Thread(target=work)
    t.start()
    t.join()
    assert not failed, failed
    bsk.stream_check()
    assert torch.equal(out, want)


@pytest.mark.parametrize("n,m,k", [(3, 40, 64), (200, 264, 128), (130, 133, 100)])
def test_results_side_by_side_in_the_same_rows(n, m, k):
    """h, g and u as columns of one buffer, then dx beside x: the bits of separate buffers, and nothing else written."""
    t = torch.bfloat16
    x, wg, wu, dh = draw(1, n, k), draw(2, m, k, size=k ** -0.5), draw(3, m, k, size=k ** -0.5), draw(4, n, m)
    sep = [torch.empty(n, m, dtype=t, device="cuda") for _ in range(3)]
    dx = torch.empty(n, k, dtype=t, device="cuda")
    bsk.gated_linear(0, wg, wu, k, x, k, None, None, sep[0], m, sep[1], sep[2], m, m, k, n, bsk.ACT_SILU)
    bsk.gated_linear_backward(0, wg, wu, k, x, k, sep[1], sep[2], m, dh, m, dx, k, None, None, k, None, None, 0, 0, m, k, n, bsk.ACT_SILU)
    row = 3 * m + 5
    wide = torch.full((n, row), 7.0, dtype=t, device="cuda")
    both = torch.full((n, 2 * k), 7.0, dtype=t, device="cuda")
    both[:, :k] = x
    bsk.gated_linear(0, wg, wu, k, both, 2 * k, None, None, wide, row, wide[:, m:], wide[:, 2 * m:], row, m, k, n, bsk.ACT_SILU)
    bsk.gated_linear_backward(0, wg, wu, k, both, 2 * k, wide[:, m:], wide[:, 2 * m:], row, dh, m, both[:, k:], 2 * k, None, None, k,
                              None, None, 0, 0, m, k, n, bsk.ACT_SILU)
    for i in range(3):
        assert torch.equal(wide[:, i * m:(i + 1) * m], sep[i])
    assert bool((wide[:, 3 * m:] == 7.0).all())
    assert torch.equal(both[:, :k], x) and torch.equal(both[:, k:], dx)


def test_rows_far_apart():
    """Rows 3 GB apart (offsets past 31 bits of elements and 32 of bytes): the bits of packed ones."""
    n, m, k, far, t = 3, 72, 64, 1_500_000_008, torch.bfloat16
    if torch.cuda.mem_get_info()[0] < 120e9:
        pytest.skip("needs 120 GB")

    def apart(rows, width, dtype=t, stride=far):
        buf = torch.empty((rows - 1) * stride + width, dtype=dtype, device="cuda")
        return buf.as_strided((rows, width), (stride, 1))

    x, dh, wg, wu = draw(1, n, k), draw(2, n, m), draw(3, m, k, size=k ** -0.5), draw(4, m, k, size=k ** -0.5)
    h, g, u = (torch.empty(n, m, dtype=t, device="cuda") for _ in range(3))
    dx = torch.empty(n, k, dtype=t, device="cuda")
    bsk.gated_linear(0, wg, wu, k, x, k, None, None, h, m, g, u, m, m, k, n, bsk.ACT_SILU)
    bsk.gated_linear_backward(0, wg, wu, k, x, k, g, u, m, dh, m, dx, k, None, None, k, None, None, 0, 0, m, k, n, bsk.ACT_SILU)
    xf, hf, gf, uf, dhf, dxf = apart(n, k), apart(n, m), apart(n, m), apart(n, m), apart(n, m), apart(n, k)
    xf.copy_(x)
    dhf.copy_(dh)
    bsk.gated_linear(0, wg, wu, k, xf, far, None, None, hf, far, gf, uf, far, m, k, n, bsk.ACT_SILU)
    bsk.gated_linear_backward(0, wg, wu, k, xf, far, gf, uf, far, dhf, far, dxf, far, None, None, k, None, None, 0, 0, m, k, n,
                              bsk.ACT_SILU)
    for a, b in ((hf, h), (gf, g), (uf, u), (dxf, dx)):
        assert torch.equal(a, b)
    # weights and their FP32 gradients: three output features
    m = 3
    dwg, dwu = (torch.zeros(m, k, device="cuda") for _ in range(2))
    g3, u3, dh3, h3 = (v[:, :m].contiguous() for v in (g, u, dh, h))
    bsk.gated_linear(0, wg, wu, k, x, k, None, None, h3, m, g3, u3, m, m, k, n, bsk.ACT_SILU)
    bsk.gated_linear_backward(0, wg, wu, k, x, k, g3, u3, m, dh3, m, dx, k, dwg, dwu, k, None, None, 0, 0, m, k, n, bsk.ACT_SILU)
    del hf, gf, uf, dxf, xf, dhf
    wgf, wuf, dwgf, dwuf = apart(m, k), apart(m, k), apart(m, k, torch.float32), apart(m, k, torch.float32)
    wgf.copy_(wg[:m])
    wuf.copy_(wu[:m])
    dx2, h2 = torch.empty_like(dx), torch.empty_like(h3)
    bsk.gated_linear(0, wgf, wuf, far, x, k, None, None, h2, m, None, None, m, m, k, n, bsk.ACT_SILU)
    bsk.gated_linear_backward(0, wgf, wuf, far, x, k, g3, u3, m, dh3, m, dx2, k, dwgf, dwuf, far, None, None, 0, 0, m, k, n, bsk.ACT_SILU)
    for a, b in ((h2, h3), (dx2, dx), (dwgf, dwg), (dwuf, dwu)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("n,m,k", [(90, 136, 259), (200, 300, 260), (40, 1000, 67), (1000, 72, 515)])
@pytest.mark.parametrize("accumulate_into", [False, True])
def test_gradients_of_odd_width_in_aligned_rows(n, m, k, accumulate_into):
    """Rows 16-byte aligned, their length not whole 16-byte units: what lies between them stays (checked in backward)."""
    to8 = lambda v: -v % 8  # noqa: E731
    pads = (to8(k), to8(k), to8(m), to8(m), to8(k), to8(k))
    for gated in (False, True):
        for kernel in (0, 1, 2):
            bsk.set_option("linear_kernel", kernel)
            try:
                backward(gated, n, m, k, pads=pads, accumulate_into=accumulate_into)
                backward(gated, n, m, k, "f16", "gelu", f32=False, pads=pads, accumulate_into=accumulate_into)
            finally:
                bsk.set_option("linear_kernel", 0)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("act", ["none", "relu", "gelu", "gelu_tanh", "silu"])
@pytest.mark.parametrize("n", [2, 70, 300])
def test_one_bad_value_reaches_only_what_it_enters(n, act, bad):
    m, k, j, r, c = 136, 72, 37, 1, 50
    kind = dict(none=0, relu=1, gelu=2, gelu_tanh=3, silu=4)[act]
    t = torch.bfloat16
    x, w, w2, dy = draw(1, n, k), draw(2, m, k, size=k ** -0.5), draw(3, m, k, size=k ** -0.5), draw(4, n, m)
    x[:, c] = x[:, c].abs() + 0.5
    z, u = draw(5, n, m), draw(6, n, m)

    def forward(wx):
        y, h = (torch.empty(n, m, dtype=t, device="cuda") for _ in range(2))
        bsk.linear_act(0, wx, k, x, k, None, None, m, y, m, None, m, m, k, n, kind)
        bsk.gated_linear(0, wx, w2, k, x, k, None, None, h, m, None, None, m, m, k, n, kind)
        return y, h

    def backward_of(zx):
        dx, dgx = (torch.empty(n, k, dtype=t, device="cuda") for _ in range(2))
        dw, dg, du = (torch.empty(m, k, device="cuda") for _ in range(3))
        db, dbg, dbu = (torch.empty(m, device="cuda") for _ in range(3))
        bsk.linear_act_backward(0, w, k, x, k, zx, m, dy, m, dx, k, dw, k, db, 0, 0, m, k, n, kind)
        bsk.gated_linear_backward(0, w, w2, k, x, k, zx, u, m, dy, m, dgx, k, dg, du, k, dbg, dbu, 0, 0, m, k, n, kind)
        return (dx, dgx), (dw, db, dg, dbg, du, dbu)

    wx, zx = w.clone(), z.clone()
    wx[j, c] = bad
    zx[r, j] = bad
    # The activations take one reciprocal for the product of four values (of columns 4 i to 4 i + 3), each a
    # number from 1 to 2^30 whatever its z: the three beside another z may so have other last bits (five
    # roundings), but stay finite.  All other columns keep their bits.
    others = [i for i in range(m) if i // 4 != j // 4]
    beside = [i for i in range(m) if i // 4 == j // 4 and i != j]
    for got, want in zip(forward(wx), forward(w)):
        assert torch.equal(got[:, others], want[:, others]) and torch.isfinite(got[:, beside]).all()
        if bad != bad:
            assert torch.isnan(got[:, j]).all()
    rows = [i for i in range(n) if i != r]
    for got, want in zip(backward_of(zx), backward_of(z)):
        for a, b in zip(got, want):
            keep = rows if a.shape[0] == n and a.dtype == t else others
            assert torch.equal(a[keep], b[keep])
            assert keep is rows or torch.isfinite(a[beside]).all()
            if bad != bad and act != "none":
                assert torch.isnan(a[r] if keep is rows else a[j]).any()


@pytest.mark.parametrize("kernel,split", [(0, 0), (1, 1), (1, 4), (2, 0)])
@pytest.mark.parametrize("n,m,k", [(6, 131, 1032), (70, 520, 520), (300, 133, 1100)])
def test_residual_in_place_in_every_kernel(kernel, split, n, m, k):
    bsk.set_option("linear_kernel", kernel)
    bsk.set_option("split_k", split)
    try:
        for keep in (False, True):
            a = forward(False, n, m, k, residual=True, inplace=True, keep=keep)
            assert torch.equal(a, forward(False, n, m, k, residual=True, keep=keep))
    finally:
        bsk.set_option("linear_kernel", 0)
        bsk.set_option("split_k", 0)


@pytest.mark.parametrize("seed", range(12))
def test_random_calls(seed):
    rng = random.Random(seed)
    log = lambda lo, hi: int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))  # noqa: E731
    options = ("linear_kernel", "linear_tile", "split_k", "pdl", "group_m")
    try:
        for _ in range(12):
            for name, values in zip(options, ((0, 0, 1, 2), (0, 0, 32, 64, 96, 128, 192, 256), (0, 0, 1, 2, 4, 8), (0, 0, 1), (0, 1, 3))):
                bsk.set_option(name, rng.choice(values))
            n, m, k = log(1, 900), log(1, 1200), log(1, 1500)
            pads = tuple(rng.choice((0, 0, 1, 3, 8, 64)) for _ in range(6))
            first = rng.choice((0, 0, 8, 1))
            kind, act, gated = rng.choice(("bf16", "f16")), rng.choice(ref.ACTS), rng.random() < 0.5
            if rng.random() < 0.5:
                forward(gated, n, m, k, kind, act, bias=rng.random() < 0.5, residual=not gated and rng.random() < 0.5,
                        keep=rng.random() < 0.5, pads=pads[:4], first=first, seed=seed)
            else:
                backward(gated, n, m, k, kind, act, f32=rng.random() < 0.5, accumulate_into=rng.random() < 0.5, pads=pads, first=first,
                         seed=seed)
    finally:
        for name in options:
            bsk.set_option(name, 0)
