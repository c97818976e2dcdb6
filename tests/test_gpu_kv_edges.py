"""GPU parity of the paged-cache calls where a number format, a range or a
bound ends: token arrays whose first rows belong to no sequence, scales of a
quantised cache far apart or at their least, softmax scales and scores at the
ends of FP32, loose bounds.  Against the definition in 64 bits, within the bound of
kv_reference.attention_bound unless a test says otherwise."""
import math

import pytest
import torch

import kv_reference as ref
import test_gpu_kv_attention as att
from bf16_gemm_skinny_gb300 import _native as bsk
from bf16_gemm_skinny_gb300 import build as bsk_build

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def lib():
    import oracle

    bsk_build.build()
    oracle.build()
    torch.cuda.init()
    yield bsk.load()


@pytest.fixture
def kernel():
    """Sets the kernel: 1 many rows (an E4M3 cache converted tile by tile), 2 few rows."""
    yield lambda k: bsk.set_option("kv_kernel", k)
    bsk.set_option("kv_kernel", 0)


def bits(t):
    return t.cpu().view(torch.int16) if t.dtype == torch.bfloat16 else t.cpu()


# ---------------------------------------------------------------------------
# Token rows before cu_tokens[0]
# ---------------------------------------------------------------------------
def leading(e4m3, first=3):
    """Two sequences with 2 and 4 new tokens, whose rows begin at `first`."""
    p = ref.Problem(51, [20, 9], [2, 4], heads=2, group=2, dim=64, page=16, e4m3=e4m3)
    g = torch.Generator().manual_seed(1)
    p.cu = [c + first for c in p.cu]
    p.tokens += first
    p.fused = torch.randn(p.tokens, p.stride, generator=g).bfloat16()
    p.q = p.fused[:, :p.hq * p.dim].reshape(p.tokens, p.hq, p.dim)
    return p


@pytest.mark.parametrize("e4m3", [False, True])
def test_append_leaves_rows_before_the_first_sequence_alone(e4m3):
    p = leading(e4m3)
    want = [x if x is None else x.clone() for x in (p.k, p.v, p.ks, p.vs)]
    for r, s, pos in ref.new_positions(p.cu, p.lens):
        at = p.tables[s][pos // p.page], pos % p.page
        for i, col in ((0, p.hq), (1, p.hq + p.heads)):
            x = p.fused[r, col * p.dim:(col + p.heads) * p.dim].reshape(p.heads, p.dim)
            if e4m3:
                want[i][at], want[i + 2][at] = ref.quantise(x)
            else:
                want[i][at] = x
    d = p.device()
    k, v = d["fused"][:, p.hq * p.dim:], d["fused"][:, (p.hq + p.heads) * p.dim:]
    bsk.kv_cache_append(int(e4m3), d["k"], d["v"], d["ks"], d["vs"], k, p.stride, v, p.stride, d["cu"], d["tables"],
                        d["lens"], 2, p.tokens, *p.shape())
    for name, w in zip(("k", "v", "ks", "vs"), want):
        assert w is None or torch.equal(bits(d[name]), bits(w)), name


@pytest.mark.parametrize("e4m3", [False, True])
def test_gather_leaves_rows_before_the_first_sequence_alone(e4m3):
    p = leading(e4m3)
    d = p.device()
    out = [torch.full((p.tokens, p.heads, p.dim), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    bsk.kv_cache_gather(int(e4m3), d["k"], d["v"], d["ks"], d["vs"], *out, d["cu"], d["tables"], d["lens"], 2, p.tokens,
                        *p.shape())
    for o, x in zip(out, p.values()):
        want = torch.full((p.tokens, p.heads, p.dim), 7.0, dtype=torch.bfloat16)
        for r, s, pos in ref.new_positions(p.cu, p.lens):
            want[r] = x[p.tables[s][pos // p.page], pos % p.page].bfloat16()
        assert torch.equal(bits(o), bits(want))


@pytest.mark.parametrize("e4m3", [False, True])
def test_attention_leaves_rows_before_the_first_sequence_alone(e4m3):
    p = leading(e4m3)
    got = att.run(p)
    assert torch.isnan(got[:3]).all()
    got[:3] = 0
    att.check(p, got)


# ---------------------------------------------------------------------------
# Bounds
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("new,group", [([1], 2), ([5, 0, 140], 8), ([300], 2)])
def test_a_loose_bound_of_new_tokens(e4m3, new, group):
    """max_chunk far above the tokens there are: as with the exact bound."""
    lens = [n + 40 for n in new]
    p = ref.Problem(82, lens, new, 1, group, 64, 16, e4m3)
    want = att.run(p, max_chunk=sum(new))
    att.check(p, want)
    for loose in (2 ** 31 - 1, 2 ** 30 + 5, sum(new) + 1):
        assert torch.equal(att.run(p, max_chunk=loose), want)


# ---------------------------------------------------------------------------
# Softmax scales and scores at the ends of FP32
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("which,new", [(0, 5), (1, 5), (2, 5), (1, 70), (0, 200)])
@pytest.mark.parametrize("scale", [0.0, 1e-45, 1e-38, 1e-30, -1e-8, 0.125])
def test_small_scales_with_small_queries(kernel, which, new, scale):
    """Rows of queries that are zero, 2^-40, 2^-110 or as usual: with no scale to speak of, the mean of what they see."""
    p = ref.Problem(71, [330], [new], 1, 2, 64, 16, True)
    for r in range(new):
        p.fused[r, :128] = (p.fused[r, :128].float() * (0.0, 2.0 ** -40, 1.0, 2.0 ** -110)[r % 4]).bfloat16()
    p.q = p.fused[:new, :128].reshape(new, 2, 64)
    kernel(which)
    att.check(p, att.run(p, scale=scale), scale=scale)
    att.check(p, att.run(p, 17, 2, scale=scale), 17, 2, scale=scale)


@pytest.mark.parametrize("which,new", [(0, 3), (1, 3), (2, 3), (1, 70), (0, 200)])
@pytest.mark.parametrize("e4m3", [False, True])
def test_large_scales_with_large_queries_on_zero_keys(kernel, e4m3, which, new):
    """Scores of 0 however large scale and query are: the mean of what a token sees."""
    p = ref.Problem(72, [230], [new], 1, 2, 64, 16, e4m3)
    p.k[p.used] = 0
    if e4m3:
        p.ks[p.used] = 127
    p.fused[:, :128] = (p.fused[:, :128].float() * 2.0 ** 100).bfloat16()
    p.q = p.fused[:new, :128].reshape(new, 2, 64)
    kernel(which)
    for scale in (2.3e38, 2.0 ** 60, -1.0):
        att.check(p, att.run(p, scale=scale), scale=scale)


# ---------------------------------------------------------------------------
# Scales of a quantised cache's values
# ---------------------------------------------------------------------------
def put(p, t, x=None, y=None):
    """Position t of sequence 0: keys x, values y."""
    b, o = p.tables[0][t // p.page], t % p.page
    if x is not None:
        p.k[b, o], p.ks[b, o] = ref.quantise(x.bfloat16())
    if y is not None:
        p.v[b, o], p.vs[b, o] = ref.quantise(y.bfloat16())


def flat_tail(n, new, group, dim, tail, spread, where, peak_value=1.0):
    """One sequence of n positions whose scores are the same but for two: one key with 2^tail times the others' weight,
    and one whose value is 2^spread times as large and either has no weight or is seen by the last token only."""
    p = ref.Problem(61, [n], [new], 1, group, dim, 16)
    g = torch.Generator().manual_seed(62)
    p.e4m3 = True
    p.k = torch.zeros(p.k.shape, dtype=torch.uint8)
    p.v = torch.randint(0x28, 0x7f, p.v.shape, generator=g, dtype=torch.uint8)     # 0.25 .. 448, all positive
    p.ks = torch.full(p.k.shape[:-1], 127, dtype=torch.uint8)
    p.vs = p.ks.clone()
    p.fused[:, :group * dim] = 1.0
    p.q = p.fused[:, :group * dim].reshape(new, group, dim)
    one = torch.ones(1, dim)
    score = 1 / (dim * (1 / math.sqrt(dim)))                                       # a constant key's value per unit of score
    put(p, 3, one * (tail * math.log(2) * score), None if peak_value else 0 * one)
    t = n - 1 if where == "unseen" else 7
    if where == "weightless":
        put(p, t, one * (-100 * score))
    if spread:
        p.vs[p.tables[0][t // 16], t % 16] = 127 + spread
    return p


TAILS = [(4, 2000, 10), (9, 2000, 10), (12, 4000, 11), (14, 4000, 11), (16, 4000, 10), (20, 200, 7.5), (20, 4000, 9)]


@pytest.mark.parametrize("where", ["weightless", "unseen"])
@pytest.mark.parametrize("which,new,dim", [(0, 4, 128), (2, 4, 64), (2, 4, 256), (1, 4, 128), (1, 70, 64), (1, 70, 256), (0, 300, 128)])
@pytest.mark.parametrize("spread,n,tail", TAILS)
def test_a_large_value_of_no_weight_costs_the_others_nothing(kernel, spread, n, tail, which, new, dim, where):
    p = flat_tail(max(n, new), new, 2, dim, tail, spread, where)
    kernel(which)
    att.check(p, att.run(p))
    att.check(p, att.run(p, segments=3))


@pytest.mark.parametrize("which,new", [(0, 2), (1, 2), (2, 40)])
def test_a_flat_tail_beside_a_key_without_value(kernel, which, new):
    """Weights of 2^-22 of the row's largest, whose own value is zero: FP16 weights beside E4M3 values hold them to 2^-10."""
    p = flat_tail(4000, new, 2, 128, 22, 0, "weightless", peak_value=0.0)
    kernel(which)
    att.check(p, att.run(p))


@pytest.mark.parametrize("which", [0, 1])
@pytest.mark.parametrize("spread,tail", [(14, 14), (12, 16.5), (8, 18)])
def test_long_flat_tails(kernel, which, spread, tail):
    p = flat_tail(30000, 2, 2, 64, tail, spread, "weightless")
    k, v = p.values()
    out, span, reach = ref.attention_on_gpu(p.q, k, v, p.tables, p.cu, p.lens, 1, 16, 1 / 8)
    kernel(which)
    assert ((att.run(p).double() - out).abs() <= ref.attention_bound(out, span, reach, 1 / 8, 64, 30000)).all()


@pytest.mark.parametrize("which", [0, 1, 2])
@pytest.mark.parametrize("step", [3, -3, 17, -17])
def test_scales_that_rise_and_fall(kernel, which, step):
    """Scales from 2^-40 to 2^40 in steps along the sequence; windows of like and of unlike rows."""
    n = 400
    p = ref.Problem(63, [n], [60], 1, 2, 64, 16, True)
    for t in range(n):
        e = (t // 20 * step) % 81 - 40
        p.vs[p.tables[0][t // 16], t % 16] = 127 + e
    kernel(which)
    for window, sinks in ((0, 0), (15, 0), (40, 2)):
        att.check(p, att.run(p, window, sinks), window, sinks)


# ---------------------------------------------------------------------------
# The least scale (2^-117)
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("which,new", [(0, 3), (1, 3), (2, 3), (1, 90), (0, 200)])
@pytest.mark.parametrize("others", ["none", "zero", "large"])
def test_values_under_the_least_scale(kernel, which, new, others):
    """Values of 2^-112 to 2^-122 (their scale is held at 2^-117), alone, beside rows of zeros, and beside rows of
    ordinary size that most tokens do not see."""
    n = 300
    p = ref.Problem(64, [n], [new], 1, 2, 64, 16, True)
    g = torch.Generator().manual_seed(65)
    for t in range(n):
        x = torch.randn(1, 64, generator=g) * 2.0 ** (-112 - t % 11)
        if others == "zero" and t % 3 == 1:
            x = x * 0
        if others == "large" and t in (n - 1, n - 101):
            x = x.sign()
        put(p, t, None, x)
    kernel(which)
    assert int(p.vs.min()) == 10
    for window, sinks in ((0, 0), (20, 0)):
        att.check(p, att.run(p, window, sinks), window, sinks)


@pytest.mark.parametrize("which", [0, 1, 2])
def test_rows_of_zeros_among_ordinary_values(kernel, which):
    """Zero rows have the least scale: whole tiles of them, before, between and after others."""
    n = 500
    p = ref.Problem(66, [n], [6], 1, 2, 64, 16, True)
    for t in range(n):
        if t < 130 or t % 5 == 0 or t > 400:
            put(p, t, None, torch.zeros(1, 64))
    kernel(which)
    for window, sinks in ((0, 0), (60, 3), (480, 0)):
        att.check(p, att.run(p, window, sinks), window, sinks)


# ---------------------------------------------------------------------------
# Scales of a quantised cache's keys
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("which,new", [(0, 2), (1, 2), (2, 2), (1, 70)])
@pytest.mark.parametrize("e", [80, 100, 112, 119])
def test_large_keys_with_small_queries(kernel, which, new, e):
    """Keys about 2^e beside queries about 2^-e: ordinary scores."""
    p = ref.Problem(73, [200], [new], 1, 2, 64, 16, True)
    p.ks = (p.ks.int() + e).clamp(max=247).to(torch.uint8)
    p.fused[:, :128] = (p.fused[:, :128].float() * 2.0 ** -e).bfloat16()
    p.q = p.fused[:new, :128].reshape(new, 2, 64)
    kernel(which)
    att.check(p, att.run(p))


# ---------------------------------------------------------------------------
# Workspaces
# ---------------------------------------------------------------------------
@pytest.fixture
def workspace_kb():
    yield lambda kb: bsk.set_option("kv_workspace_kb", kb)
    bsk.set_option("kv_workspace_kb", 0)


@pytest.mark.parametrize("segments", [0, 1, 3])
def test_no_memory_for_the_flat_copy(workspace_kb, segments):
    """A quantised cache read by many rows is converted tile by tile where its BF16 copy finds no room."""
    p = ref.Problem(91, [900, 700], [300, 150], 2, 2, 128, 16, True)
    plan = bsk.plan_kv_attention(bsk.CACHE_E4M3, 2, 450, 300, 4, 2, 128, 900, num_segments=segments)
    copy = plan["flat_rows"] * 2 * 2 * 128 * 4
    assert copy > 0
    att.check(p, att.run(p, segments=segments))
    workspace_kb(copy // 1024 - 1)
    if segments == 3 and 450 * 4 * 3 * 130 * 4 > (copy // 1024 - 1) * 1024:
        with pytest.raises(bsk.BskError) as exc:   # the segments' own workspace does not fit either
            att.run(p, segments=segments)
        assert exc.value.status == 5
        return
    att.check(p, att.run(p, segments=segments))
    att.check(p, att.run(p, 100, 3, segments=segments), 100, 3)


def test_no_memory_for_the_segments(workspace_kb):
    p = ref.Problem(92, [900], [1], 2, 2, 128, 16, True)
    workspace_kb(1)
    with pytest.raises(bsk.BskError) as exc:
        att.run(p, segments=8)
    assert exc.value.status == 5 and "workspace" in str(exc.value)
    workspace_kb(0)
    att.check(p, att.run(p, segments=8))


@pytest.mark.parametrize("e4m3", [False, True])
def test_no_memory_for_segments_of_its_own_choice(workspace_kb, e4m3):
    p = ref.Problem(93, [3000], [1], 1, 2, 128, 16, e4m3)
    assert bsk.plan_kv_attention(int(e4m3), 1, 1, 1, 2, 1, 128, 3000)["segments"] > 1
    workspace_kb(1)
    att.check(p, att.run(p))


# ---------------------------------------------------------------------------
# Positions at the ends of 32 bits
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("new", [25, 200])
def test_a_window_of_any_size_beside_positions_below_zero(e4m3, new):
    """More new tokens than positions, and windows up to 2^31 - 1."""
    p = ref.Problem(81, [10, 30], [new, 5], 2, 2, 64, 16, e4m3)
    for window in (2 ** 31 - 1, 2 ** 31 - 8, 1000, 4):
        got = att.run(p, window, 0, max_len=32)
        assert not got[:new - 10].any()
        att.check(p, got, window, 0)


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("new", [1, 40])
def test_the_longest_sequence(e4m3, new):
    """2^31 - 256 positions in pages of 2^20 that all share two blocks, seen through a window with sinks."""
    page, blocks, dim, n = 2 ** 20, 2, 64, 2 ** 31 - 256
    g = torch.Generator(device="cuda").manual_seed(5)
    dt = torch.uint8 if e4m3 else torch.bfloat16
    k, v = (torch.randint(0x20, 0x40, (blocks, page, 1, dim), generator=g, device="cuda", dtype=torch.uint8) if e4m3 else
            torch.randn(blocks, page, 1, dim, generator=g, device="cuda", dtype=torch.float32).bfloat16() for _ in range(2))
    s = [torch.full((blocks, page, 1), 127, dtype=torch.uint8, device="cuda") if e4m3 else None for _ in range(2)]
    assert k.dtype == dt
    tables = (torch.arange(2048, dtype=torch.int32, device="cuda") % 2).reshape(1, -1)
    lens = torch.tensor([n], dtype=torch.int32, device="cuda")
    cu = torch.tensor([0, new], dtype=torch.int32, device="cuda")
    q = torch.randn(new, 2 * dim, generator=g, device="cuda").bfloat16()
    window, sinks = 200, 70
    def values(c, sc):
        at = torch.cat([torch.arange(sinks), torch.arange(n - new - window, n)])
        rows = ((at // page) % 2 * page + at % page).cuda()
        x = c.reshape(-1, dim)[rows]
        return at, (ref.dequantise(x.cpu(), torch.full((len(at),), 127, dtype=torch.uint8)) if e4m3 else x.cpu().double())
    at, kk = values(k, s[0])
    _, vv = values(v, s[1])
    out = torch.full((new, 2 * dim), math.nan, dtype=torch.bfloat16, device="cuda")
    bsk.chunk_attention(int(e4m3), k, v, *s, q, 2 * dim, out, 2 * dim, cu, tables, lens, 1, new, new, 2, 1, dim, page, 2048,
                        blocks, n, 1 / 8, window, sinks)
    got = out.cpu().reshape(new, 2, dim).double()
    for i in range(new):
        p = n - new + i
        seen = (at <= p) & ((at > p - window) | (at < sinks))
        for h in range(2):
            qq = q[i, h * dim:(h + 1) * dim].cpu().double()
            w = torch.softmax((kk @ qq / 8).masked_fill(~seen, -math.inf), 0)
            want, spread = w @ vv, w @ vv.abs()
            bound = ref.attention_bound(want, spread, (kk.abs() @ qq.abs()).max(), 1 / 8, dim, int(seen.sum()))
            assert ((got[i, h] - want).abs() <= bound).all(), (i, h)
