"""GPU parity of chunk_attention and decode_attention with the definition in 64
bits, within the bound of kv_reference.attention_bound.  Every place of the
cache that no token holds is NaN, and so is the output before the call."""
import math

import pytest
import torch

import kv_reference as ref
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


def run(p, window=0, sinks=0, segments=0, scale=None, decode=False, d=None, out_pad=0, max_chunk=None, max_len=None):
    d = d or p.device()
    scale = 1 / math.sqrt(p.dim) if scale is None else scale
    width = p.hq * p.dim
    buf = torch.full((p.tokens + 1, width + out_pad), math.nan, dtype=torch.bfloat16, device="cuda")
    kind = bsk.CACHE_E4M3 if p.e4m3 else bsk.CACHE_BF16
    max_len = max(p.lens) if max_len is None else max_len
    cache = (kind, d["k"], d["v"], d["ks"], d["vs"], d["fused"], p.stride, buf, width + out_pad)
    tail = (p.hq, *p.shape(), max_len, scale, window, sinks, segments)
    if decode:
        bsk.decode_attention(*cache, d["tables"], d["lens"], len(p.lens), *tail)
    else:
        chunk = max(b - a for a, b in zip(p.cu, p.cu[1:])) if max_chunk is None else max_chunk
        bsk.chunk_attention(*cache, d["cu"], d["tables"], d["lens"], len(p.lens), p.tokens, chunk, *tail)
    assert torch.isnan(buf[p.tokens]).all() and torch.isnan(buf[:, width:]).all()
    return buf[:p.tokens, :width].reshape(p.tokens, p.hq, p.dim).cpu()


def check(p, got, window=0, sinks=0, scale=None, num_blocks=None):
    scale = 1 / math.sqrt(p.dim) if scale is None else scale
    k, v = p.values()
    out, spread, reach = ref.attention(p.q, k, v, p.tables, p.cu, p.lens, p.heads, p.page, scale, window, sinks,
                                       num_blocks)
    bound = ref.attention_bound(out, spread, reach, scale, p.dim, max(p.lens))
    err = (got.double() - out).abs()
    bad = ~(err <= bound)
    assert not bad.any(), (f"{int(bad.sum())} of {bad.numel()} outputs off; first at {bad.nonzero()[0].tolist()}: "
                           f"{got[bad][0].item()} against {out[bad][0].item()}, bound {bound[bad][0].item():.3g}")


CHUNKS = [
    # lens, new, heads, group, dim, page
    ([1], [1], 1, 1, 64, 16),
    ([130], [130], 1, 1, 64, 16),
    ([300, 5, 129], [70, 5, 1], 2, 2, 128, 16),
    ([257, 128], [64, 128], 1, 4, 256, 784),
    ([200], [33], 2, 8, 64, 31),
    ([150, 0, 90], [150, 0, 17], 3, 3, 64, 7),
    ([520], [40], 1, 5, 128, 1),
    ([90, 700], [3, 6], 2, 16, 64, 64),
]


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("lens,new,heads,group,dim,page", CHUNKS)
def test_chunks(lens, new, heads, group, dim, page, e4m3):
    p = ref.Problem(11, lens, new, heads, group, dim, page, e4m3)
    check(p, run(p))


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 3), (16, 0), (100, 4), (128, 128), (37, 200), (100000, 1)])
def test_window_and_sinks(window, sinks, e4m3):
    p = ref.Problem(12, [400, 700, 50], [45, 20, 50], 2, 2, 64, 16, e4m3)
    check(p, run(p, window, sinks), window, sinks)


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("segments", [1, 2, 3, 7, 64])
def test_segments(segments, e4m3):
    p = ref.Problem(13, [900, 64, 1], [9, 30, 1], 2, 4, 128, 16, e4m3)
    check(p, run(p, segments=segments))
    check(p, run(p, 300, 5, segments=segments), 300, 5)


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("heads,group,dim,page", [(1, 1, 64, 16), (2, 8, 128, 16), (4, 4, 256, 784), (1, 6, 64, 5)])
def test_decode(heads, group, dim, page, e4m3):
    lens = [1, 1000, 0, 128, 129, 37]
    p = ref.Problem(14, lens, [1] * 6, heads, group, dim, page, e4m3)
    p.cu = list(range(7))
    got = run(p, decode=True)
    assert not got[2].any()
    check(p, got)
    check(p, run(p, 64, 2, decode=True), 64, 2)


@pytest.mark.parametrize("scale", [0.0, -0.125, 1.0, 1e-30])
def test_scales(scale):
    p = ref.Problem(15, [200], [20], 1, 2, 64, 16)
    check(p, run(p, scale=scale), scale=scale)


def test_growing_scores_move_the_running_maximum():
    """Keys whose scores rise along the sequence by far more than any exponent holds at once."""
    p = ref.Problem(16, [640], [16], 1, 4, 64, 16)
    q = torch.ones(16, 4 * 64)
    p.fused[:, :256] = q.bfloat16()
    p.q = p.fused[:, :256].reshape(16, 4, 64)
    for t in range(640):
        p.k[p.tables[0][t // 16], t % 16] = torch.full((1, 64), t / 8.0 - 40).bfloat16()
    check(p, run(p, scale=1.0), scale=1.0)
    check(p, run(p, scale=-1.0), scale=-1.0)
    check(p, run(p, scale=1.0, segments=5), scale=1.0)


@pytest.mark.parametrize("e4m3", [False, True])
def test_infinities_and_nans_stay_with_the_tokens_that_see_them(e4m3):
    """A NaN key, a NaN value and an infinite value at positions that only some queries see."""
    p = ref.Problem(17, [300], [100], 2, 2, 64, 16, e4m3)
    for t, cache, scales, x in ((290, p.k, p.ks, math.nan), (250, p.v, p.vs, math.nan), (270, p.v, p.vs, math.inf)):
        b, o = p.tables[0][t // 16], t % 16
        if e4m3:
            cache[b, o], scales[b, o] = 0x7F, 255
        else:
            cache[b, o] = x
    got = run(p, 30, 2)
    k, v = p.values()
    out, _, _ = ref.attention(p.q, k, v, p.tables, p.cu, p.lens, 2, 16, 1 / 8, 30, 2)
    assert torch.equal(torch.isfinite(got), torch.isfinite(out))
    assert torch.equal(torch.isnan(got), torch.isnan(out))
    clean = ref.Problem(17, [300], [100], 2, 2, 64, 16, e4m3)
    want = run(clean, 30, 2)
    fine = torch.isfinite(out).all(-1).all(-1)
    assert fine.any() and not fine.all()
    assert (got[fine].double() - want[fine].double()).abs().max() <= 2.0 ** -6 * want[fine].double().abs().max()


def test_scores_of_minus_infinity():
    """Keys of -inf count for nothing; where there are no others the output is zero."""
    p = ref.Problem(18, [40], [40], 1, 1, 64, 8)
    p.fused[:, :64] = 1.0
    p.q = p.fused[:, :64].reshape(40, 1, 64)
    for t in range(0, 10):
        p.k[p.tables[0][t // 8], t % 8] = -math.inf
    got = run(p)
    assert not got[:10].any()
    one = p.v[p.tables[0][10 // 8], 10 % 8].reshape(-1)
    assert torch.equal(got[10].reshape(-1), one)
    assert torch.isfinite(got).all()


@pytest.mark.parametrize("e4m3", [False, True])
def test_bad_pages(e4m3):
    p = ref.Problem(19, [100, 60], [30, 60], 2, 2, 64, 16, e4m3)
    p.tables[0][2] = -5
    p.tables[1][0] = p.num_blocks
    d = p.device()
    with pytest.raises(bsk.BskError) as exc:
        run(p, d=d)
    assert exc.value.status == 1
    d = p.device()
    width = p.hq * p.dim
    out = torch.full((p.tokens, width), math.nan, dtype=torch.bfloat16, device="cuda")
    bsk.chunk_attention_enqueue(int(e4m3), d["k"], d["v"], d["ks"], d["vs"], d["fused"], p.stride, out, width, d["cu"],
                                d["tables"], d["lens"], 2, p.tokens, 60, p.hq, *p.shape(), 100, 0.125)
    with pytest.raises(bsk.BskError):
        bsk.stream_check()
    check(p, out.reshape(p.tokens, p.hq, p.dim).cpu(), num_blocks=p.num_blocks)


def test_more_new_tokens_than_positions_see_nothing():
    """Query positions below zero give zeros, the others are as ever."""
    p = ref.Problem(20, [10, 0], [25, 4], 2, 2, 64, 16)
    got = run(p, max_len=16)
    assert not got[:15].any() and not got[25:].any()
    check(p, got)


def test_a_chunk_longer_than_promised_is_reported():
    p = ref.Problem(21, [300], [300], 1, 1, 64, 16)
    with pytest.raises(bsk.BskError) as exc:
        run(p, max_chunk=100)
    assert exc.value.status == 1 and "max_chunk" in str(exc.value)


def test_lengths_above_the_bound_count_as_the_bound():
    p = ref.Problem(22, [300], [20], 1, 2, 64, 16)
    got = run(p, max_len=200)
    p.lens = [200]
    check(p, got)


def test_strided_output_other_stream_graph_and_repeat():
    p = ref.Problem(23, [500, 220], [60, 100], 2, 4, 128, 16, True)
    want = run(p)
    assert torch.equal(run(p, out_pad=64), want)
    assert torch.equal(run(p, segments=3), run(p, segments=3))
    d = p.device()
    width = p.hq * p.dim
    out = torch.zeros(p.tokens, width, dtype=torch.bfloat16, device="cuda")
    args = (bsk.CACHE_E4M3, d["k"], d["v"], d["ks"], d["vs"], d["fused"], p.stride, out, width, d["cu"], d["tables"],
            d["lens"], 2, p.tokens, 100, p.hq, *p.shape(), 500, 1 / math.sqrt(128), 0, 0, 0)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    bsk.chunk_attention(*args, stream=side)
    assert torch.equal(out.cpu().reshape(want.shape), want)
    out.zero_()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        bsk.chunk_attention_enqueue(*args)
    out.zero_()
    g.replay()
    g.replay()
    torch.cuda.synchronize()
    bsk.stream_check()
    assert torch.equal(out.cpu().reshape(want.shape), want)


@pytest.mark.parametrize("e4m3", [False, True])
def test_append_then_attend(e4m3):
    """The calls together, as a serving step makes them: the new tokens' rows go to the cache, then are attended."""
    p = ref.Problem(24, [90, 33], [40, 1], 2, 2, 128, 16, e4m3)
    d = p.device()
    hq, h, dim = p.hq, p.heads, p.dim
    bsk.kv_cache_append_enqueue(int(e4m3), d["k"], d["v"], d["ks"], d["vs"], d["fused"][:, hq * dim:], p.stride,
                                d["fused"][:, (hq + h) * dim:], p.stride, d["cu"], d["tables"], d["lens"], 2, p.tokens,
                                *p.shape())
    got = run(p, d=d)
    for n in ("k", "v", "ks", "vs"):
        if d[n] is not None:
            setattr(p, n, d[n].cpu())
    check(p, got)


# ---------------------------------------------------------------------------
# Each kernel by itself: the automatic choice goes by the cache's type and the
# number of query rows, these tests make it.
# ---------------------------------------------------------------------------
@pytest.fixture
def kernel():
    """Sets the kernel: 1 many rows (an E4M3 cache converted tile by tile), 2 few rows."""
    yield lambda k: bsk.set_option("kv_kernel", k)
    bsk.set_option("kv_kernel", 0)


@pytest.mark.parametrize("which", [1, 2])
@pytest.mark.parametrize("lens,new,heads,group,dim,page", CHUNKS)
def test_kernels_on_a_quantised_cache(kernel, which, lens, new, heads, group, dim, page):
    p = ref.Problem(31, lens, new, heads, group, dim, page, True)
    kernel(which)
    check(p, run(p))
    check(p, run(p, 40, 3), 40, 3)
    check(p, run(p, segments=3))


@pytest.mark.parametrize("heads,group,dim,page,lens,new,window,sinks", [
    (2, 4, 256, 784, [3000], [130], 0, 0),
    (2, 2, 128, 16, [1500, 700, 2049], [128, 5, 300], 0, 0),
    (1, 8, 64, 31, [1800], [257], 0, 0),
    (2, 4, 128, 64, [2500, 300], [200, 300], 500, 7),
    (1, 4, 256, 16, [2000], [512], 0, 0),
    (1, 8, 64, 128, [4097], [600], 1024, 130),
])
@pytest.mark.parametrize("e4m3", [False, True])
def test_long_chunks(heads, group, dim, page, lens, new, window, sinks, e4m3):
    """Enough rows for the flat copy of a quantised cache, many tiles, pages that end inside tiles."""
    p = ref.Problem(32, lens, new, heads, group, dim, page, e4m3)
    k, v = p.values()
    scale = 1 / math.sqrt(dim)
    out, spread, reach = ref.attention_on_gpu(p.q, k, v, p.tables, p.cu, p.lens, heads, page, scale, window, sinks)
    bound = ref.attention_bound(out, spread, reach, scale, dim, max(lens))
    for segments in (0, 1, 4):
        got = run(p, window, sinks, segments=segments)
        bad = ~((got.double() - out).abs() <= bound)
        assert not bad.any(), (segments, int(bad.sum()), bad.nonzero()[0].tolist())


@pytest.mark.parametrize("heads,group,dim,page,lens", [
    (4, 4, 256, 784, [9000]), (2, 8, 128, 16, [5000, 17, 3001]), (1, 8, 64, 7, [6000, 6001])])
@pytest.mark.parametrize("e4m3", [False, True])
def test_long_decode(heads, group, dim, page, lens, e4m3):
    p = ref.Problem(33, lens, [1] * len(lens), heads, group, dim, page, e4m3)
    k, v = p.values()
    scale = 1 / math.sqrt(dim)
    for window, sinks in ((0, 0), (1000, 4)):
        out, spread, reach = ref.attention_on_gpu(p.q, k, v, p.tables, p.cu, p.lens, heads, page, scale, window, sinks)
        bound = ref.attention_bound(out, spread, reach, scale, dim, max(lens))
        got = run(p, window, sinks, decode=True)
        assert ((got.double() - out).abs() <= bound).all()


@pytest.mark.parametrize("which", [0, 1, 2])
@pytest.mark.parametrize("new", [4, 130])
def test_value_scales_far_apart(kernel, which, new):
    """Rows of V from 2^-60 to 2^60 in one sequence, some of them zero: each token's output to its own precision."""
    p = ref.Problem(34, [260], [new], 1, 2, 128, 16, True)
    g = torch.Generator().manual_seed(3)
    for t in range(260):
        b, o = p.tables[0][t // 16], t % 16
        x = torch.randn(1, 128, generator=g).bfloat16()
        x = x * (0.0 if t % 7 == 3 else 2.0 ** (60 - t * 120 // 259))
        p.v[b, o], p.vs[b, o] = ref.quantise(x)
    kernel(which)
    check(p, run(p))
    check(p, run(p, 3, 0), 3, 0)       # a window of rows of much the same size
    check(p, run(p, segments=2))


@pytest.mark.parametrize("which", [0, 1, 2])
def test_all_zero_and_tiny_values(kernel, which):
    p = ref.Problem(35, [200], [3], 1, 2, 64, 16, True)
    zero = torch.zeros(1, 64).bfloat16()
    for t in range(200):
        p.v[p.tables[0][t // 16], t % 16], p.vs[p.tables[0][t // 16], t % 16] = ref.quantise(zero)
    kernel(which)
    assert not run(p).any()


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("big", [2.0 ** 40, 2.0 ** -100])
def test_queries_of_any_size(e4m3, big):
    """Queries far from 1 with a scale that brings the scores back: FP16 beside E4M3 keys loses nothing."""
    p = ref.Problem(36, [150], [2], 1, 4, 64, 16, e4m3)
    p.fused[:, :256] = (p.fused[:, :256].float() * big).bfloat16()
    p.q = p.fused[:2, :256].reshape(2, 4, 64)
    check(p, run(p, scale=0.125 / big), scale=0.125 / big)


@pytest.mark.parametrize("new", [100, 300])
def test_nans_in_a_quantised_cache_stay_with_the_tokens_that_see_them(new):
    """As above, with few and with many rows (the flat copy)."""
    p = ref.Problem(37, [400], [new], 1, 4, 128, 16, True)
    for t in (390, 250):
        p.v[p.tables[0][t // 16], t % 16], p.vs[p.tables[0][t // 16], t % 16] = 0x7F, 255
    got = run(p, 40, 0)
    first = 400 - new
    seen = [any(q - 40 < t <= q for t in (390, 250)) for q in range(first, 400)]
    nan = torch.isnan(got).all(-1).all(-1)
    assert nan.tolist() == seen and torch.isfinite(got[~nan]).all()
    clean = ref.Problem(37, [400], [new], 1, 4, 128, 16, True)
    want = run(clean, 40, 0)[~nan].double()
    assert (got[~nan].double() - want).abs().max() <= 2.0 ** -6 * want.abs().max()


@pytest.mark.parametrize("e4m3", [False, True])
def test_bad_pages_under_many_rows(e4m3):
    p = ref.Problem(38, [600], [300], 1, 2, 64, 16, e4m3)
    p.tables[0][5], p.tables[0][30] = -1, p.num_blocks + 3
    d = p.device()
    with pytest.raises(bsk.BskError):
        run(p, d=d)
    out = torch.full((300, 128), math.nan, dtype=torch.bfloat16, device="cuda")
    bsk.chunk_attention_enqueue(int(e4m3), d["k"], d["v"], d["ks"], d["vs"], d["fused"], p.stride, out, 128, d["cu"],
                                d["tables"], d["lens"], 1, 300, 300, 2, *p.shape(), 600, 0.125)
    with pytest.raises(bsk.BskError):
        bsk.stream_check()
    check(p, out.reshape(300, 2, 64).cpu(), num_blocks=p.num_blocks)


def test_attention_past_32_bits():
    """A cache of over 2^31 rows' bytes: the pages at its end are read where they are."""
    heads, dim, page = 8, 256, 1024
    for kind in (bsk.CACHE_BF16, bsk.CACHE_E4M3):
        blocks = 2 ** 32 // (heads * dim * page) + 2
        dt = torch.bfloat16 if kind == bsk.CACHE_BF16 else torch.uint8
        k = torch.zeros(blocks, page, heads, dim, dtype=dt, device="cuda")
        v = torch.zeros(blocks, page, heads, dim, dtype=dt, device="cuda")
        s = [None, None] if dt == torch.bfloat16 else [torch.full((blocks, page, heads), 127, dtype=torch.uint8, device="cuda")
                                                       for _ in range(2)]
        one = 1.0 if dt == torch.bfloat16 else 0x38        # E4M3 1.0
        v[-1, :, 5] = one
        tables = torch.tensor([[blocks - 1]], dtype=torch.int32, device="cuda")
        lens = torch.tensor([page], dtype=torch.int32, device="cuda")
        for new in (1, 300):
            cu = torch.tensor([0, new], dtype=torch.int32, device="cuda")
            q = torch.randn(new, heads * dim, device="cuda").bfloat16()
            out = torch.full((new, heads * dim), math.nan, dtype=torch.bfloat16, device="cuda")
            bsk.chunk_attention(kind, k, v, *s, q, heads * dim, out, heads * dim, cu, tables, lens, 1, new, new, heads,
                                heads, dim, page, 1, blocks, page, 1 / 16)
            o = out.reshape(new, heads, dim)
            assert (o[:, 5] == 1).all() and not o[:, :5].any() and not o[:, 6:].any()


@pytest.mark.parametrize("which", [0, 1])
@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("heads,group,dim,page", [(1, 4, 64, 8), (2, 2, 128, 64), (1, 2, 256, 31), (2, 4, 128, 16)])
def test_lengths_around_a_tile_after_a_cache_of_nans(kernel, which, heads, group, dim, page, e4m3):
    """Tiles with few keys: what an earlier call left in shared memory (NaN here) is no part of them."""
    lens = [1, 15, 16, 17, 33, 63, 64, 65, 79, 127, 128, 129, 145, 193]
    new = [1, 15, 3, 17, 33, 60, 64, 2, 79, 127, 128, 120, 1, 190]
    nan = ref.Problem(41, [700], [200], heads, group, dim, page, e4m3)
    d = nan.device()
    if e4m3:
        d["ks"].fill_(255), d["vs"].fill_(255)
        d["k"].fill_(127), d["v"].fill_(127)
    else:
        d["k"].fill_(math.nan), d["v"].fill_(math.nan)
    p = ref.Problem(42, lens, new, heads, group, dim, page, e4m3)
    kernel(which)
    for window, sinks in ((0, 0), (40, 3)):
        for _ in range(3):
            assert torch.isnan(run(nan, d=d)).all()
        check(p, run(p, window, sinks), window, sinks)
