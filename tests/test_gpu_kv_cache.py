"""GPU parity of kv_cache_append and kv_cache_gather with the definitions, bit for bit."""
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


def kind(p):
    return bsk.CACHE_E4M3 if p.e4m3 else bsk.CACHE_BF16


def bits(t):
    return t.cpu().view(torch.int16) if t.dtype == torch.bfloat16 else t.cpu()


def append(p, d, cu="cu"):
    hq, h, dim = p.hq, p.heads, p.dim
    k, v = d["fused"][:, hq * dim:], d["fused"][:, (hq + h) * dim:]
    bsk.kv_cache_append(kind(p), d["k"], d["v"], d["ks"], d["vs"], k, p.stride, v, p.stride,
                        None if cu is None else d[cu], d["tables"], d["lens"], len(p.lens), p.tokens, *p.shape())


def expected(p):
    """The cache after the append."""
    k, v = p.k.clone(), p.v.clone()
    ks, vs = (None, None) if not p.e4m3 else (p.ks.clone(), p.vs.clone())
    hq, h, dim = p.hq, p.heads, p.dim
    for r, s, pos in ref.new_positions(p.cu, p.lens):
        if pos < 0:
            continue
        b, o = p.tables[s][pos // p.page], pos % p.page
        for cache, scales, at in ((k, ks, hq), (v, vs, hq + h)):
            x = p.fused[r, at * dim:(at + h) * dim].reshape(h, dim)
            if p.e4m3:
                cache[b, o], scales[b, o] = ref.quantise(x)
            else:
                cache[b, o] = x
    return k, v, ks, vs


CASES = [
    # lens, new, heads, dim, page
    ([1], [1], 1, 64, 8), ([5, 40, 17], [5, 1, 16], 2, 64, 16), ([33, 64], [32, 33], 3, 128, 31),
    ([100], [100], 4, 256, 784), ([9, 0, 3], [2, 0, 3], 5, 64, 1), ([20, 30], [0, 25], 1, 256, 7),
]


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("lens,new,heads,dim,page", CASES)
def test_append(lens, new, heads, dim, page, e4m3):
    p = ref.Problem(1, lens, new, heads=heads, dim=dim, page=page, e4m3=e4m3)
    d = p.device()
    append(p, d)
    for name, want in zip(("k", "v", "ks", "vs"), expected(p)):
        if want is not None:
            assert torch.equal(bits(d[name]), bits(want)), name


@pytest.mark.parametrize("e4m3", [False, True])
def test_append_one_token_per_sequence(e4m3):
    """cu_tokens NULL; more sequences than a warp has lanes."""
    lens = [1 + (7 * i) % 50 for i in range(77)]
    p = ref.Problem(2, lens, [1] * 77, heads=2, dim=128, page=16, e4m3=e4m3)
    d = p.device()
    append(p, d, cu=None)
    for name, want in zip(("k", "v", "ks", "vs"), expected(p)):
        if want is not None:
            assert torch.equal(bits(d[name]), bits(want)), name


def test_many_sequences_find_their_tokens():
    """Over 32 x 32 sequences, many of them without new tokens."""
    new = [(i * 5) % 3 for i in range(1100)]
    lens = [n + i % 4 for i, n in enumerate(new)]
    p = ref.Problem(3, lens, new, heads=1, dim=64, page=4)
    d = p.device()
    append(p, d)
    k, v, _, _ = expected(p)
    assert torch.equal(bits(d["k"]), bits(k)) and torch.equal(bits(d["v"]), bits(v))


def test_quantisation_of_special_rows():
    """Zeros, subnormals, the largest values, exact ties, a border of the scale, Inf and NaN."""
    dim = 64
    rows = torch.zeros(10, dim)
    rows[1, 3] = 2.0 ** -133                        # BF16's least subnormal
    rows[2] = torch.finfo(torch.bfloat16).max
    rows[3] = torch.linspace(-448, 448, dim)
    rows[4, :6] = torch.tensor([448.0, 17.0, 19.0, -21.0, 2.0 ** -10, 3 * 2.0 ** -10])   # ties
    rows[5, :2] = torch.tensor([450.0, 1.0])        # just over 448: one scale up
    rows[6, 5] = math.inf
    rows[7, 63] = math.nan
    rows[8] = -(2.0 ** -126)
    rows[9, 0] = -0.0
    p = ref.Problem(4, [10], [10], heads=1, group=1, dim=dim, page=16, e4m3=True)
    p.fused[:, dim:2 * dim] = rows.bfloat16()
    p.fused[:, 2 * dim:] = rows.flip(0).bfloat16()
    d = p.device()
    append(p, d)
    for name, want in zip(("k", "v", "ks", "vs"), expected(p)):
        assert torch.equal(bits(d[name]), bits(want)), name
    out = [torch.empty(10, 1, dim, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    bsk.kv_cache_gather(kind(p), d["k"], d["v"], d["ks"], d["vs"], *out, d["cu"], d["tables"], d["lens"], 1, 10,
                        *p.shape())
    back = out[0].cpu().double().reshape(10, dim)
    x = rows.bfloat16().double()
    assert torch.isnan(back[6:8]).all() and torch.equal(back[0], x[0])
    fine = torch.tensor([1, 2, 3, 4, 5, 8, 9])
    top = x[fine].abs().amax(-1, keepdim=True)
    # half a step of E4M3 (2^-4), or half of its least step under the row's scale
    assert ((back - x)[fine].abs() <= torch.maximum(x[fine].abs() * 2.0 ** -4, top * 2.0 ** -17 + 2.0 ** -127)).all()


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("lens,new,heads,dim,page", CASES)
def test_gather(lens, new, heads, dim, page, e4m3):
    p = ref.Problem(5, lens, new, heads=heads, dim=dim, page=page, e4m3=e4m3)
    d = p.device()
    out = [torch.full((p.tokens, heads, dim), math.nan, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    bsk.kv_cache_gather(kind(p), d["k"], d["v"], d["ks"], d["vs"], *out, d["cu"], d["tables"], d["lens"], len(lens),
                        p.tokens, *p.shape())
    k, v = p.values()
    for r, s, pos in ref.new_positions(p.cu, p.lens):
        for got, want in ((out[0], k), (out[1], v)):
            w = want[p.tables[s][pos // page], pos % page] if pos >= 0 else torch.zeros(heads, dim, dtype=torch.float64)
            assert torch.equal(got[r].cpu().double(), w)


def test_bad_pages_are_skipped_and_reported():
    p = ref.Problem(6, [40], [40], heads=2, dim=64, page=16, e4m3=True)
    p.tables[0][1] = p.num_blocks + 7
    d = p.device()
    before = d["k"].clone()
    with pytest.raises(bsk.BskError) as exc:
        append(p, d)
    assert exc.value.status == 1
    changed = (d["k"] != before).any(-1).any(-1).cpu()
    places = {(p.tables[0][t // 16], t % 16) for t in range(40) if t // 16 != 1}
    assert {(i, j) for i, j in changed.nonzero().tolist()} <= places
    out = [torch.empty(40, 2, 64, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    with pytest.raises(bsk.BskError):
        bsk.kv_cache_gather(kind(p), d["k"], d["v"], d["ks"], d["vs"], *out, d["cu"], d["tables"], d["lens"], 1, 40,
                            *p.shape())
    assert not out[0][16:32].any() and out[0][:16].any()
    # a table that is too short for the length, and more new tokens than the sequence is long
    q = ref.Problem(7, [20], [20], heads=1, dim=64, page=16)
    d = q.device()
    d["lens"] += 100
    with pytest.raises(bsk.BskError):
        append(q, d)
    q = ref.Problem(8, [20], [25], heads=1, dim=64, page=16)
    d = q.device()
    append(q, d)
    k, v, _, _ = expected(q)
    assert torch.equal(bits(d["k"]), bits(k)) and torch.equal(bits(d["v"]), bits(v))


def test_rows_outside_every_sequence_are_left_alone():
    """num_tokens above cu_tokens' end; the library keeps the rest of the output."""
    p = ref.Problem(9, [8, 8], [3, 4], heads=2, dim=64, page=8)
    d = p.device()
    out = [torch.full((12, 2, 64), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    bsk.kv_cache_gather(kind(p), d["k"], d["v"], None, None, *out, d["cu"], d["tables"], d["lens"], 2, 12, *p.shape())
    assert (out[0][7:] == 7).all() and (out[1][7:] == 7).all()


def test_place_past_32_bits():
    """A cache of more than 2^32 elements: the last block is written and read back."""
    heads, dim, page = 8, 256, 1024
    blocks = 2 ** 32 // (heads * dim * page) + 2
    cache = [torch.zeros(blocks, page, heads, dim, dtype=torch.uint8, device="cuda") for _ in range(2)]
    scales = [torch.zeros(blocks, page, heads, dtype=torch.uint8, device="cuda") for _ in range(2)]
    x = torch.randn(2, heads, dim, device="cuda").bfloat16()
    tables = torch.tensor([[blocks - 1]], dtype=torch.int32, device="cuda")
    lens = torch.tensor([page], dtype=torch.int32, device="cuda")
    args = (None, tables, lens, 1, 1, heads, dim, page, 1, blocks)
    bsk.kv_cache_append(bsk.CACHE_E4M3, *cache, *scales, x[0], heads * dim, x[1], heads * dim, *args)
    out = [torch.empty(1, heads, dim, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    bsk.kv_cache_gather(bsk.CACHE_E4M3, *cache, *scales, *out, *args)
    for i in range(2):
        codes, byte = ref.quantise(x[i].cpu())
        assert torch.equal(cache[i][-1, -1].cpu(), codes) and torch.equal(scales[i][-1, -1].cpu(), byte)
        assert torch.equal(out[i][0].cpu().double(), ref.dequantise(codes, byte))
        assert not cache[i][:-1].any()
