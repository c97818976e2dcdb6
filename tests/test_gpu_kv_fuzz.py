"""Attention over the paged cache on seeded random problems (shapes, pages,
lengths, chunks, windows, sinks, segments, kernels, scales of keys and values
near and far apart), against the definition in 64 bits.  The bound is that of
kv_reference.attention_bound and, for FP16 weights beside E4M3 values, 2^-32
of a row's largest weight for each visible value."""
import math
import random

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
    bsk.set_option("kv_kernel", 0)


def e4m3_rows(g, shape, low, high, zeros):
    """Random codes with scale exponents low .. high, a part of the rows all zeros; their values."""
    codes = torch.randint(0, 256, shape, generator=g, device="cuda", dtype=torch.uint8)
    codes[(codes & 127) == 127] = 0                     # NaN
    scales = (127 + torch.randint(low, high + 1, shape[:-1], generator=g, device="cuda")).clamp(10, 247).to(torch.uint8)
    none = torch.rand(shape[:-1], generator=g, device="cuda") < zeros
    codes[none], scales[none] = 0, 10
    values = ref.e4m3_values().cuda()[codes.long()] * 2.0 ** (scales.double() - 127).unsqueeze(-1)
    return codes, scales, values


@pytest.mark.parametrize("e4m3", [True, False])
@pytest.mark.parametrize("seed", range(20))
def test_random_problems(request, seed, e4m3):
    rng = random.Random(request.node.name)
    g = torch.Generator(device="cuda").manual_seed(rng.randrange(2 ** 31))
    for _ in range(4):
        dim, heads, group = rng.choice((64, 128, 256)), rng.choice((1, 2, 3)), rng.choice((1, 2, 4, 5, 8))
        page, n, hq = rng.choice((1, 7, 16, 31, 64, 784)), rng.choice((1, 2, 3)), heads * group
        lens = [rng.choice((0, 1, 5, 63, 64, 65, 200, 700, 2500)) + rng.randint(0, 40) for _ in range(n)]
        new = [rng.choice((0, 1, 1, 2, 5, 30, 130, 300)) for _ in range(n)]
        new[0] = max(new[0], 1)
        cu = [rng.choice((0, 0, 3))]
        for x in new:
            cu.append(cu[-1] + x)
        tokens, most = cu[-1] + rng.choice((0, 2)), max(1, max(-(-x // page) for x in lens))
        blocks = sum(-(-x // page) for x in lens) + 2
        order = torch.randperm(blocks, generator=g, device="cuda").int()
        tables, at = torch.full((n, most), -1, dtype=torch.int32, device="cuda"), 0
        for s, x in enumerate(lens):
            tables[s, :-(-x // page)] = order[at:at - (-x // page)]
            at -= -x // page
        shape, ke = (blocks, page, heads, dim), 0
        if e4m3:
            middle, spread, zeros = rng.choice(((0, 2, 0.05), (-20, 18, 0.05), (60, 60, 0.05), (0, 3, 0.3), (-117, 0, 0.1)))
            ke = rng.choice((0, 0, -60, 60, 105))
            k, ks, kv = e4m3_rows(g, shape, ke - rng.choice((2, 12)), ke, 0.0)
            v, vs, vv = e4m3_rows(g, shape, middle - spread, middle, zeros)
        else:
            k, v = (torch.randn(shape, generator=g, device="cuda").bfloat16() for _ in range(2))
            ks = vs = None
            kv, vv = k.double(), v.double()
        q = (torch.randn(tokens, hq * dim, generator=g, device="cuda") * 2.0 ** (-ke - 8 if e4m3 else 0)).bfloat16()
        if rng.random() < 0.2:
            q[cu[0]] = 0
        scale = rng.choice((1.0, 1.0, -1.0, 0.1, 0.0)) / math.sqrt(dim)
        window, sinks = rng.choice((0, 0, 1, 7, 64, 300, 2 ** 31 - 1)), rng.choice((0, 0, 1, 5, 80))
        out = torch.full((tokens, hq * dim), 7.0, dtype=torch.bfloat16, device="cuda")
        bsk.set_option("kv_kernel", rng.choice((0, 0, 1, 2)))
        bsk.chunk_attention(int(e4m3), k, v, ks, vs, q, hq * dim, out, hq * dim, torch.tensor(cu, dtype=torch.int32, device="cuda"),
                            tables, torch.tensor(lens, dtype=torch.int32, device="cuda"), n, tokens,
                            rng.choice((max(new), tokens + 5, 2 ** 31 - 1)), hq, heads, dim, page, most, blocks, max(lens),
                            scale, window, sinks, rng.choice((0, 0, 1, 2, 5, 33)))
        assert (out[:cu[0]] == 7).all() and (out[cu[-1]:] == 7).all()
        kv, vv = kv.reshape(-1, heads, dim), vv.reshape(-1, heads, dim)
        for s in range(n):
            t = torch.arange(lens[s], device="cuda")
            p = torch.arange(lens[s] - new[s], lens[s], device="cuda")[:, None]
            rows = tables[s][t // page].long() * page + t % page
            seen = (t <= p) & ((t > p - window) | (t < sinks)) if window else t <= p
            for h in range(hq):
                got = out[cu[s]:cu[s + 1], h * dim:(h + 1) * dim].double()
                if lens[s] == 0:
                    assert not got.any()
                    continue
                x = q[cu[s]:cu[s + 1], h * dim:(h + 1) * dim].double()
                keys, values = kv[rows, h // group], vv[rows, h // group]
                w = torch.softmax((x @ keys.T * scale).masked_fill(~seen, -math.inf), -1)
                w[~seen.any(-1)] = 0
                want, spread = w @ values, w @ values.abs()
                reach = (x.abs() @ keys.abs().T).masked_fill(~seen, 0).amax(-1)
                bound = ref.attention_bound(want, spread, reach, scale, dim, lens[s])
                if e4m3:
                    bound = bound + 2.0 ** -32 * w.amax(-1, keepdim=True) * (seen.double() @ values.abs())
                bad = ~((got - want).abs() <= bound)
                assert not bad.any(), (s, h, int(bad.sum()), bad.nonzero()[0].tolist(), dict(
                    dim=dim, heads=heads, group=group, page=page, lens=lens, new=new, scale=scale, window=window, sinks=sinks))
