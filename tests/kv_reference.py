"""The paged cache and the attention over it in 64 bits, for the parity tests:
plain loops over sequences and positions, written from the definitions in
include/bsk.h, on CPU tensors."""
from __future__ import annotations

import math

import torch

import oracle


def e4m3_values() -> torch.Tensor:
    """The 256 values of the E4M3 codes (NaN for 0x7F and 0xFF)."""
    return torch.from_numpy(oracle.fp8_decode(torch.arange(256, dtype=torch.uint8).numpy(), "e4m3")).double()


def quantise(x: torch.Tensor):
    """Rows of BF16 values -> (codes, scale bytes), by search: the least exponent
    whose scale covers the row, then the nearest code (ties to the even one)."""
    table = e4m3_values()[:127]                       # 0 .. 448, ascending
    rows = x.double().reshape(-1, x.shape[-1])
    codes = torch.empty(rows.shape, dtype=torch.uint8)
    scales = torch.empty(rows.shape[0], dtype=torch.uint8)
    for i, r in enumerate(rows):
        if not torch.isfinite(r).all():
            codes[i], scales[i] = 0x7F, 255
            continue
        top, e = r.abs().max().item(), -117
        while top > 448.0 * 2.0 ** e:
            e += 1
        scales[i] = e + 127
        y = r.abs() * 2.0 ** -e
        hi = torch.searchsorted(table, y).clamp(max=126)
        lo = (hi - 1).clamp(min=0)
        d = (y - table[lo]) - (table[hi] - y)
        if e == 120:                                   # 256 * 2^120 is no BF16 value
            lo, hi = lo.clamp(max=119), hi.clamp(max=119)
        code = torch.where(d < 0, lo, torch.where(d > 0, hi, torch.where(lo % 2 == 0, lo, hi)))
        codes[i] = (code + 128 * torch.signbit(r)).to(torch.uint8)
    return codes.reshape(x.shape), scales.reshape(x.shape[:-1])


def dequantise(codes: torch.Tensor, scales: torch.Tensor) -> torch.Tensor:
    s = torch.where(scales == 255, torch.tensor(math.nan, dtype=torch.float64), 2.0 ** (scales.double() - 127))
    return e4m3_values()[codes.long()] * s.unsqueeze(-1)


def new_positions(cu, lens):
    """(row, sequence, position) of every new token."""
    for s in range(len(lens)):
        n = cu[s + 1] - cu[s]
        for i in range(n):
            yield cu[s] + i, s, lens[s] - n + i


def attention(q, k, v, tables, cu, lens, heads, page, scale, window=0, sinks=0, num_blocks=None):
    """q [T, Hq, D]; k, v [blocks, page, heads, D] (values, 64 bits).  Returns (out, spread, reach): the
    output, sum_j w_j |v_j| per element, and per (token, head) the largest sum_d |q_d k_jd| of its keys."""
    T, hq, D = q.shape
    out = torch.zeros(T, hq, D, dtype=torch.float64)
    spread = torch.zeros_like(out)
    reach = torch.zeros(T, hq, dtype=torch.float64)
    q = q.double()
    rows = {}
    for s in range(len(lens)):
        rows[s] = [(t, tables[s][t // page] * page + t % page) for t in range(max(lens[s], 0))
                   if num_blocks is None or 0 <= tables[s][t // page] < num_blocks]
    flat_k, flat_v = k.reshape(-1, heads, D), v.reshape(-1, heads, D)
    for r, s, p in new_positions(cu, lens):
        at = [i for t, i in rows[s] if t <= p and (window == 0 or t > p - window or t < sinks)]
        if not at:
            continue
        at = torch.tensor(at)
        for h in range(hq):
            j = h // (hq // heads)
            x = (flat_k[at, j] @ q[r, h]) * scale
            w = torch.exp(x - x.max())
            w = w / w.sum()
            out[r, h] = w @ flat_v[at, j]
            spread[r, h] = w @ flat_v[at, j].abs()
            reach[r, h] = (flat_k[at, j].abs() @ q[r, h].abs()).max()
    return out, spread, reach


def bf16_half_step(x: torch.Tensor) -> torch.Tensor:
    """Half the distance of BF16 values around |x|."""
    e = torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -126)))
    return 2.0 ** (e - 8)


def attention_bound(out, spread, reach, scale, dim, count):
    """How far the kernels' output may be from the exact one:
    each score is a sum of `dim` exact products in FP32 whose additions need not
    round to nearest (2^-23 of the magnitudes' sum each) and is scaled once
    (2^-24); with 2^-21 for exp2 that moves a weight by eps relatively, numerator
    and denominator alike; the weight is rounded to BF16 (2^-9 of itself, half a
    step being 2^-9 of the value above it: 2^-8 counts the worst place in the
    binade), the sums over `count` tokens add 2^-23 each, and the output is
    rounded once."""
    eps = (dim * 2.0 ** -23 + 2.0 ** -23) * abs(scale) * reach.unsqueeze(-1) * 1.01 + 2.0 ** -21
    return spread * (2.0 ** -8 + 2 * eps + count * 2.0 ** -22) + bf16_half_step(out.abs() + spread * 2.0 ** -8)


class Problem:
    """A random paged cache with shuffled blocks, the new tokens' q, k and v side
    by side in one array, and NaN in every place of the cache that no token
    holds."""

    def __init__(self, seed, lens, new, heads=2, group=2, dim=64, page=16, e4m3=False, spare=3, fill=math.nan):
        g = torch.Generator().manual_seed(seed)
        self.lens, self.heads, self.group, self.dim, self.page, self.e4m3 = list(lens), heads, group, dim, page, e4m3
        self.hq = heads * group
        self.cu = [0]
        for n in new:
            self.cu.append(self.cu[-1] + n)
        self.tokens = self.cu[-1]
        need = [-(-max(n, 0) // page) for n in lens]
        self.max_blocks = max(1, max(need))
        self.num_blocks = sum(need) + spare
        order = torch.randperm(self.num_blocks, generator=g).tolist()
        self.tables = [[-1] * self.max_blocks for _ in lens]
        at = 0
        for s, n in enumerate(need):
            self.tables[s][:n] = order[at:at + n]
            at += n
        shape = (self.num_blocks, page, heads, dim)
        size = 2.0 ** torch.randint(-3, 4, (dim,), generator=g).double()
        k = (torch.randn(shape, generator=g) * size.clamp(max=1).float()).bfloat16()
        v = (torch.randn(shape, generator=g) * size.float()).bfloat16()
        self.fused = torch.randn(max(1, self.tokens), (self.hq + 2 * heads) * dim, generator=g).bfloat16()
        self.stride = self.fused.shape[1]
        self.q = self.fused[:self.tokens, :self.hq * dim].reshape(self.tokens, self.hq, dim)
        used = torch.zeros(self.num_blocks * page, dtype=torch.bool)
        for s, n in enumerate(lens):
            for t in range(n):
                used[self.tables[s][t // page] * page + t % page] = True
        self.used = used.reshape(self.num_blocks, page)
        if e4m3:
            self.k, self.ks = quantise(k)
            self.v, self.vs = quantise(v)
            if math.isnan(fill):
                for c, s in ((self.k, self.ks), (self.v, self.vs)):
                    c[~self.used], s[~self.used] = 0x7F, 255
        else:
            self.k, self.v, self.ks, self.vs = k, v, None, None
            k[~self.used] = fill
            v[~self.used] = fill

    def values(self):
        if self.e4m3:
            return dequantise(self.k, self.ks), dequantise(self.v, self.vs)
        return self.k.double(), self.v.double()

    def device(self):
        """The tensors on the GPU, as the calls take them."""
        d = {n: (None if getattr(self, n) is None else getattr(self, n).cuda().contiguous())
             for n in ("k", "v", "ks", "vs", "fused")}
        d["tables"] = torch.tensor(self.tables, dtype=torch.int32).cuda()
        d["lens"] = torch.tensor(self.lens, dtype=torch.int32).cuda()
        d["cu"] = torch.tensor(self.cu, dtype=torch.int32).cuda()
        return d

    def shape(self):
        return self.heads, self.dim, self.page, self.max_blocks, self.num_blocks


def attention_on_gpu(q, k, v, tables, cu, lens, heads, page, scale, window=0, sinks=0):
    """attention() for long sequences: the same definition in 64 bits, by whole sequences on the GPU.
    Every page is good and every query position exists."""
    T, hq, D = q.shape
    out = torch.zeros(T, hq, D, dtype=torch.float64, device="cuda")
    spread, reach = torch.zeros_like(out), torch.zeros(T, hq, dtype=torch.float64, device="cuda")
    q, k, v = q.cuda().double(), k.cuda().reshape(-1, heads, D), v.cuda().reshape(-1, heads, D)
    for s, n in enumerate(lens):
        a, b = cu[s], cu[s + 1]
        if a == b:
            continue
        at = torch.tensor([tables[s][t // page] * page + t % page for t in range(n)], device="cuda")
        t = torch.arange(n, device="cuda")
        p = torch.arange(n - (b - a), n, device="cuda")[:, None]
        seen = t <= p
        if window:
            seen &= (t > p - window) | (t < sinks)
        for h in range(hq):
            kk, vv = k[at, h // (hq // heads)], v[at, h // (hq // heads)]
            x = (q[a:b, h] @ kk.T * scale).masked_fill(~seen, -math.inf)
            w = torch.softmax(x, -1)
            out[a:b, h], spread[a:b, h] = w @ vv, w @ vv.abs()
            reach[a:b, h] = (q[a:b, h].abs() @ kk.abs().T).masked_fill(~seen, 0).amax(-1)
    return out.cpu(), spread.cpu(), reach.cpu()
