"""One attention layer served over a paged, quantised KV cache: two requests'
prompts come in chunks, then both decode token by token.

Every step is three kinds of calls, in stream order and without a host
synchronisation between them: the fused q, k, v projection (gemv_bf16), the new
tokens' keys and values into their pages (kv_cache_append, quantised to E4M3 as
they are written), and attention over everything cached (chunk_attention for
prompts, decode_attention for single tokens), here with a sliding window and
four sink tokens.  Random weights stand for a model's.

    python examples/paged_serving.py
"""
import os
import sys

import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), ".."))
import bf16_gemm_skinny_gb300 as bsk  # noqa: E402

HEADS, GROUP, DIM, PAGE, WIDTH = 4, 4, 128, 64, 1024     # KV heads, query heads each, head and page size, model width
HQ = HEADS * GROUP
WINDOW, SINKS = 256, 4


class Layer:
    def __init__(self, requests: int, max_len: int, seed: int = 0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.rows = (HQ + 2 * HEADS) * DIM
        self.w = (0.05 * torch.randn(self.rows, WIDTH, generator=g, device="cuda")).bfloat16()
        self.per_seq = -(-max_len // PAGE)
        self.blocks = requests * self.per_seq
        shape = (self.blocks, PAGE, HEADS)
        self.k, self.v = (torch.zeros(*shape, DIM, dtype=torch.uint8, device="cuda") for _ in range(2))
        self.ks, self.vs = (torch.zeros(*shape, dtype=torch.uint8, device="cuda") for _ in range(2))
        self.tables = torch.randperm(self.blocks, generator=g, device="cuda").to(torch.int32).view(requests, -1)
        self.lens = torch.zeros(requests, dtype=torch.int32, device="cuda")
        self.max_len, self.requests = max_len, requests

    def __call__(self, x: torch.Tensor, new: list[int]) -> torch.Tensor:
        """x: the new tokens' [sum(new), WIDTH] BF16, request by request; returns [sum(new), HQ, DIM]."""
        tokens = x.shape[0]
        qkv = torch.empty(tokens, self.rows, dtype=torch.bfloat16, device="cuda")
        bsk.gemv_bf16_enqueue(self.w, x, qkv, self.rows, WIDTH, tokens)
        decode = all(n == 1 for n in new)
        cu = None if decode else torch.tensor([sum(new[:i]) for i in range(len(new) + 1)], dtype=torch.int32, device="cuda")
        self.lens += torch.tensor(new, dtype=torch.int32, device="cuda")
        cache = (bsk.CACHE_E4M3, self.k, self.v, self.ks, self.vs)
        shape = (HEADS, DIM, PAGE, self.per_seq, self.blocks)
        bsk.kv_cache_append_enqueue(*cache, qkv[:, HQ * DIM:], self.rows, qkv[:, (HQ + HEADS) * DIM:], self.rows, cu,
                                    self.tables, self.lens, self.requests, tokens, *shape)
        out = torch.empty(tokens, HQ, DIM, dtype=torch.bfloat16, device="cuda")
        rest = (HQ, *shape, self.max_len, DIM ** -0.5, WINDOW, SINKS)
        if decode:
            bsk.decode_attention_enqueue(*cache, qkv, self.rows, out, HQ * DIM, self.tables, self.lens, self.requests, *rest)
        else:
            bsk.chunk_attention_enqueue(*cache, qkv, self.rows, out, HQ * DIM, cu, self.tables, self.lens, self.requests,
                                        tokens, max(new), *rest)
        return out

    def cached(self, request: int) -> list[torch.Tensor]:
        """A request's cached keys and values, as BF16 [length, HEADS, DIM]."""
        n = int(self.lens[request])
        out = [torch.empty(n, HEADS, DIM, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
        cu = torch.tensor([0, n], dtype=torch.int32, device="cuda")
        bsk.kv_cache_gather(bsk.CACHE_E4M3, self.k, self.v, self.ks, self.vs, *out, cu, self.tables[request:request + 1],
                            self.lens[request:request + 1], 1, n, HEADS, DIM, PAGE, self.per_seq, self.blocks)
        return out


def serve(chunk: int, prompts=(700, 333), steps: int = 20, seed: int = 0):
    """Both prompts in chunks of `chunk` tokens, then `steps` tokens each; the outputs of every token by request."""
    g = torch.Generator(device="cuda").manual_seed(seed + 1)
    x = [torch.randn(n + steps, WIDTH, generator=g, device="cuda").bfloat16() for n in prompts]
    layer, at, out = Layer(len(prompts), max(prompts) + steps, seed), [0] * len(prompts), [[] for _ in prompts]
    while any(a < n for a, n in zip(at, prompts)):
        new = [min(chunk, n - a) for a, n in zip(at, prompts)]
        y = layer(torch.cat([t[a:a + n] for t, a, n in zip(x, at, new)]), new)
        for i, part in enumerate(y.split(new)):
            out[i].append(part)
        at = [a + n for a, n in zip(at, new)]
    for _ in range(steps):
        y = layer(torch.stack([t[a] for t, a in zip(x, at)]), [1] * len(prompts))
        for i, part in enumerate(y.split(1)):
            out[i].append(part)
        at = [a + 1 for a in at]
    bsk.stream_check()
    return layer, [torch.cat(o) for o in out]


if __name__ == "__main__":
    layer, outs = serve(256)
    for i, o in enumerate(outs):
        k, _ = layer.cached(i)
        print(f"request {i}: {o.shape[0]} tokens, {k.shape[0]} cached, last output's norm {o[-1].float().norm():.4f}")
