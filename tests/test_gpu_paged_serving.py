"""The example examples/paged_serving.py: its calls together, at different chunk
sizes, against the definition on the keys and values that the cache holds."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    from bf16_gemm_skinny_gb300 import build

    build.build()
    torch.cuda.init()
    spec = importlib.util.spec_from_file_location("paged_serving", os.path.join(ROOT, "examples", "paged_serving.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_chunk_sizes_agree_with_the_definition(example):
    """Each chunk size's outputs are those of softmax attention in 64 bits over what was cached.  A weight is
    rounded to 16 bits (2^-8 at the worst), the output once (2^-9 relative), scores in FP32: 2^-7 of the values'
    weighted magnitudes covers them."""
    for chunk in (64, 300, 1000):
        layer, outs = example.serve(chunk)
        for r, out in enumerate(outs):
            k, v = (t.double() for t in layer.cached(r))
            n = k.shape[0]
            g = torch.Generator(device="cuda").manual_seed(1)
            x = [torch.randn(m, example.WIDTH, generator=g, device="cuda").bfloat16() for m in (720, 353)][r]
            qkv = torch.empty(n, layer.rows, dtype=torch.bfloat16, device="cuda")
            example.bsk.gemv_bf16(layer.w, x, qkv, layer.rows, example.WIDTH, n)
            q = qkv[:, :example.HQ * example.DIM].view(n, example.HQ, example.DIM).double()
            t = torch.arange(n, device="cuda")
            p = t[:, None]
            seen = (t <= p) & ((t > p - example.WINDOW) | (t < example.SINKS))
            for h in range(example.HQ):
                j = h // example.GROUP
                s = (q[:, h] @ k[:, j].T * example.DIM ** -0.5).masked_fill(~seen, -torch.inf)
                w = torch.softmax(s, -1)
                # gemv_bf16 sums in another order for another number of tokens: q may differ by one BF16 step,
                # which moves a weight by up to 2^-8 of its score's terms
                reach = (q[:, h].abs() @ k[:, j].abs().T * example.DIM ** -0.5).masked_fill(~seen, 0).amax(-1, keepdim=True)
                bound = (w @ v[:, j].abs()) * (2.0 ** -7 + 2 * 2.0 ** -8 * reach)
                assert ((out[:, h].double() - w @ v[:, j]).abs() <= bound + 1e-30).all(), (chunk, r, h)


def test_cache_holds_the_projections(example):
    """What is read back is the projected keys to within half a step of E4M3."""
    layer, _ = example.serve(200, prompts=(150, 90), steps=3)
    k, _ = layer.cached(1)
    assert k.shape[0] == 93 and torch.isfinite(k).all() and k.abs().amax() > 0
