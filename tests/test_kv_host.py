"""Refusals of the paged-cache calls: every bad argument is turned down with
BSK_ERR_INVALID_ARG before a device is touched (no GPU needed)."""
import pytest

from bf16_gemm_skinny_gb300 import _native as bsk
from bf16_gemm_skinny_gb300 import build as bsk_build

A = 1 << 20   # stands for a device address; nothing is read from it


@pytest.fixture(scope="module", autouse=True)
def lib():
    bsk_build.build()
    return bsk.load()


CACHE = dict(cache_type=0, k_cache=A, v_cache=64 * A, k_scales=None, v_scales=None)
BATCH = dict(cu_tokens=A, block_tables=A, seq_lens=A, num_seqs=2, num_tokens=10)
SHAPE = dict(num_kv_heads=2, head_dim=64, block_size=16, max_blocks=4, num_blocks=8)
APPEND = {**CACHE, "k": 128 * A, "k_stride": 128, "v": 192 * A, "v_stride": 128, **BATCH, **SHAPE}
GATHER = {**CACHE, "k_out": 128 * A, "v_out": 192 * A, **BATCH, **SHAPE}
CHUNK = {**CACHE, "q": 128 * A, "q_stride": 512, "out": 192 * A, "out_stride": 256, **BATCH, "max_chunk": 8,
         "num_q_heads": 4, **SHAPE, "max_seq_len": 64, "softmax_scale": 0.125, "window": 0, "sinks": 0}
DECODE = {k: v for k, v in CHUNK.items() if k not in ("cu_tokens", "num_tokens", "max_chunk")}

COMMON = [
    dict(cache_type=2), dict(cache_type=-1), dict(num_seqs=-1), dict(num_kv_heads=0), dict(head_dim=96),
    dict(block_size=0), dict(max_blocks=0), dict(num_blocks=-3), dict(k_cache=None), dict(v_cache=A + 8),
    dict(block_tables=None), dict(seq_lens=None), dict(cache_type=1), dict(k_scales=A),
    dict(num_blocks=1 << 20, block_size=1 << 20),
]


def refused(fn, base, change):
    with pytest.raises(bsk.BskError) as exc:
        fn(**{**base, **change}, stream=0)
    assert exc.value.status == 1, str(exc.value)
    assert bsk.last_error()


@pytest.mark.parametrize("change", COMMON + [
    dict(num_tokens=-1), dict(k=None), dict(v=None), dict(k=128 * A + 2), dict(k_stride=120), dict(v_stride=132),
    dict(cu_tokens=None), dict(k=A), dict(v_cache=A)])
@pytest.mark.parametrize("form", ["", "_enqueue"])
def test_append(change, form):
    refused(getattr(bsk, "kv_cache_append" + form), APPEND, change)


@pytest.mark.parametrize("change", COMMON + [
    dict(num_tokens=-1), dict(k_out=None), dict(v_out=192 * A + 8), dict(v_out=128 * A), dict(k_out=A),
    dict(cu_tokens=None)])
@pytest.mark.parametrize("form", ["", "_enqueue"])
def test_gather(change, form):
    refused(getattr(bsk, "kv_cache_gather" + form), GATHER, change)


ATTENTION = COMMON + [
    dict(num_q_heads=3), dict(num_q_heads=0), dict(q=None), dict(out=None), dict(q=128 * A + 4), dict(q_stride=248),
    dict(out_stride=260), dict(max_seq_len=65), dict(max_seq_len=-1), dict(softmax_scale=float("nan")),
    dict(softmax_scale=float("inf")), dict(window=-1), dict(sinks=-1), dict(num_segments=-1), dict(num_segments=257),
    dict(out=A), dict(out=128 * A)]


@pytest.mark.parametrize("change", ATTENTION + [dict(num_tokens=-1), dict(max_chunk=0), dict(cu_tokens=None)])
@pytest.mark.parametrize("form", ["", "_enqueue"])
def test_chunk_attention(change, form):
    refused(getattr(bsk, "chunk_attention" + form), CHUNK, change)


@pytest.mark.parametrize("change", ATTENTION)
@pytest.mark.parametrize("form", ["", "_enqueue"])
def test_decode_attention(change, form):
    refused(getattr(bsk, "decode_attention" + form), DECODE, change)


def test_nothing_to_do_is_no_error():
    """No sequences or no tokens: accepted before any pointer is looked at."""
    none = dict(k_cache=None, v_cache=None, block_tables=None, seq_lens=None)
    bsk.kv_cache_append(**{**APPEND, **none, "num_tokens": 0}, stream=0)
    bsk.kv_cache_gather(**{**GATHER, **none, "num_seqs": 0}, stream=0)
    bsk.chunk_attention(**{**CHUNK, **none, "num_tokens": 0, "q": None, "out": None}, stream=0)
    bsk.decode_attention(**{**DECODE, **none, "num_seqs": 0, "q": None, "out": None}, stream=0)
