"""The Python side of the calls on the paged cache: how arguments are taken (no GPU: calls without tokens)."""
import numpy as np
import pytest

from bf16_gemm_skinny_gb300 import _native as bsk


def append(k_cache=None, k_stride=256, num_seqs=0, num_tokens=0, stream=0, block_tables=None):
    bsk.kv_cache_append_enqueue(bsk.CACHE_BF16, k_cache, None, None, None, None, k_stride, None, 256, None, block_tables,
                                None, num_seqs, num_tokens, 4, 64, 16, 8, 8, stream)


class Tensor:
    """What a tensor has to have."""

    def __init__(self, address):
        self.address = address

    def data_ptr(self):
        return self.address


@pytest.mark.parametrize("cache", [None, 0, 4096, 2**64 - 16, Tensor(4096), np.zeros(8, np.uint16)])
def test_addresses(cache):
    append(cache)   # no tokens: nothing is read


@pytest.mark.parametrize("cache", ["4096", 4096.0, object()])
def test_what_has_no_address(cache):
    with pytest.raises((TypeError, AttributeError)):
        append(cache)


def test_an_error_inside_data_ptr_is_passed_on():
    class Freed:
        def data_ptr(self):
            raise RuntimeError("freed")

    with pytest.raises(RuntimeError, match="freed"):
        append(Freed())


def test_addresses_reach_the_checks():
    with pytest.raises(bsk.BskError, match="16-byte aligned"):
        bsk.kv_cache_append_enqueue(
            bsk.CACHE_BF16, Tensor(4104), 8192, None, None, 16, 256, 16, 256, None, 64, 64, 1, 1, 4, 64, 16, 8, 8, 0)
    with pytest.raises(bsk.BskError, match="NULL"):
        append(4096, num_seqs=1, num_tokens=1)


@pytest.mark.parametrize("value", [2**31, -2**31 - 1, 2**70])
def test_integers_out_of_range(value):
    with pytest.raises(OverflowError):
        append(k_stride=value)


def test_wrong_types_and_counts():
    with pytest.raises(TypeError):
        append(k_stride=1.5)
    with pytest.raises(TypeError):
        append(k_stride=None)
    with pytest.raises(TypeError, match="arguments"):
        bsk._load_calls().kv_cache_append(0)
    with pytest.raises(bsk.BskError, match="softmax_scale|finite"):
        bsk.decode_attention_enqueue(bsk.CACHE_BF16, 4096, 8192, None, None, 16, 256, 65536, 256, 64, 64, 1, 4, 4, 64, 16,
                                     8, 8, 128, float("nan"), stream=0)
