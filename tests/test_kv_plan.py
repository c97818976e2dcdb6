"""What the attention over the paged cache launches, by the planner hook (no GPU)."""
import pytest

from bf16_gemm_skinny_gb300 import _native as bsk
from bf16_gemm_skinny_gb300 import build as bsk_build


@pytest.fixture(scope="module", autouse=True)
def lib():
    bsk_build.build()
    return bsk.load()


BOTH = [bsk.CACHE_BF16, bsk.CACHE_E4M3]


@pytest.mark.parametrize("cache", BOTH)
@pytest.mark.parametrize("group", [1, 2, 8])
@pytest.mark.parametrize("tokens", [1, 7, 300])
@pytest.mark.parametrize("loose", [301, 2 ** 20, 2 ** 31 - 1])
def test_a_loose_bound_of_new_tokens_plans_as_the_number_of_tokens(cache, group, tokens, loose):
    """max_chunk decides the kernel, the grid and the flat copy; rows up to max_chunk * group are 32-bit numbers."""
    shape = dict(num_q_heads=2 * group, num_kv_heads=2, head_dim=128, max_seq_len=4000)
    want = bsk.plan_kv_attention(cache, 1, tokens, tokens, **shape)
    assert want["tiles"] == -(-tokens * group // want["cta_rows"])
    assert bsk.plan_kv_attention(cache, 1, tokens, loose, **shape) == want


@pytest.mark.parametrize("cache", BOTH)
def test_one_token_each_plans_as_chunks_of_one(cache):
    shape = dict(num_q_heads=16, num_kv_heads=4, head_dim=256, max_seq_len=9000)
    want = bsk.plan_kv_attention(cache, 40, 40, 1, one_token_each=True, **shape)
    assert want["tiles"] == 1
    assert bsk.plan_kv_attention(cache, 40, 40, 2 ** 31 - 1, one_token_each=True, **shape) == want


@pytest.mark.parametrize("scale", [2.4e38, -3.4e38])
def test_a_scale_whose_product_with_log2_e_is_infinite_is_refused(scale):
    with pytest.raises(bsk.BskError, match="softmax_scale"):
        bsk.decode_attention_enqueue(bsk.CACHE_BF16, 4096, 1 << 20, None, None, 16, 256, 1 << 25, 256, 64, 64, 1, 4, 4, 64, 16,
                                     8, 8, 128, scale, stream=0)


@pytest.mark.parametrize("dim,heads,group,chunk,singles,copied", [
    (128, 8, 8, 256, 63, False), (128, 8, 8, 512, 31, True), (128, 8, 8, 4096, 31, True), (128, 8, 8, 256, 0, True),
    (64, 8, 8, 256, 63, True), (64, 8, 8, 256, 100, False),
    (256, 4, 4, 256, 63, False), (256, 4, 4, 2048, 31, False), (256, 4, 4, 2048, 3, True), (256, 4, 4, 256, 0, True),
])
def test_one_prompt_among_single_tokens_has_the_whole_cache_copied_only_where_it_pays(dim, heads, group, chunk, singles,
                                                                                      copied):
    """The BF16 copy of a quantised cache goes by the rows that read a sequence on average, not by the longest chunk's."""
    plan = bsk.plan_kv_attention(bsk.CACHE_E4M3, singles + 1, singles + chunk, chunk, heads * group, heads, dim, 8000 if singles < 64 else 4000)
    assert (plan["flat_rows"] > 0) == copied


@pytest.mark.parametrize("length", [2 ** 31 - 255, 2 ** 31 - 1])
def test_lengths_whose_whole_tiles_pass_32_bits_are_refused(length):
    with pytest.raises(bsk.BskError, match="max_seq_len"):
        bsk.decode_attention_enqueue(bsk.CACHE_BF16, 4096, 1 << 30, None, None, 16, 256, 1 << 40, 256, 64, 64, 1, 4, 4, 64, 1 << 20,
                                     2048, 2, length, 0.125, 100, 0, stream=0)
