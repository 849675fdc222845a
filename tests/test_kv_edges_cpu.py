"""The paged cache on the host at its edges: the largest sizes, and what the references hold where steps are taken back."""
import pytest

import deterministic_split_lora_amd as dsl
from deterministic_split_lora_amd import _binding as B
from tests.test_kv_cpu import FAKE, append, attention, cache

LARGEST_CHUNK = (1 << 63) - 256


@pytest.mark.parametrize("chunk", [1 << 31, 1 << 62, LARGEST_CHUNK])
def test_any_chunk_of_the_length_or_more_is_one(chunk):
    """Sizes that no launch takes are refused, however long the chunk, and one chunk needs no workspace."""
    many = cache(n_seqs=60000, max_pages=1 << 24, ld_table=1 << 24)
    huge = dict(T=(1 << 28) - 1, max_new=1 << 20, ws=None, wsb=0)
    for max_len in (100, 1280, 1 << 30):
        assert attention(many, chunk=1 << 30, max_len=max_len, **huge) == B.LORA_ERR_SHAPE
        assert attention(many, chunk=chunk, max_len=max_len, **huge) == B.LORA_ERR_SHAPE
        assert dsl.lora_kv_attention_workspace_bytes(4, 8, 2, 128, 1, max_len, chunk) == 0
    assert attention(chunk=chunk, ws=None, wsb=0, lse=None, ld_lse=0, out=FAKE + 2) == B.LORA_ERR_ALIGN


def test_a_step_without_tokens():
    """Tensors without elements have no address; the norm's weights are there all the same."""
    assert append(T=0, q=None, q_out=None, k=None, v=None) == B.LORA_OK
    assert append(T=0, q=None, q_out=None, k=None, v=None, rope_dim=8) == B.LORA_ERR_UNSUPPORTED
    assert append(T=1, q=None, q_out=None) == B.LORA_ERR_UNSUPPORTED
