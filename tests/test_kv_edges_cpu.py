"""The paged cache on the host at its edges: the largest sizes, and what the references hold where steps are taken back."""
import numpy as np
import pytest

import deterministic_split_lora_amd as dsl
from deterministic_split_lora_amd import _binding as B
from oracle import kv
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


def test_reference_keeps_a_scale_that_a_rejected_token_raised():
    """What include/lora_det.h says of tokens that are taken back: their byte stays, and codes rounded to it stay so."""
    D = 64
    x = np.zeros((6, 1, D))
    x[:, 0, 0] = [1.75, 1.0, 1.0, 1.0, 1.0, 1.0]               # byte 119, codes of 2^8 the value
    x[:, 0, 1] = 2.0 ** -13                                     # code 2^-5 at that byte
    draft = np.zeros((1, 1, D))
    draft[0, 0, 0] = 1.75 * 2.0 ** 6                            # byte 125: the small values' codes would be 2^-11: 0
    states = []
    for reject in (False, True):
        c = {"k": np.zeros((1, 1, 16, D), np.uint8), "v": np.zeros((1, 1, 1, D, 16), np.uint8),
             "ks": np.zeros((1, 1, 1), np.uint8), "vs": np.zeros((1, 1, 1), np.uint8)}
        kv.append(c, x[:4], x[:4], np.array([[0]]), [4], [0, 4], 16)
        new = np.concatenate([x[4:5], draft]) if reject else x[4:5]
        kv.append(c, new, new, np.array([[0]]), [4 + len(new)], [0, len(new)], 16)
        kv.append(c, x[5:], x[5:], np.array([[0]]), [6], [0, 1], 16)
        states.append(c)
    plain, after = states
    assert plain["ks"][0, 0, 0] == plain["vs"][0, 0, 0] == 119 and after["ks"][0, 0, 0] == after["vs"][0, 0, 0] == 125
    value = lambda c: kv.sequence(c, np.array([[0]]), 0, 6, 16)  # noqa: E731
    for name in (0, 1):
        assert np.array_equal(value(plain)[name][:, 0, :2], x[:, 0, :2])
        assert np.array_equal(value(after)[name][:, 0, 0], x[:, 0, 0]) and not value(after)[name][:, 0, 1].any()
