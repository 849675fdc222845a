"""Attention over the paged 8-bit cache at its edges: every kernel variant (rows of a key head that the waves split, two
tiles of them, many) with windows, pages that are not there, blocks that were never written and values that are NaN."""
import numpy as np
import pytest

from tests.helpers import gpu_available, torch
from tests.kv_helpers import Batch, attend, heads_bf16

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not gpu_available(), reason="needs a GPU")]

NEW = [1, 5, 40]                                                # with 8 rows a token: 8, 40 and 320 rows of a key head


def bits(t):
    return t.view(torch().int16 if t.dtype == torch().bfloat16 else torch().int32)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("P", [16, 64, 128])
@pytest.mark.parametrize("new", NEW)
def test_blocks_before_the_window_may_hold_anything(D, P, new):
    """Codes and scales of blocks that no query of the step sees any more: NaN, the largest, scales that are none."""
    t = torch()
    window = 10
    batch = Batch([(new, 150), (new, 107)], P, 1, D, seed=3).fill()
    q, qg = heads_bf16(batch.T, 8, D, 1.0, 4, "q")
    want, wlse = attend(qg, batch.gpu(), new, window=window)
    for scale in (0, 247, 254, 255):
        for code in (0x7E, 0xFE, 0x7F):
            for b, n in ((0, 150), (1, 107)):
                for block in range((n - new - window + 1) // 16):
                    page, w = batch.table[b, block * 16 // P], block * 16 % P // 16
                    batch.cache["ks"][page, :, w] = batch.cache["vs"][page, :, w] = scale
                    batch.cache["k"][page, :, w * 16:(w + 1) * 16] = code
                    batch.cache["v"][page, :, w] = code
            out, lse = attend(qg, batch.gpu(), new, window=window)
            assert not bool(t.isnan(out).any()), (scale, code)
            assert t.equal(bits(out), bits(want)) and t.equal(bits(lse), bits(wlse)), (scale, code)
