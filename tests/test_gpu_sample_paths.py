"""Sampling rows that the usual paths pass on to the general one, or nearly: masks
of finite lowest values, logits ordered by index, flat rows, large top-k; NaN and
minus zero.  Tokens exactly as the 64-bit reference draws them."""
import numpy as np
import pytest

from oracle import step
from synth import rng_for
from tests.helpers import gpu_available
from tests.test_gpu_sample_edges import rows_against_reference
from tests.test_gpu_step import gpu_logits, run_sample, safe_p

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not gpu_available(), reason="needs a GPU")]

SETTINGS = [(1.0, 0, 1.0, 0.0), (0.7, 50, 1.0, 0.0), (1.3, 0, 0.8, 0.0), (1.0, 0, 1.0, 0.05), (1.0, 40, 0.6, 0.02),
            (0.0, 0, 1.0, 0.0), (0.0, 9, 0.5, 0.3)]


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("V", [9, 700, 32000, 100003])
def test_nan_counts_as_masked(V, bf16):
    """NaN of either sign among the logits, greedy rows and every cut."""
    rng = rng_for(V, "nan")
    l = rng.standard_normal((len(SETTINGS), V)) * 2.0
    l[rng.random(l.shape) < 0.3] = np.nan
    l[rng.random(l.shape) < 0.1] = -np.nan
    l[:, 4] = 3.0
    rows_against_reference(l, bf16, SETTINGS)


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("V", [12, 3000, 50000])
def test_minus_zero_ties_with_zero(V, bf16):
    """Zeros of both signs above everything else: among them the index alone decides."""
    rng = rng_for(V, "zero")
    l = np.where(rng.random((7, V)) < 0.5, 0.0, -0.0)
    l[:, V // 2:] = -40.0
    l[:, 0] = -0.0
    l[:, 1] = 0.0
    n = V // 2
    rows_against_reference(l, bf16, [(0.0, 0, 1.0, 0.0), (1.0, 1, 1.0, 0.0), (1.0, 3, 1.0, 0.0), (1.0, 0, 1.0, 0.0),
                                     (1.0, 0, 2.5 / n, 0.0), (1.0, 0, 1.0, 0.5), (1.0, n + 2, 1.0, 0.5)],
                           [0, 0, 2, n - 1, 2, n - 1, n - 1])


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("lowest", [-1e9, -3.3e38])
def test_masks_of_a_finite_lowest_value(lowest, bf16):
    """Most logits at a mask's finite value, some threads' all of them, and a few thousand alive."""
    V = 64000
    rng = rng_for(7, "mask")
    l = np.full((7, V), lowest)
    for i in range(7):
        alive = rng.permutation(V)[:(3000, 40, 3000, 3000, 1, 900, 3000)[i]]
        l[i, alive] = rng.standard_normal(alive.size) * 2.0
    rows_against_reference(l, bf16, [(1.0, 50, 1.0, 0.0), (1.0, 50, 1.0, 0.0), (1.0, 0, 0.9, 0.0), (1.0, 0, 1.0, 0.01),
                                     (1.0, 5, 0.5, 0.0), (0.8, 900, 1.0, 0.0), (0.0, 0, 1.0, 0.0)])


@pytest.mark.parametrize("bf16", [False, True])
def test_logits_that_fall_with_the_index(bf16):
    """As in vocabularies ordered by frequency: the largest logits are neighbours."""
    V = 128259
    l = -3.0 * np.log1p(np.arange(V) / 50.0) + rng_for(8, "ordered").standard_normal((6, V))
    rows_against_reference(l, bf16, [(1.0, 50, 1.0, 0.0), (1.0, 200, 1.0, 0.0), (1.0, 400, 1.0, 0.0),
                                     (1.0, 1024, 1.0, 0.0), (1.0, 0, 1.0, 0.0), (0.0, 0, 1.0, 0.0)])


@pytest.mark.parametrize("V", [20000, 128259])
def test_flat_rows_and_large_top_k(V):
    """High temperatures, whose cuts fall among thousands of nearly equal weights, and top-k of hundreds.  Fp32: no ties."""
    l = rng_for(V, "flat").standard_normal((8, V))
    base = step.kept_weights(l[0].astype(np.float32).astype(np.float64), 4.0)
    p = safe_p(np.sort(base)[::-1], V // 2)
    rows_against_reference(l, False, [(4.0, 0, 1.0, 0.0), (8.0, 512, 1.0, 0.0), (1.0, 600, 1.0, 0.0),
                                      (1.0, 700, 1.0, 0.0), (1.0, 1000, 1.0, 0.0), (1.0, 1024, 1.0, 0.0),
                                      (2.0, 5000, 1.0, 0.0), (1.0, 0, 1.0, 0.0)])
    # top-p among nearly equal weights: off by one kept token (2^-14 of the sum and less) moves a share by as much, so
    # the random number is put at a token's middle and the token may be a neighbour in index among the kept
    g, val = gpu_logits(l[:1], False)
    kept = step.kept_weights(val[0], 4.0, 0, np.float32(p))
    tokens, _ = run_sample(g, [0.5], temperature=[4.0], top_p=[p])
    share = np.cumsum(kept) / kept.sum()
    slack = 2.0 / np.count_nonzero(kept)
    assert np.searchsorted(share, 0.5 - slack) <= tokens[0] <= np.searchsorted(share, 0.5 + slack)
    assert kept[tokens[0]] > 0
