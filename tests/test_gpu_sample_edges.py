"""Sampling from logits that differ by almost nothing or by more than a float
holds.  Tokens exactly as the 64-bit reference draws them."""
import numpy as np
import pytest

from oracle import step
from synth import rng_for
from tests.helpers import gpu_available
from tests.test_gpu_step import gpu_logits, run_sample, steady

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not gpu_available(), reason="needs a GPU")]


def rows_against_reference(l, bf16, settings, picks=None, pad=1):
    """Each row of l with its (T, k, p, m): the token in the middle of whose share the random number lies (`picks`, or any
    wide enough one), and the logarithm of its share."""
    g, val = gpu_logits(l, bf16, pad=pad)
    rng = rng_for(l.shape[1], "edges")
    want, u, lp, weight = [], [], [], []
    for i, (T, k, p, m) in enumerate(settings):
        kept = step.kept_weights(val[i], np.float32(T), k, np.float32(p), np.float32(m))
        tok, x = steady(kept, rng)
        if picks is not None:
            tok, x = picks[i], float((np.cumsum(kept)[picks[i]] - kept[picks[i]] / 2) / kept.sum())
        want.append(tok)
        u.append(x)
        lp.append(np.log(kept[tok] / kept.sum()))
        weight.append(kept[tok])
    T, k, p, m = zip(*settings)
    tokens, logprobs = run_sample(g, u, temperature=T, top_k=k, top_p=p, min_p=m)
    assert tokens.tolist() == want
    # A weight's exponent z (no lower than -22.2, where weights end) has three roundings of 2^-24 and its exponential one
    # or two more: the logarithms of the weight and of the sum are each within 22.2 2^-22.  The weight's own rounding to
    # a whole number may go the other way, and the quotient and its logarithm are fp32.
    w = np.array(weight, dtype=np.float64)
    assert np.all(np.abs(logprobs - lp) <= 2 * 22.2 * 2.0 ** -22 + 1.0 / w + 2.0 ** -22 * (1.0 + np.abs(lp)))


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("V", [40, 5000, 60000])
def test_top_k_of_logits_that_hardly_differ(V, bf16):
    """The span of the logits is so small that bins over it have an infinite reciprocal; every row gets a token."""
    l = np.zeros((6, V))
    l[:, 17] = 1e-37
    l[3, 20] = -1e-37
    l[4] = -1e-38
    l[4, 17] = 0.0
    l[5, 5:] = -np.inf
    l[5, 3] = 2e-38
    rows_against_reference(l, bf16, [(1.0, 5, 1.0, 0.0), (1.0, 30, 1.0, 0.0), (0.5, 5, 0.7, 0.0), (1.0, 2, 1.0, 0.5),
                                     (1.0, 7, 1.0, 0.0), (1.0, 4, 1.0, 0.0)])


@pytest.mark.parametrize("bf16", [False, True])
def test_top_k_of_few_logits_far_apart(bf16):
    """Fewer maxima of threads than k, close together, and the other logits very far below them, at a temperature that
    gives those a weight all the same."""
    l = np.full((12, 16), -1e12)
    l[:, 0] = 0.0
    l[:, [8] if bf16 else [4, 8, 12]] = -1e-30
    kept = step.kept_weights(l[0], 1e12, 10)
    picks = np.flatnonzero(kept).tolist()
    assert len(picks) == 10
    rows_against_reference(l, bf16, [(1e12, 10, 1.0, 0.0)] * 12, (picks + picks)[:12], pad=0)


@pytest.mark.parametrize("bf16", [False, True])
def test_differences_beyond_the_largest_float(bf16):
    """Logits of either sign near the type's ends at temperatures near them too: every token is drawn once by its share,
    with and without cuts."""
    l = np.array([3e38, -3e38, 1e38, 0.0, -1e38, -2e38, 2.5e38, -3.3e38])
    V = l.size
    rows, settings, picks = [], [], []
    for T, k, p, m in [(3e38, 0, 1.0, 0.0), (1e38, 0, 1.0, 0.0), (2e37, 0, 1.0, 0.0), (3e38, 7, 1.0, 0.0),
                       (3e38, 0, 0.95, 0.0), (1e38, 5, 1.0, 0.0), (3e38, 0, 1.0, 0.15), (3e38, 7, 0.92, 0.0)]:
        # the logits as the type holds them
        _, val = gpu_logits(l[None], bf16)
        kept = step.kept_weights(val[0], np.float32(T), k, np.float32(p), np.float32(m))
        for i in np.flatnonzero(kept > kept.sum() * 2.0 ** -18):
            rows.append(l)
            settings.append((T, k, p, m))
            picks.append(int(i))
    assert settings.count((3e38, 0, 1.0, 0.0)) == V, "every token has a weight at this temperature"
    rows_against_reference(np.stack(rows), bf16, settings, picks)
