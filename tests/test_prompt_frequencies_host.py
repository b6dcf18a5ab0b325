"""The frequencies of a longer context, between the ends that stay or are divided. CPU only."""

import math

import pytest
import torch

import linear_attention_state_chunked_gb300 as L


@pytest.mark.parametrize("fast,slow", [(32.0, 1.0), (16.0, 2.0)])
def test_yarn_ramp_is_linear_in_the_turns(fast, slow):
    """Of a pair's frequency f stays keep f, and (1 - keep) f is divided by the factor, where
    keep = (turns - slow) / (fast - slow) with turns = trained f / 2 pi."""
    factor, trained = 8.0, 4096
    f = 10000.0 ** (-torch.arange(0, 128, 2).double() / 128)
    g, _ = L.rope_frequencies(128, yarn=factor, trained=trained, beta_fast=fast, beta_slow=slow, device="cpu")
    between = 0
    for x, y in zip(f.tolist(), g.tolist()):
        turns = trained * x / (2 * math.pi)
        keep = min(1.0, max(0.0, (turns - slow) / (fast - slow)))
        between += 0.0 < keep < 1.0
        assert math.isclose(y, x * keep + x * (1.0 - keep) / factor, rel_tol=2.0 ** -23)
    assert between > 5


def test_yarn_ramp_at_the_documented_turns():
    """A pair of 5.7 turns keeps 0.15 of its frequency; a ramp by the pair's index, which is linear
    in the logarithm of the turns, would keep 0.50."""
    base, trained, factor = 10000.0, 4096, 4.0
    i = -128 / 2 * math.log(5.7 * 2 * math.pi / trained) / math.log(base)  # the pair of 5.7 turns, between two
    g, _ = L.rope_frequencies(128, base, yarn=factor, trained=trained, device="cpu")
    f, _ = L.rope_frequencies(128, base, device="cpu")
    keep = ((g / f).double() - 1 / factor) / (1 - 1 / factor)
    lo, hi = keep[math.ceil(i)], keep[math.floor(i)]
    assert lo < (5.7 - 1) / 31 < hi and abs((5.7 - 1) / 31 - 0.15) < 0.005
    assert hi < 0.5 and abs(math.log(5.7) / math.log(32) - 0.50) < 0.005
