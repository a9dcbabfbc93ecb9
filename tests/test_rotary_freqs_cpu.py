"""The table of scaled contexts."""
import math

import pytest

import gated_delta_rule_72_b200 as gdn
from tests.test_mixer_cpu import _turns


@pytest.mark.parametrize("factor", [0.5, 0.999])
def test_yarn_does_not_shorten(factor):
    """0.1 ln(factor) + 1 would scale below 1 without notice."""
    with pytest.raises(ValueError, match="factor"):
        gdn.rotary_freqs(64, scaling="yarn", factor=factor, original_len=4096, device="cpu")


def test_yarn_of_factor_one_changes_nothing():
    f, s = gdn.rotary_freqs(64, scaling="yarn", factor=1.0, original_len=4096, device="cpu")
    g, _ = gdn.rotary_freqs(64, device="cpu")
    assert s == 1.0 and _turns(f) == pytest.approx(_turns(g), rel=1e-15)


def test_yarn_ramp_is_linear_in_the_turns():
    n, factor, slow, fast = 4096, 8.0, 1.0, 32.0
    f, _ = gdn.rotary_freqs(64, scaling="yarn", factor=factor, original_len=n, device="cpu")
    for j, got in enumerate(_turns(f)):
        th = 10000.0 ** (-2.0 * j / 64)
        w = min(1.0, max(0.0, (n * th / (2 * math.pi) - slow) / (fast - slow)))
        assert got == pytest.approx(th * (w + (1 - w) / factor), rel=1e-13), j
