"""What a value that is not finite reaches: nothing of other sequences and
heads, no output of an earlier chunk; where a scan goes token by token, no
earlier output at all."""
import pytest
import torch

import gated_delta_rule_72_b200 as gdn
from tests.test_mixer_gpu import BF16, F32, _conv_case, _ssm_case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("name", ["q", "k", "v", "dt"])
@pytest.mark.parametrize("dtype,T,chunk", [(F32, 1, 1), (F32, 20, 1), (BF16, 20, 1), (F32, 300, 64), (BF16, 300, 128),
                                           (BF16, 1000, 128)])
def test_scan_with_a_value_that_is_not_finite(dtype, T, chunk, name, bad):
    c = _ssm_case(2, T, 2, 2, 128, 64, dtype, T)
    c = {n: t.clone() for n, t in c.items()}
    o, s = gdn.ssm_scan(**c)
    at = (2 * T) // 3
    c[name][1, at, 1] = bad                               # one sequence, one head
    o2, s2 = gdn.ssm_scan(**c)
    assert torch.equal(o[0], o2[0]) and torch.equal(s[0], s2[0])
    assert torch.equal(o[1, :, 0], o2[1, :, 0]) and torch.equal(s[1, 0], s2[1, 0])
    first = at // chunk * chunk
    assert torch.equal(o[1, :first], o2[1, :first])
    if name != "v":                                       # (v meets the zeros of the masked scores)
        assert torch.equal(o[1, :at], o2[1, :at])
    if bad != bad and name != "q":
        assert torch.isnan(o2[1, at:, 1]).all() and torch.isnan(s2[1, 1]).all()
    elif name == "q":
        assert torch.equal(s[1, 1], s2[1, 1]) and torch.equal(o[1, at + 1:], o2[1, at + 1:])


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_convolution_with_a_value_that_is_not_finite(dtype):
    x, w, bias, state = _conv_case(2, 100, 24, 4, dtype, 3)
    x = x.clone()
    y, last = gdn.short_conv(x, w, bias, state)
    x[1, 40, 5] = float("nan")
    y2, last2 = gdn.short_conv(x, w, bias, state)
    reached = torch.zeros_like(y, dtype=torch.bool)
    reached[1, 40:44, 5] = True
    assert torch.isnan(y2[reached]).all() and torch.equal(y[~reached], y2[~reached]) and torch.equal(last, last2)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("T", [1, 4])
@pytest.mark.parametrize("a", [-0.1, -3.0])
def test_infinite_state_element_of_a_step(dtype, T, a):
    """An infinite element stays what it is, the others do not learn of it, however
    much the token forgets."""
    c = _ssm_case(2, T, 2, 1, 64, 64, dtype, 4)
    c = {n: t.clone() for n, t in c.items()}
    c["A"].fill_(a)
    c["dt"] = torch.ones(2, T, 2, device="cuda")
    c["dt_bias"] = None
    _, s = gdn.ssm_scan(**c, softplus=False)
    c["state"][1, 0, 3, 5] = float("inf")
    _, s2 = gdn.ssm_scan(**c, softplus=False)
    other = torch.ones_like(s, dtype=torch.bool)
    other[1, 0, 3, 5] = False
    assert torch.equal(s[other], s2[other]) and s2[1, 0, 3, 5] == float("inf")


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("T", [300, 1000])
def test_infinite_state_element_of_a_prompt(dtype, T):
    c = _ssm_case(2, T, 2, 1, 64, 64, dtype, 5)
    c = {n: t.clone() for n, t in c.items()}
    c["A"].fill_(-0.01)
    c["dt"] = torch.ones(2, T, 2, device="cuda")
    c["dt_bias"] = None
    o, s = gdn.ssm_scan(**c, softplus=False)
    c["state"][1, 0, 3, 5] = float("inf")
    o2, s2 = gdn.ssm_scan(**c, softplus=False)
    other = torch.ones_like(s, dtype=torch.bool)
    other[1, 0, 3, 5] = False
    assert torch.equal(s[other], s2[other]) and s2[1, 0, 3, 5] == float("inf")
    column = torch.ones_like(o, dtype=torch.bool)
    column[1, :, 0, 5] = False
    assert torch.equal(o[column], o2[column])
