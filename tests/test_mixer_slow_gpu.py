"""Heads that forget slowly, token by token: the decays' rounding does not add
up to one side."""
import pytest
import torch

import gated_delta_rule_72_b200 as gdn
from tests.test_mixer_gpu import BF16, F32, _gen, _randn
from tests.test_mixer_paths_gpu import _kernels
from tests.test_mixer_regimes_gpu import final_state

pytestmark = pytest.mark.gpu


def _case(T, H, dk, dv, dtype, seed):
    g = _gen(seed)
    c = dict(k=_randn(g, 1, T, 1, dk, dtype=dtype), v=_randn(g, 1, T, H, dv, dtype=dtype),
             A=-torch.exp(torch.linspace(-12, 4, H, device="cuda")), state=_randn(g, 1, H, dk, dv))
    d = torch.nn.functional.softplus(_randn(g, 1, T, H) - 8)
    return c, d, _randn(g, 1, T, 1, dk, dtype=dtype)


def _check(c, d, s, T, nearest):
    # each token: the rounding of the products and of the sum, 2^-24 each, to either side:
    # they add up like the root of their number (twice that for the worst of the heads);
    # nearest: with the decays that fp32 holds
    if nearest:
        a = torch.exp(d.double() * c["A"].double()).float().double()
        c, d = dict(c, A=torch.ones_like(c["A"])), (d.double(), torch.log(a))
        after = d[1].flip(1).cumsum(1).flip(1)
        want = torch.einsum("bth,btk,bthv->bhkv", d[0] * torch.exp(after - d[1]), c["k"][:, :, 0].double(),
                            c["v"].double()) + torch.exp(after[:, 0])[..., None, None] * c["state"].double()
    else:
        want = final_state(c, d)
    err = float(((s.double() - want).flatten(2).norm(dim=2) / want.flatten(2).norm(dim=2)).max())
    print("%d tokens: %.2e" % (T, err))
    assert err <= (2 * T ** 0.5 + 8) * 2.0 ** -24, err


@pytest.mark.parametrize("dk,dv", [(128, 64), (64, 128)])
def test_walk_of_fp32_columns(dk, dv):
    T = 700
    c, d, q = _case(T, 70, dk, dv, F32, dk)
    (_, s), names = _kernels(lambda: gdn.ssm_scan(q, dt=d, softplus=False, **c))
    assert names == {"ssm_cols"}, names
    _check(c, d, s, T, True)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("n", [1, 5])
def test_steps(dtype, n):
    """3,000 tokens in calls of one, and of five."""
    T = 3000
    c, d, q = _case(T, 16, 64, 64, dtype, n)
    s = c["state"].clone()
    for t in range(0, T, n):
        gdn.ssm_step(q[:, t:t + n], c["k"][:, t:t + n], c["v"][:, t:t + n], d[:, t:t + n], c["A"], s, softplus=False)
    _check(c, d, s, T, n > 1)
