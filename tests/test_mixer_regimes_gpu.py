"""The scan's final state where a sequence forgets all and then remembers."""
import pytest
import torch

import gated_delta_rule_72_b200 as gdn
from tests.test_mixer_gpu import BF16, _gen, _randn
from tests.test_mixer_paths_gpu import _kernels

pytestmark = pytest.mark.gpu


def final_state(c, d):
    """sum_j P(T, j) d_j k_j v_j^T (and the initial state) in 64 bits, decays as sums of logs."""
    B, T, G, dk = c["k"].shape
    H = c["v"].shape[2]
    la = d.double() * c["A"].double()
    after = la.flip(1).cumsum(1).flip(1)                 # decay of tokens j .. T-1
    w = d.double() * torch.exp(after - la)               # of those behind j
    k = c["k"].double().repeat_interleave(H // G, 2)
    S = torch.einsum("bth,bthk,bthv->bhkv", w, k, c["v"].double())
    if c.get("state") is not None:
        S = S + torch.exp(after[:, 0])[..., None, None] * c["state"].double()
    return S


@pytest.mark.parametrize("T", [1024, 4096])
@pytest.mark.parametrize("at", [0, 1, 2])
@pytest.mark.parametrize("H,dv", [(2, 64), (1, 128)])
def test_segments_that_forget_before_others_that_remember(T, at, H, dv):
    """256 tokens of an early segment that each clear the state, and ones behind them
    that neither forget nor write much: the state is what the last of the
    clearing tokens wrote, decayed by the sum of many small steps."""
    g = _gen(T + at)
    c = dict(k=_randn(g, 1, T, 1, 128, dtype=BF16), v=_randn(g, 1, T, H, dv, dtype=BF16),
             A=-torch.full((H,), 10.0, device="cuda"), state=_randn(g, 1, H, 128, dv))
    q = _randn(g, 1, T, 1, 128, dtype=BF16)
    d = torch.full((1, T, H), 1e-6, device="cuda")
    d[:, 256 * at:256 * (at + 1)] = 5.0 + torch.rand(1, 256, H, generator=g, device="cuda")
    (_, s), names = _kernels(lambda: gdn.ssm_scan(q, dt=d, softplus=False, **c))
    assert names == {"ssm_tail", "ssm_walk"}
    want = final_state(c, d)
    # a segment is one chunk (T = 1024) or two: 24 or 48 products onto a state, each cut
    # off by at most 2^-23 of it, once in the contributions and once in the last walk;
    # weights and decays by 2^-22 each
    L = 1 if T == 1024 else 2
    err = float((s.double() - want).norm() / want.norm())
    assert err <= (2 * 24 * L + 8) * 2.0 ** -23, err
