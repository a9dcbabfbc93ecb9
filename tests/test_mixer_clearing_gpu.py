"""Heads that clear the state with every token: A as far below zero as fp32
holds, and -inf.  A token without a step (and every place behind a sequence's
end) changes nothing all the same."""
import pytest
import torch

import gated_delta_rule_72_b200 as gdn
from tests import mixer_ref as ref
from tests.test_mixer_gpu import BF16, F32, _gen, _inside, _ssm_bounds, _ssm_case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("A", [-3e38, float("-inf")])
@pytest.mark.parametrize("T,H", [(1, 2), (20, 2), (50, 48), (200, 2), (1000, 2)])
def test_heads_that_clear_the_state(dtype, A, T, H):
    B = 8 if T == 50 else 2
    c = _ssm_case(B, T, H, 1, 128, 64, dtype, T + H)
    g = _gen(T)
    d = 0.5 + torch.rand(B, T, H, generator=g, device="cuda")
    d[torch.rand(B, T, H, generator=g, device="cuda") < 0.3] = 0.0
    d[1, T // 2:] = 0.0                                  # nothing behind the middle
    c.update(dt=d, dt_bias=None, A=torch.full((H,), -3e38, device="cuda"))
    c["A"][0] = -1.0
    lengths = torch.full((B,), T, dtype=torch.int32, device="cuda")
    lengths[0] = max(T - 3, 0)
    for lens in (None, lengths):
        want, ws, mag, N = ref.ssm(c["q"], c["k"], c["v"], c["dt"], c["A"], c["D"], None, c["state"], False, lens)
        e = dict(c, A=torch.where(c["A"] < -2, torch.full_like(c["A"], A), c["A"]))
        o, s = gdn.ssm_scan(**e, softplus=False, lengths=lens)
        bo, bs = _ssm_bounds(c, T, want, mag, N)
        _inside(o, want, bo + 1e-37, "o")
        _inside(s, ws, bs + 1e-37, "state")
