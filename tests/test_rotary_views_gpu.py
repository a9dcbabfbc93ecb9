"""Rotary positions in place, q, k and v of a head beside one another."""
import pytest
import torch

import gated_delta_rule_72_b200 as gdn
from tests.test_mixer_gpu import BF16, F32, _gen, _randn

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("B,T", [(1, 1), (2, 1), (1, 33), (2, 33)])
@pytest.mark.parametrize("rot", [64, 24])
def test_heads_of_q_k_and_v_in_turn(dtype, B, T, rot):
    """[B, T, H, 3, d]: the views' spans overlap, their elements do not."""
    qkv = _randn(_gen(B + T), B, T, 5, 3, 64, dtype=dtype)
    freqs, _ = gdn.rotary_freqs(rot, device="cuda")
    pos = torch.arange(T, device="cuda").repeat(B, 1) + 7
    q, k, v = qkv.unbind(3)
    keep = v.clone()
    a, b = gdn.rotary(q, k, pos, freqs)
    gdn.rotary(q, k, pos, freqs, q_out=q, k_out=k)
    assert torch.equal(q, a) and torch.equal(k, b) and torch.equal(v, keep)
    # q turned into the place of v, k where it is
    c, d = gdn.rotary(q, k, pos, freqs)
    gdn.rotary(q, k, pos, freqs, q_out=v, k_out=k)
    assert torch.equal(v, c) and torch.equal(k, d) and torch.equal(q, a)
