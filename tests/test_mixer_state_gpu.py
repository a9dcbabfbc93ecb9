"""How exact the tensor-core scan keeps the state."""
import pytest
import torch

import gated_delta_rule_72_b200 as gdn
from tests.test_mixer_gpu import BF16, _gen, _randn
from tests.test_mixer_regimes_gpu import final_state

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dk,dv,H", [(128, 128, 1), (128, 64, 2), (64, 64, 1)])
@pytest.mark.parametrize("T,at", [(40, 3), (128, 127), (384, 130), (1000, 5), (1000, 999)])
def test_state_of_one_token_keeps_24_bits(T, at, dk, dv, H):
    """One token writes, nothing forgets: the state is d k v^T with the rounding
    of d v, its split into bf16 terms and one cut of the sum for each of three terms.
    (Two terms would be off by up to 2^-17.)"""
    g = _gen(T + at + dk)
    q, k = (_randn(g, 1, T, 1, dk, dtype=BF16) for _ in range(2))
    v = torch.zeros(1, T, H, dv, dtype=BF16, device="cuda")
    v[:, at] = _randn(g, 1, H, dv, dtype=BF16)
    d = 0.1 + torch.rand(1, T, H, generator=g, device="cuda")
    _, s = gdn.ssm_scan(q, k, v, d, torch.zeros(H, device="cuda"), softplus=False)
    want = d[:, at].double()[..., None, None] * k[:, at, :, :, None].double() * v[:, at, :, None].double()
    over = ((s.double() - want).abs() - 6 * 2.0 ** -23 * want.abs()).max()
    assert float(over) <= 0, float(((s.double() - want).abs() / want.abs().clamp_min(1e-30)).max())


def check_long_walk(B, T, H, G, dk, dv):
    """Heads from ones that never forget to ones that forget within a chunk.  A
    chunk's sum is made of 24 products, each of which cuts off up to 2^-23 of the sum
    so far, 2^-24 in the mean; the cuts go towards zero, so those of the
    chunks add up like the chunks do.  Adding a chunk rounds by up to 2^-24 of the state,
    to either side; weights and decays are off by 2^-22."""
    g = _gen(T)
    c = dict(q=_randn(g, B, T, G, dk, dtype=BF16), k=_randn(g, B, T, G, dk, dtype=BF16),
             v=_randn(g, B, T, H, dv, dtype=BF16))
    A = -torch.exp(torch.linspace(-9, 3, H, device="cuda"))
    A[0] = 0.0
    dt = _randn(g, B, T, H) - 4
    state = _randn(g, B, H, dk, dv)
    _, s = gdn.ssm_scan(c["q"], c["k"], c["v"], dt, A, state=state)
    d = torch.nn.functional.softplus(dt.double())
    want = final_state(dict(c, A=A, state=state), d)
    err = float(((s.double() - want).flatten(2).norm(dim=2) / want.flatten(2).norm(dim=2)).max())
    print("state error of the worst head: %.2e" % err)
    assert err <= (24 + 4 + (T / 128) ** 0.5) * 2.0 ** -24, err


@pytest.mark.parametrize("B,T,H,G,dk,dv", [(1, 4096, 80, 8, 128, 128), (1, 20000, 75, 75, 64, 64),
                                           (4, 16384, 32, 8, 128, 128), (2, 300, 40, 1, 64, 128)])
def test_state_of_whole_walks(B, T, H, G, dk, dv):
    check_long_walk(B, T, H, G, dk, dv)


@pytest.mark.parametrize("B,T,H,G,dk,dv", [(1, 32760, 24, 1, 128, 64), (2, 1560, 16, 16, 128, 128),
                                           (1, 20000, 1, 1, 64, 64), (1, 100000, 75, 75, 128, 128)])
def test_state_of_segmented_walks(B, T, H, G, dk, dv):
    """(Contributions of the segments are made of the same sums and join the walk with
    one rounding each.)"""
    check_long_walk(B, T, H, G, dk, dv)
