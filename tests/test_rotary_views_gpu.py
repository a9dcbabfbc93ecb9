"""Rotary positions in place, q, k and v of a head beside one another."""
import random

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


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_time_major_tensor_of_q_and_k(dtype):
    """[T, B, heads, d] memory: a batch's rows stand between one another's tokens."""
    qk = _randn(_gen(3), 33, 3, 7, 64, dtype=dtype).transpose(0, 1)
    q, k = qk[:, :, :5], qk[:, :, 5:]
    freqs, _ = gdn.rotary_freqs(64, device="cuda")
    pos = torch.arange(33, device="cuda").repeat(3, 1)
    a, b = gdn.rotary(q, k, pos, freqs)
    gdn.rotary(q, k, pos, freqs, q_out=q, k_out=k)
    assert torch.equal(q, a) and torch.equal(k, b)


def _elements(t):
    """Offsets of a view's elements in its memory."""
    off = torch.full((1,), t.storage_offset())
    for n, s in zip(t.shape, t.stride()):
        off = (off[:, None] + torch.arange(n) * s).flatten()
    return off


@pytest.mark.parametrize("seed", range(4))
def test_views_of_one_buffer(seed):
    """q and k turned in place in random views of one buffer: done as in tensors of
    their own where no element is shared, refused where one is."""
    rng = random.Random(seed)
    d, done, refused = 8, 0, 0
    freqs, _ = gdn.rotary_freqs(d, device="cuda")
    for _ in range(300):
        B, T, Hq, Hk = (rng.randint(1, 3) for _ in range(4))
        # nested strides in a random order of the dimensions, room for two heads' worth between
        order = rng.sample([("B", B), ("T", T), ("H", max(Hq, Hk))], 3)
        strides, ext = {}, d
        for name, n in order:
            strides[name] = ext * rng.choice([1, 1, 2, 3]) + rng.choice([0, 0, 3, 8])
            ext = (n - 1) * strides[name] + ext
        off = rng.choice([0, d, 2 * d, strides["H"] // 2, strides["T"] // 2, strides["B"] // 2, Hq * strides["H"],
                          rng.randint(0, ext)])
        buf = torch.randn(ext + off + 64, device="cuda")
        st = (strides["B"], strides["T"], strides["H"], 1)
        q, k = buf.as_strided((B, T, Hq, d), st, 0), buf.as_strided((B, T, Hk, d), st, off)
        eq, ek = _elements(q), _elements(k)
        assert eq.unique().numel() == eq.numel() and ek.unique().numel() == ek.numel()
        shared = bool(torch.isin(eq, ek).any())
        pos = torch.arange(T, device="cuda").repeat(B, 1) + 1
        a, b = gdn.rotary(q, k, pos, freqs)
        if shared:
            with pytest.raises(gdn.GDNError):
                gdn.rotary(q, k, pos, freqs, q_out=q, k_out=k)
            refused += 1
        else:
            gdn.rotary(q, k, pos, freqs, q_out=q, k_out=k)
            assert torch.equal(q, a) and torch.equal(k, b)
            done += 1
    assert done > 50 and refused > 50, (done, refused)
