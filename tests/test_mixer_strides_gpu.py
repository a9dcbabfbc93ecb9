"""Views whose batch stride is below their token stride (time-major memory)."""
import pytest
import torch

import gated_delta_rule_72_b200 as gdn
from tests.test_mixer_gpu import BF16, F32, _conv_case, _ssm_case

pytestmark = pytest.mark.gpu


def _time_major(t, pad=0):
    """The same values in [T, B, ...] memory, seen as [B, T, ...]."""
    B, T = t.shape[:2]
    flat = t[0, 0].numel()
    buf = torch.full((T, B, flat + pad), float("nan"), dtype=t.dtype, device="cuda")
    buf[..., :flat] = t.transpose(0, 1).reshape(T, B, flat)
    return buf[..., :flat].unflatten(-1, t.shape[2:]).transpose(0, 1)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("T", [1, 20, 300, 1000])
def test_scan_of_time_major_views(dtype, T):
    c = _ssm_case(3, T, 4, 2, 128, 64, dtype, T)
    c = {n: t.contiguous() for n, t in c.items()}
    lengths = torch.tensor([T, T // 2, max(T - 1, 0)], dtype=torch.int32, device="cuda")
    for lens in (None, lengths):
        o, s = gdn.ssm_scan(**c, lengths=lens)
        m = {n: _time_major(t, pad=8) if n in ("q", "k", "v", "dt") else t for n, t in c.items()}
        assert T == 1 or m["v"].stride(0) < m["v"].stride(1)
        o2, s2 = gdn.ssm_scan(**m, lengths=lens)
        assert torch.equal(o, o2) and torch.equal(s, s2)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("C,pad", [(64, 8), (37, 3)])
def test_convolution_of_time_major_views(dtype, C, pad):
    x, w, bias, state = _conv_case(3, 200, C, 4, dtype, C)
    y, last = gdn.short_conv(x, w, bias, state)
    y2, last2 = gdn.short_conv(_time_major(x, pad), w, bias, state)
    assert torch.equal(y, y2) and torch.equal(last, last2)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_rotary_of_time_major_views(dtype):
    c = _ssm_case(3, 77, 4, 2, 128, 64, dtype, 5)
    freqs, _ = gdn.rotary_freqs(128, device="cuda")
    pos = torch.arange(77, device="cuda").repeat(3, 1)
    q, k = c["q"].contiguous(), c["k"].contiguous()
    a, b = gdn.rotary(q, k, pos, freqs)
    q2, k2 = _time_major(q, 8), _time_major(k, 1)
    a2, b2 = gdn.rotary(q2, k2, pos, freqs)
    assert torch.equal(a, a2) and torch.equal(b, b2)
    gdn.rotary(q2, k2, pos, freqs, q_out=q2, k_out=k2)
    assert torch.equal(a, q2) and torch.equal(b, k2)
