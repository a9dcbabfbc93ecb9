"""The convolution's silu far out, on sums that are exact."""
import pytest
import torch

import gated_delta_rule_72_b200 as gdn
from tests.mixer_ref import HALF, U32
from tests.test_mixer_gpu import BF16, F32

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("C", [64, 5])
def test_silu_of_exact_sums(dtype, C):
    """One tap of one, so the sum is the input itself: silu to a relative
    (8 + |y|) steps (the exponential's argument is rounded once, |y| log2 e) down to
    y = -87; 0 or what fp32 has below it further out."""
    T = 4096
    x = torch.linspace(-120, 120, T * C, device="cuda").view(1, T, C).to(dtype)
    w = torch.zeros(C, 4, device="cuda")
    w[:, 3] = 1.0
    y, _ = gdn.short_conv(x, w)
    want = x.double() * torch.sigmoid(x.double())
    err = (8 + x.double().abs()) * 2 * U32 * want.abs()
    err = err + HALF[dtype] * (want.abs() + err)
    err = torch.where(x.double() < -87, torch.full_like(err, 1.5e-36), err)
    over = (y.double() - want).abs() - err
    assert torch.isfinite(y).all() and float(over.max()) <= 0, float(x.flatten()[over.argmax()])
