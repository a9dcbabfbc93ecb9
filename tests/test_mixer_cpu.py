"""Operators around the scan, without a GPU: refusals of the C-ABI and of the
Python entry points, and the rotary table."""
import math

import pytest
import torch

import gated_delta_rule_72_b200 as gdn
from gated_delta_rule_72_b200 import _lib, build

FAKE = 1 << 20
MB = 1 << 24


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()
    return _lib.load()


def _conv(**kw):
    a = dict(x=FAKE, x_batch_stride=64 * 8, x_token_stride=64, w=FAKE + MB, bias=None, state_in=None,
             state_out=None, y=FAKE + 2 * MB, lengths=None, B=2, T=8, C=64, K=4, silu=1, dt=1, stream=None)
    a.update(kw)
    return _lib.gdn_short_conv(*a.values())


def test_short_conv_refusals():
    assert _conv(dt=2) == -3
    assert _conv(K=1) == -5 and _conv(K=5) == -5
    assert _conv(B=0) == -2 and _conv(T=-1) == -2 and _conv(C=0) == -2 and _conv(B=65536) == -2
    assert _conv(x=None) == -1 and _conv(w=None) == -1 and _conv(y=None) == -1
    assert _conv(x=FAKE + 1) == -4 and _conv(y=FAKE + 2 * MB + 8) == -4 and _conv(state_in=FAKE + 3 * MB + 4) == -4
    assert _conv(lengths=FAKE + 2) == -4
    assert _conv(x_token_stride=63) == -2 and _conv(x_batch_stride=0) == -2
    assert _conv(y=FAKE) == -2                                      # y over x
    assert _conv(y=FAKE + 64 * 8 * 2) == -2
    assert _conv(state_in=FAKE + 2 * MB) == -2                      # state under y
    assert _conv(state_in=FAKE + 4 * MB, state_out=FAKE + 4 * MB + 64) == -2
    assert _conv(T=0, x=None, y=None) == 0                          # nothing to do


def _ssm(**kw):
    a = dict(q=FAKE, q_strides=(8 * 128, 128), k=FAKE + MB, k_strides=(8 * 128, 128), v=FAKE + 2 * MB,
             v_strides=(8 * 256, 256), dt=FAKE + 3 * MB, dt_strides=(32, 4), A=FAKE + 4 * MB, D=None, dt_bias=None,
             state_in=None, state_out=None, o=FAKE + 5 * MB, lengths=None, B=2, T=8, H=4, G=2, dk=64, dv=64,
             softplus=1, t=1, dt_t=0, workspace=None, ws_bytes=0, stream=None)
    a.update(kw)
    return _lib.gdn_ssm_scan(*a.values())


def test_ssm_scan_refusals():
    assert _ssm(t=5) == -3 and _ssm(dt_t=-1) == -3 and _ssm(t=0, dt_t=1) == -3
    assert _ssm(dk=96) == -5 and _ssm(dv=32) == -5
    assert _ssm(B=0) == -2 and _ssm(T=-1) == -2 and _ssm(G=3) == -2 and _ssm(G=0) == -2 and _ssm(H=0) == -2
    assert _ssm(B=16384) == -2                                      # B * H > 65535
    for name in ("q", "k", "v", "dt", "A", "o"):
        assert _ssm(**{name: None}) == -1, name
    for name in ("q", "k", "v", "o", "state_in", "state_out"):
        assert _ssm(**{name: FAKE + 6 * MB + 8}) == -4, name
    assert _ssm(A=FAKE + 2) == -4 and _ssm(D=FAKE + 1) == -4 and _ssm(dt_bias=FAKE + 3) == -4
    assert _ssm(dt=FAKE + 2) == -4
    assert _ssm(q_strides=(8 * 128, 132)) == -4                     # rows off 16 bytes
    assert _ssm(q_strides=(8 * 128, 64)) == -2                      # rows overlap
    assert _ssm(dt_strides=(32, 2)) == -2
    assert _ssm(o=FAKE + 2 * MB) == -2                              # o over v
    assert _ssm(o=FAKE + 3 * MB) == -2                              # o over dt
    assert _ssm(state_out=FAKE) == -2
    assert _ssm(state_in=FAKE + 6 * MB, state_out=FAKE + 6 * MB + 256) == -2
    assert _ssm(T=0, q=None, k=None, v=None, dt=None, A=None, o=None) == 0


def _rot(**kw):
    st = (4 * 2 * 64, 2 * 64, 64)
    a = dict(q=FAKE, q_strides=st, q_out=FAKE + MB, q_out_strides=st, Hq=2, k=FAKE + 2 * MB, k_strides=st,
             k_out=FAKE + 3 * MB, k_out_strides=st, Hk=2, pos=FAKE + 4 * MB, pos_bits=64, axes=1, freqs=FAKE + 5 * MB,
             scale=1.0, B=2, T=4, d=64, rot=32, interleaved=0, dt=1, stream=None)
    a.update(kw)
    return _lib.gdn_rotary(*a.values())


def test_rotary_refusals():
    assert _rot(dt=3) == -3 and _rot(pos_bits=16) == -3
    assert _rot(rot=31) == -5 and _rot(rot=0) == -5 and _rot(rot=66) == -5 and _rot(d=2048) == -5
    assert _rot(B=0) == -2 and _rot(T=-1) == -2 and _rot(Hq=0) == -2 and _rot(axes=0) == -2 and _rot(axes=9) == -2
    assert _rot(scale=float("nan")) == -2 and _rot(scale=float("inf")) == -2
    for name in ("q", "q_out", "k", "k_out", "pos", "freqs"):
        assert _rot(**{name: None}) == -1, name
    assert _rot(q=FAKE + 1) == -4 and _rot(pos=FAKE + 4 * MB + 4) == -4 and _rot(freqs=FAKE + 5 * MB + 4) == -4
    st = (4 * 2 * 64, 2 * 64, 64)
    assert _rot(q_out=FAKE + 64) == -2                              # partly over its input
    assert _rot(q_out=FAKE + 2 * MB) == -2                          # over the other input
    assert _rot(k_out=FAKE + MB) == -2                              # both results in one place
    assert _rot(q_out_strides=(4 * 2 * 64, 2 * 64, 0)) == -2        # an output that overlaps itself
    assert _rot(q_out_strides=(0, 2 * 64, 64)) == -2
    assert _rot(q=FAKE, k=FAKE, q_out=FAKE, k_out=FAKE) == -2       # one tensor, turned twice
    assert _rot(q_strides=(0, 128, 64), q_out_strides=(0, 128, 64), q_out=FAKE) == -2   # in place, shared rows
    assert _rot(T=0, q=None, q_out=None, k=None, k_out=None, pos=None, freqs=None) == 0
    del st


def test_python_calls_refuse_cpu_tensors():
    x = torch.zeros(1, 4, 64)
    with pytest.raises(ValueError):
        gdn.short_conv(x, torch.zeros(64, 4))
    q = torch.zeros(1, 4, 1, 64)
    with pytest.raises(ValueError):
        gdn.ssm_scan(q, q, q, torch.zeros(1, 4, 1), torch.zeros(1))
    f, _ = gdn.rotary_freqs(64, device="cpu")
    with pytest.raises(ValueError):
        gdn.rotary(q, None, torch.zeros(1, 4, dtype=torch.int64), f)


@pytest.mark.parametrize("kw", [dict(rot_dim=63), dict(rot_dim=0), dict(rot_dim=64, scaling="other"),
                                dict(rot_dim=64, base=0.0), dict(rot_dim=64, factor=-1.0),
                                dict(rot_dim=64, axes=(32, 30)), dict(rot_dim=64, axes=(33, 31)),
                                dict(rot_dim=64, scaling="yarn"), dict(rot_dim=2, scaling="ntk")])
def test_rotary_freqs_refusals(kw):
    with pytest.raises(ValueError):
        gdn.rotary_freqs(device="cpu", **kw)


def _turns(freqs):
    """The table's angles per position, in radians."""
    return [(int(p) % 2 ** 64) / 2.0 ** 64 * 2 * math.pi for p in freqs[0]]


def test_rotary_table_holds_the_angles():
    f, scale = gdn.rotary_freqs(8, base=100.0, device="cpu")
    assert scale == 1.0 and f.shape == (2, 4) and f[1].tolist() == [0, 0, 0, 0]
    assert _turns(f) == pytest.approx([1.0, 100 ** -0.25, 100 ** -0.5, 100 ** -0.75], rel=1e-15)
    f, _ = gdn.rotary_freqs(8, base=100.0, scaling="linear", factor=4.0, device="cpu")
    assert _turns(f)[0] == pytest.approx(0.25, rel=1e-15)
    f, _ = gdn.rotary_freqs(8, base=100.0, scaling="ntk", factor=4.0, device="cpu")
    # the last pair turns factor times slower, the first as before
    assert _turns(f)[0] == pytest.approx(1.0, rel=1e-15)
    assert _turns(f)[3] == pytest.approx(100 ** -0.75 / 4.0, rel=1e-14)
    f, s = gdn.rotary_freqs(64, scaling="yarn", factor=8.0, original_len=4096, device="cpu")
    g, _ = gdn.rotary_freqs(64, device="cpu")
    assert s == pytest.approx(0.1 * math.log(8.0) + 1.0)
    a, b = _turns(f), _turns(g)
    assert a[0] == b[0] and a[-1] == pytest.approx(b[-1] / 8.0, rel=1e-14)
    assert all(b[i] / 8.0 <= a[i] * (1 + 1e-12) and a[i] <= b[i] * (1 + 1e-12) for i in range(32))
    f, _ = gdn.rotary_freqs(128, axes=(44, 42, 42), device="cpu")
    assert f[1].tolist() == [0] * 22 + [1] * 21 + [2] * 21
    assert _turns(f)[22] == pytest.approx(1.0, rel=1e-15) and _turns(f)[43] == pytest.approx(1.0, rel=1e-15)


def test_rotary_angle_of_far_positions_is_exact():
    """The product of a position and the table's phase, modulo one turn, is the
    angle to 2^-32 of a turn: 2^-65 of the table times a position of 2^31."""
    from fractions import Fraction
    two_pi = 2 * Fraction("3.14159265358979323846264338327950288419716939937510")
    f, _ = gdn.rotary_freqs(64, device="cpu")
    for pos in (1, 12345, 1 << 20, (1 << 31) - 1, -7):
        for j, p in enumerate(f[0].tolist()):
            got = Fraction(pos * p % 2 ** 64, 2 ** 64)
            ref = pos * Fraction(10000.0 ** (-2.0 * j / 64)) / two_pi
            d = (got - ref) % 1
            assert min(d, 1 - d) <= Fraction(abs(pos), 2 ** 64), (pos, j)


def test_workspace_size_of_refused_sizes_is_zero():
    assert gdn.ssm_workspace_size(0, 256, 4, 1, 64, 64) == 0
    assert gdn.ssm_workspace_size(1, 256, 4, 3, 64, 64) == 0
    assert gdn.ssm_workspace_size(1, 256, 4, 1, 96, 64) == 0
    assert gdn.ssm_workspace_size(1, 0, 4, 1, 64, 64) == 0


def test_steps_need_a_state():
    x = torch.zeros(1, 1, 8)
    with pytest.raises(ValueError, match="state"):
        gdn.short_conv_step(x, torch.zeros(8, 4), None, None)
    q = torch.zeros(1, 1, 1, 64)
    with pytest.raises(ValueError, match="state"):
        gdn.ssm_step(q, q, q, torch.zeros(1, 1, 1), torch.zeros(1), None)
