"""Operators around the scan on the GPU, against their 64-bit definitions."""
import pytest
import torch

import gated_delta_rule_72_b200 as gdn
from tests import mixer_ref as ref
from tests.mixer_ref import HALF, U32

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


def _gen(seed):
    return torch.Generator("cuda").manual_seed(seed)


def _randn(g, *shape, dtype=F32):
    return torch.randn(*shape, generator=g, device="cuda").to(dtype)


def _inside(x, want, bound, what):
    d = (x.double() - want).abs()
    assert torch.isfinite(x).all(), what
    worst = float((d - bound).max())
    assert worst <= 0, (what, worst, float(d.max()))


# ---------------------------------------------------------------- convolution
def _conv_case(B, T, C, K, dtype, seed, pad=0):
    g = _gen(seed)
    wide = _randn(g, B, T, C + pad, dtype=dtype)
    return (wide[:, :, pad:], _randn(g, C, K), _randn(g, C), _randn(g, B, K - 1, C, dtype=dtype))


def _check_conv(x, w, bias, state, silu, lengths, y, last):
    want, want_last, err = ref.conv(x, w, bias, state, silu, lengths)
    _inside(y, want, err + HALF[x.dtype] * (want.abs() + err) + 1e-37, "y")
    assert torch.equal(last.double(), want_last)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("K", [2, 3, 4])
@pytest.mark.parametrize("T,C,pad", [(1, 64, 0), (2, 24, 8), (3, 5, 0), (63, 1283, 37), (64, 128, 0), (65, 72, 3),
                                     (200, 256, 64)])
def test_short_conv(dtype, K, T, C, pad):
    x, w, bias, state = _conv_case(2, T, C, K, dtype, 10 * T + K, pad)
    for silu in (True, False):
        y, last = gdn.short_conv(x, w, bias, state, silu=silu)
        _check_conv(x, w, bias, state, silu, None, y, last)
    y, last = gdn.short_conv(x, w, silu=False)
    _check_conv(x, w, None, None, False, None, y, last)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_short_conv_padded_batch(dtype):
    """Sequences of no, one, two, all and out-of-range tokens; what stands
    behind a sequence is neither read nor written."""
    B, T, C, K = 7, 40, 48, 4
    x, w, bias, state = _conv_case(B, T, C, K, dtype, 5)
    x = x.clone()
    lengths = torch.tensor([0, 1, 2, 17, 40, -3, 99], dtype=torch.int32, device="cuda")
    for b, n in enumerate(ref.live(lengths, B, T)):
        x[b, n:] = float("nan")
    out = torch.full((B, T, C), 7.0, dtype=dtype, device="cuda")
    y, last = gdn.short_conv(x, w, bias, state, lengths=lengths, out=out)
    assert y is out
    for b, n in enumerate(ref.live(lengths, B, T)):
        assert (y[b, n:] == 7).all()
        y[b, n:] = 0
    _check_conv(x, w, bias, state, True, lengths, y, last)
    y, _ = gdn.short_conv(x, w, bias, state, lengths=lengths)
    assert all((y[b, n:] == 0).all() for b, n in enumerate(ref.live(lengths, B, T)))


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_short_conv_pieces_equal_one_call(dtype):
    """A sequence in pieces of uneven lengths (a piece shorter than the filter,
    single tokens), the state updated in place: bit for bit the one call."""
    B, T, C, K = 2, 150, 40, 4
    x, w, bias, _ = _conv_case(B, T, C, K, dtype, 6)
    want, last = gdn.short_conv(x, w, bias)
    state = torch.zeros(B, K - 1, C, dtype=dtype, device="cuda")
    t, outs = 0, []
    for n in (1, 2, 1, 70, 0, 3, 73):
        outs.append(gdn.short_conv_step(x[:, t:t + n], w, bias, state))
        t += n
    assert t == T
    assert torch.equal(torch.cat(outs, 1), want) and torch.equal(state, last)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_short_conv_far_values(dtype):
    """Sums far out on both sides of the silu, where its exponential over- and
    underflows."""
    x, w, bias, state = _conv_case(1, 64, 64, 4, dtype, 8)
    x = (x * 60).to(dtype)
    y, last = gdn.short_conv(x, w, bias, state)
    _check_conv(x, w, bias, state, True, None, y, last)


# ------------------------------------------------------------------- the scan
def _ssm_case(B, T, H, G, dk, dv, dtype, seed, dt_type=None, fast=False):
    g = _gen(seed)
    mixed = _randn(g, B, T, H * dv + 2 * G * dk, dtype=dtype)
    v = mixed[..., :H * dv].view(B, T, H, dv)
    k = mixed[..., H * dv:H * dv + G * dk].view(B, T, G, dk)
    q = mixed[..., H * dv + G * dk:].view(B, T, G, dk)
    dt = (_randn(g, B, T, H) - (0.0 if fast else 3.0)).to(dt_type or F32)
    A = -(0.5 + 8 * torch.rand(H, generator=g, device="cuda"))
    return dict(q=q, k=k, v=v, dt=dt, A=A, D=_randn(g, H), dt_bias=0.3 * _randn(g, H),
                state=_randn(g, B, H, dk, dv))


def _ssm_bounds(c, T, o, mag, N):
    """fp32 recurrence: three roundings a state element and token, dk of the
    readout, and the decays' own error (exp and the product d A: 4 steps plus
    |d A| <= 100 of them below e^-100 = 0); a bf16 readout mask and a bf16
    copy of the state add one bf16 rounding of every term of o, a state built
    from a hi/lo pair 2^-16 of its terms."""
    dk = c["q"].shape[-1]
    steps = (3 * T + dk + 110) * U32
    half = HALF[c["q"].dtype]
    if c["q"].dtype == BF16:
        return half * o.abs() + 1.01 * half * mag + 2 * steps * mag, 2.0 ** -16 * N + 2 * steps * N
    return 2 * steps * mag + half * o.abs(), 2 * steps * N


def _check_ssm(c, o, s, lengths=None, **kw):
    a = dict(c, **kw)
    want, ws, mag, N = ref.ssm(a["q"], a["k"], a["v"], a["dt"], a["A"], a["D"], a["dt_bias"], a["state"],
                               a.get("softplus", True), lengths)
    bo, bs = _ssm_bounds(c, c["q"].shape[1], want, mag, N)
    _inside(o, want, bo + 1e-37, "o")
    _inside(s, ws, bs + 1e-37, "state")


@pytest.mark.parametrize("dtype,dt_type", [(F32, F32), (BF16, F32), (BF16, BF16)])
@pytest.mark.parametrize("dk,dv", [(64, 64), (128, 128), (64, 128), (128, 64)])
@pytest.mark.parametrize("T", [1, 2, 17, 127, 128, 129, 300])
def test_ssm_scan(dtype, dt_type, dk, dv, T):
    B, H, G = 2, 6, 2
    c = _ssm_case(B, T, H, G, dk, dv, dtype, T + dk + 2 * dv, dt_type)
    o, s = gdn.ssm_scan(**c)
    _check_ssm(c, o, s)
    none = dict(D=None, dt_bias=None, state=None)
    o, s = gdn.ssm_scan(c["q"], c["k"], c["v"], c["dt"], c["A"])
    _check_ssm(c, o, s, **none)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("H,G", [(1, 1), (3, 1), (4, 4), (5, 5), (7, 1), (8, 2)])
def test_ssm_head_groups(dtype, H, G):
    c = _ssm_case(1, 200, H, G, 64, 64, dtype, 7 * H + G)
    o, s = gdn.ssm_scan(**c)
    _check_ssm(c, o, s)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_ssm_steps_given_directly(dtype):
    """Step sizes without the softplus, zeros among them (a token that neither
    decays nor writes), and decays that clear the state at once."""
    c = _ssm_case(2, 260, 4, 2, 128, 64, dtype, 3)
    g = _gen(4)
    d = torch.rand(2, 260, 4, generator=g, device="cuda") * 0.1
    d[:, 5:9] = 0
    d[:, 50] = 60.0            # e^{-30} and less
    d[:, 128] = 1e4            # zero in fp32
    d[:, 200:] = 0
    c.update(dt=d, dt_bias=None)
    o, s = gdn.ssm_scan(**c, softplus=False)
    _check_ssm(c, o, s, softplus=False)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("T", [1, 60, 300])
def test_ssm_padded_batch(dtype, T):
    B = 6
    c = _ssm_case(B, T, 4, 1, 128, 64, dtype, T)
    lengths = torch.tensor([0, 1, T, T // 2, -1, T + 5], dtype=torch.int32, device="cuda")
    c = {n: t.clone() for n, t in c.items()}
    for b, n in enumerate(ref.live(lengths, B, T)):
        for name in ("q", "k", "v", "dt"):
            c[name][b, n:] = float("nan")
    out = torch.full((B, T, 4, 64), 7.0, dtype=dtype, device="cuda")
    o, s = gdn.ssm_scan(**c, lengths=lengths, out=out)
    for b, n in enumerate(ref.live(lengths, B, T)):
        assert (o[b, n:] == 7).all()
        o[b, n:] = 0
    clean = {n: (torch.nan_to_num(t) if n in ("q", "k", "v", "dt") else t) for n, t in c.items()}
    _check_ssm(clean, o, s, lengths=lengths)
    for b in (0, 4):
        assert torch.equal(s[b], c["state"][b])
    o, _ = gdn.ssm_scan(**c, lengths=lengths)
    assert all((o[b, n:] == 0).all() for b, n in enumerate(ref.live(lengths, B, T)))


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_ssm_pieces_in_place(dtype):
    """A sequence in pieces, the state updated in place, single tokens among
    them; the bounds of one call of the whole length."""
    T = 400
    c = _ssm_case(2, T, 4, 2, 128, 128, dtype, 12)
    state = c["state"].clone()
    t, outs = 0, []
    for n in (1, 1, 2, 130, 0, 256, 9, 1):
        sl = {m: c[m][:, t:t + n] for m in ("q", "k", "v", "dt")}
        outs.append(gdn.ssm_step(sl["q"], sl["k"], sl["v"], sl["dt"], c["A"], state, c["D"], c["dt_bias"]))
        t += n
    assert t == T
    _check_ssm(c, torch.cat(outs, 1), state)


def test_ssm_wide_batch_of_single_tokens():
    c = _ssm_case(200, 1, 8, 1, 128, 64, BF16, 8)
    s = c.pop("state")
    keep = s.clone()
    o = gdn.ssm_step(state=s, **c)
    _check_ssm(dict(c, state=keep), o, s)


# --------------------------------------------------------------------- rotary
def _theta(freqs):
    import math
    t = [(int(p) % 2 ** 64) / 2.0 ** 64 * 2 * math.pi for p in freqs[0].tolist()]
    return torch.tensor(t, dtype=torch.float64, device="cuda"), freqs[1]


def _check_rotary(x, y, pos, freqs, interleaved, scale=1.0):
    theta, axis = _theta(freqs)
    want = ref.rotary(x, pos, theta, axis, interleaved, scale)
    # |cos|, |sin| off by a few fp32 steps of one (angle 2^-26 of a turn,
    # sincospi, the scale), two products and their sum; 64-bit angles of the
    # definition itself: |pos| theta 2^-52
    rot = 2 * theta.shape[0]
    mag = x.double()[..., :rot].abs()
    j = torch.arange(rot // 2, device="cuda")
    i0, i1 = (2 * j, 2 * j + 1) if interleaved else (j, j + rot // 2)
    m = torch.zeros_like(x, dtype=torch.float64)
    pair = mag[..., i0] + mag[..., i1]
    m[..., i0], m[..., i1] = pair, pair
    err = m * abs(scale) * (8 * U32 + float(pos.abs().max()) * 2.0 ** -51)
    _inside(y, want, err + HALF[x.dtype] * (want.abs() + err), "rotary")
    assert torch.equal(y[..., rot:], x[..., rot:])


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("d,rot", [(128, 128), (128, 64), (64, 64), (64, 12), (96, 50), (7, 6), (2, 2)])
@pytest.mark.parametrize("B,T", [(1, 1), (3, 77)])
def test_rotary(dtype, interleaved, d, rot, B, T):
    g = _gen(d + rot + T)
    qkv = _randn(g, B, T, 7, d, dtype=dtype)
    q, k = qkv[:, :, :5], qkv[:, :, 5:]
    freqs, scale = gdn.rotary_freqs(rot, device="cuda")
    for pos in (torch.arange(T, device="cuda").repeat(B, 1),
                torch.randint(-(1 << 31), (1 << 31) - 1, (B, T), generator=g, device="cuda").to(torch.int32)):
        a, b = gdn.rotary(q, k, pos, freqs, interleaved=interleaved, scale=scale)
        _check_rotary(q, a, pos, freqs, interleaved)
        _check_rotary(k, b, pos, freqs, interleaved)
    # in place, both views of one tensor, and q alone
    keep = qkv.clone()
    gdn.rotary(q, k, pos, freqs, interleaved=interleaved, q_out=q, k_out=k)
    assert torch.equal(q, a) and torch.equal(k, b)
    a2, none = gdn.rotary(keep[:, :, :5], None, pos, freqs, interleaved=interleaved)
    assert none is None and torch.equal(a2, a)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_rotary_heads_before_tokens(dtype):
    """[B, heads, T, d] tensors, seen through a transposed view."""
    g = _gen(9)
    x = _randn(g, 2, 7, 33, 64, dtype=dtype)
    q, k = x[:, :4].transpose(1, 2), x[:, 4:].transpose(1, 2)
    pos = torch.arange(33, device="cuda").repeat(2, 1) + 100
    freqs, _ = gdn.rotary_freqs(64, device="cuda")
    a, b = gdn.rotary(q, k, pos, freqs)
    _check_rotary(q, a, pos, freqs, False)
    _check_rotary(k, b, pos, freqs, False)
    gdn.rotary(q, k, pos, freqs, q_out=q, k_out=k)
    assert torch.equal(q, a) and torch.equal(k, b)


def test_rotary_axes_and_scaling():
    g = _gen(11)
    x = _randn(g, 1, 500, 3, 128)
    t = torch.arange(500, device="cuda")[None]
    pos = torch.stack([t // 100, t % 100 // 10, t % 10], -1).contiguous()
    freqs, _ = gdn.rotary_freqs(128, axes=(44, 42, 42), device="cuda")
    for inter in (False, True):
        y, _ = gdn.rotary(x, None, pos, freqs, interleaved=inter)
        _check_rotary(x, y, pos, freqs, inter)
    far = t + (1 << 30)
    freqs, scale = gdn.rotary_freqs(64, scaling="yarn", factor=8.0, original_len=4096, device="cuda")
    y, _ = gdn.rotary(x, None, far, freqs, scale=scale)
    _check_rotary(x, y, far, freqs, False, scale)


def test_rotary_back_and_forth():
    """Turning by -pos undoes turning by pos (what its gradient does)."""
    g = _gen(13)
    x = _randn(g, 2, 50, 4, 128)
    pos = torch.randint(0, 1 << 20, (2, 50), generator=g, device="cuda")
    freqs, _ = gdn.rotary_freqs(128, device="cuda")
    y, _ = gdn.rotary(x, None, pos, freqs)
    z, _ = gdn.rotary(y, None, -pos, freqs)
    # two turns, each within 8 steps of the pair's magnitude (<= sqrt 2 |pair|)
    assert float((z - x).abs().max()) <= 2 * 8 * U32 * 2 * float(x.abs().max()) * 1.5


# ------------------------------------------------------------------- together
def _layer(p, x, conv_state, state, pos, kind):
    """One layer: convolution, rotary positions on q and k, scan, readout gate."""
    B, T = x.shape[:2]
    H, d = p["H"], 64
    y = gdn.short_conv_step(x, p["w"], p["b"], conv_state)
    q, k, v = (y[..., i * H * d:(i + 1) * H * d].view(B, T, H, d) for i in range(3))
    gdn.rotary(q, k, pos, p["freqs"], q_out=q, k_out=k)
    if kind == "selective":
        o = gdn.ssm_step(q, k, v, p["dt"][:, pos[0]], p["A"], state, p["D"])
    else:
        q, k = (z / z.float().norm(dim=-1, keepdim=True).clamp_min(1e-6).to(z.dtype) for z in (q, k))
        o = gdn.step(q.contiguous(), k.contiguous(), v.contiguous(), p["alpha"][:, pos[0]].contiguous(),
                     p["beta"][:, pos[0]].contiguous(), state)
    return gdn.readout_gate(o, p["z"][:, pos[0]].contiguous())


@pytest.mark.parametrize("kind", ["selective", "delta"])
def test_layer_streams_as_one_prompt(kind):
    """A layer of the operators together: a prompt of 200 tokens, and the same
    as a prompt of 150, a call of 40 and ten single tokens."""
    g = _gen(21)
    B, T, H, d = 2, 200, 4, 64
    p = dict(H=H, w=_randn(g, 3 * H * d, 4) * 0.5, b=_randn(g, 3 * H * d) * 0.1,
             freqs=gdn.rotary_freqs(d, device="cuda")[0], dt=_randn(g, B, T, H) - 3,
             A=-torch.rand(H, generator=g, device="cuda") - 0.5, D=_randn(g, H),
             alpha=0.9 + 0.1 * torch.rand(B, T, H, generator=g, device="cuda"),
             beta=torch.rand(B, T, H, generator=g, device="cuda"), z=_randn(g, B, T, H, d))
    x = _randn(g, B, T, 3 * H * d)

    def run(cuts):
        conv_state = torch.zeros(B, 3, 3 * H * d, device="cuda")
        state = torch.zeros(B, H, d, d, device="cuda")
        outs, t = [], 0
        for n in cuts:
            pos = torch.arange(t, t + n, device="cuda").repeat(B, 1)
            outs.append(_layer(p, x[:, t:t + n], conv_state, state, pos, kind))
            t += n
        return torch.cat(outs, 1), state

    a, sa = run([200])
    b, sb = run([150, 40] + [1] * 10)
    # fp32 throughout: two evaluation orders of the same sums; the delta rule's
    # fp32 path is held to 1e-4 of rms by its own tests, once each side, and the
    # readout norm does not enlarge a relative error
    for u, w in ((a, b), (sa, sb)):
        assert float((u - w).abs().max()) <= 2e-4 * float(w.pow(2).mean().sqrt()) * 8


def test_calls_on_another_stream_and_in_a_graph():
    c = _ssm_case(2, 300, 4, 2, 128, 64, BF16, 31)
    x, w, bias, state = _conv_case(2, 300, 64, 4, BF16, 32)
    pos = torch.arange(300, device="cuda").repeat(2, 1)
    freqs, _ = gdn.rotary_freqs(128, device="cuda")

    def all_calls():
        return (*gdn.short_conv(x, w, bias, state), *gdn.rotary(c["q"], c["k"], pos, freqs), *gdn.ssm_scan(**c))

    want = all_calls()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = all_calls()
    side.synchronize()
    assert all(torch.equal(u, v) for u, v in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = all_calls()
    for _ in range(3):
        for u in outs:
            u.fill_(float("nan"))
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(u, v) for u, v in zip(outs, want))


def test_empty_calls():
    c = _ssm_case(2, 4, 4, 2, 128, 64, BF16, 41)
    e = {n: (t[:, :0] if n in ("q", "k", "v", "dt") else t) for n, t in c.items()}
    o, s = gdn.ssm_scan(**e)
    assert o.shape == (2, 0, 4, 64) and torch.equal(s, c["state"])
    x, w, bias, state = _conv_case(2, 4, 64, 4, BF16, 42)
    y, last = gdn.short_conv(x[:, :0], w, bias, state)
    assert y.shape == (2, 0, 64) and torch.equal(last, state)
    y, last = gdn.short_conv(x[:, :0], w)
    assert (last == 0).all()


def test_refusals_of_the_python_calls():
    c = _ssm_case(2, 16, 4, 2, 128, 64, BF16, 51)
    for bad in (dict(A=c["A"].double()), dict(A=c["A"][:3]), dict(D=c["D"].cpu()), dict(k=c["k"].float()),
                dict(state=c["state"][:1]), dict(dt=c["dt"].half()), dict(v=c["v"][:, :, :3]),
                dict(q=c["q"].transpose(-1, -2)), dict(q=c["q"][..., ::2]),
                dict(lengths=torch.zeros(2, dtype=torch.int64, device="cuda"))):
        with pytest.raises(ValueError):
            gdn.ssm_scan(**dict(c, **bad))
    wide = torch.zeros(2, 16, 4 * 64 + 3, dtype=BF16, device="cuda")
    with pytest.raises(gdn.GDNError):                       # rows off 16 bytes
        gdn.ssm_scan(**dict(c, v=wide[..., :256].unflatten(-1, (4, 64))))
    x, w, bias, state = _conv_case(2, 16, 64, 4, BF16, 52)
    for bad in (dict(w=w[:, :1].contiguous()), dict(w=w.bfloat16()), dict(bias=bias[1:]), dict(state=state.float()),
                dict(x=x.half())):
        with pytest.raises(ValueError):
            gdn.short_conv(**dict(dict(x=x, w=w, bias=bias, state=state), **bad))
    with pytest.raises(gdn.GDNError):
        gdn.short_conv(x.expand(2, 16, 64)[:1].expand(2, 16, 64), w)          # rows shared by two sequences
    with pytest.raises(gdn.GDNError):
        gdn.short_conv(x, w, out=x)
    freqs, _ = gdn.rotary_freqs(64, device="cuda")
    q = _randn(_gen(53), 2, 16, 4, 64)
    pos = torch.arange(16, device="cuda").repeat(2, 1)
    for bad in (dict(pos=pos.float()), dict(pos=pos[:1]), dict(q=q[..., :32].contiguous()),
                dict(freqs=freqs.float()), dict(k=q.bfloat16()), dict(k_out=q)):
        with pytest.raises(ValueError):
            gdn.rotary(**dict(dict(q=q, k=None, pos=pos, freqs=freqs), **bad))
    with pytest.raises(gdn.GDNError):
        gdn.rotary(q, q, pos, freqs, q_out=q, k_out=q)
