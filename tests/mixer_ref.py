"""64-bit definitions of the operators around the scan (torch float64, the
inputs' device), and bounds of fp32 evaluations of them."""
import torch

U32 = 2.0 ** -24          # half a step of fp32, relative
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}


def live(lengths, B, T):
    return [T] * B if lengths is None else [min(max(int(n), 0), T) for n in lengths]


def conv(x, w, bias, state, silu, lengths=None):
    """(y, last inputs, bound of the fp32 error of y before its rounding)."""
    B, T, C = x.shape
    K = w.shape[1]
    y = torch.zeros(B, T, C, dtype=torch.float64, device=x.device)
    mag = torch.zeros_like(y)
    last = torch.zeros(B, K - 1, C, dtype=torch.float64, device=x.device)
    if state is not None:
        last = state.double().clone()
    for b, n in enumerate(live(lengths, B, T)):
        seq = torch.cat([last[b], x[b, :n].double()])
        for t in range(n):
            y[b, t] = (seq[t:t + K] * w.double().T).sum(0)
            mag[b, t] = (seq[t:t + K] * w.double().T).abs().sum(0)
        if bias is not None:
            y[b, :n] += bias.double()
            mag[b, :n] += bias.double().abs()
        last[b] = seq[seq.shape[0] - (K - 1):]
    # K + 1 roundings of the sum; silu's slope is below 1.1, its own few
    # fp32 operations and the exponential's 2 ulp + |y| 2^-23 stay below
    # (8 + |y|) steps of the value
    err = 1.1 * (K + 1) * U32 * mag
    if silu:
        s = y * torch.sigmoid(y)
        err = err + (8 + y.abs()) * 2 * U32 * s.abs()
        y = s
    return y, last, err


def ssm(q, k, v, dt, A, D, bias, state, softplus, lengths=None):
    """(o, final state, magnitude of o, magnitude of the state): the magnitudes
    are the same recurrence over absolute values."""
    B, T, G, dk = q.shape
    H, dv = v.shape[2], v.shape[3]
    dev = q.device
    S = torch.zeros(B, H, dk, dv, dtype=torch.float64, device=dev)
    if state is not None:
        S = state.double().clone()
    N = S.abs()
    o = torch.zeros(B, T, H, dv, dtype=torch.float64, device=dev)
    mag = torch.zeros_like(o)
    zero = torch.zeros((), dtype=torch.float64, device=dev)
    d = dt.double() + (zero if bias is None else bias.double())
    if softplus:
        d = torch.logaddexp(d, zero)
    a = torch.exp(d * A.double())
    Dd = torch.zeros(H, dtype=torch.float64, device=dev) if D is None else D.double()
    n = torch.tensor(live(lengths, B, T), device=dev)
    rep = H // G
    for t in range(T):
        on = (t < n)
        m4 = on.view(B, 1, 1, 1)
        kt = torch.where(on.view(B, 1, 1), k[:, t].double(), zero).repeat_interleave(rep, 1)
        qt = torch.where(on.view(B, 1, 1), q[:, t].double(), zero).repeat_interleave(rep, 1)
        vt = torch.where(on.view(B, 1, 1), v[:, t].double(), zero)
        at = torch.where(on.view(B, 1), a[:, t], zero + 1)[:, :, None, None]
        u = torch.where(on.view(B, 1), d[:, t], zero)[:, :, None] * vt
        S = torch.where(m4, at * S + kt[..., None] * u[:, :, None], S)
        N = torch.where(m4, at * N + (kt[..., None] * u[:, :, None]).abs(), N)
        ot = (qt[..., None] * S).sum(2) + Dd[:, None] * vt
        om = (qt[..., None].abs() * N).sum(2) + (Dd[:, None] * vt).abs()
        o[:, t] = torch.where(on.view(B, 1, 1), ot, zero)
        mag[:, t] = torch.where(on.view(B, 1, 1), om, zero)
    return o, S, mag, N


def rotary(x, pos, theta, axis, interleaved, scale=1.0):
    """theta, axis: per pair (float64, int64)."""
    rot = 2 * theta.shape[0]
    p = pos if pos.dim() == 3 else pos[..., None]
    ang = p[..., axis].double() * theta
    c, s = (scale * torch.cos(ang))[:, :, None], (scale * torch.sin(ang))[:, :, None]
    out = x.double().clone()
    j = torch.arange(rot // 2, device=x.device)
    i0, i1 = (2 * j, 2 * j + 1) if interleaved else (j, j + rot // 2)
    x0, x1 = x.double()[..., i0], x.double()[..., i1]
    out[..., i0] = x0 * c - x1 * s
    out[..., i1] = x0 * s + x1 * c
    return out
