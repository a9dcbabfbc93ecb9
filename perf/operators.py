"""The token-mixer operators around the gated scan, as a program uses them:
the short causal convolution, the selective state space scan (prompts and
single tokens) and rotary positions.

`run` computes a case in elementary torch operations (`own` false) or through
the library's entry points (`own` true); `exact` computes it in 64 bits from
the operator's definition, token by token.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # q, k and v of the 480p clip (32,760 tokens, 12 heads of 128), convolved in one call
        dict(name="conv_prompt", op="conv", B=1, T=32760, C=4608, K=4, dtype="bf16", silu=True, bias=True,
             ragged=False, state=False, pad=0),
        # fp32 prompts of different lengths in one padded batch, the input a slice of a wider
        # projection whose rows are not 16-byte aligned, state carried in
        dict(name="conv_ragged_f32", op="conv", B=3, T=1021, C=1283, K=3, dtype="f32", silu=False, bias=True,
             ragged=True, state=True, pad=37),
        # one token of 64 streams
        dict(name="conv_token", op="conv", B=64, T=1, C=4352, K=4, dtype="bf16", silu=True, bias=True,
             ragged=False, state=True, pad=0),
        # the 480p clip through one layer: few heads, long walk
        dict(name="scan_prompt", op="scan", B=1, T=32760, H=24, G=1, dk=128, dv=64, dtype="bf16", dt="bf16",
             ragged=False, state=False, gates="default"),
        # the throughput shape: 2.1 M token-heads of d = 128 with fast-forgetting gates
        dict(name="scan_skewed", op="scan", B=4, T=16384, H=32, G=8, dk=128, dv=128, dtype="bf16", dt="f32",
             ragged=False, state=False, gates="fast"),
        # one streaming call of a rollout: 1,560 tokens, the state carried
        dict(name="scan_call", op="scan", B=1, T=1560, H=16, G=2, dk=128, dv=128, dtype="bf16", dt="f32",
             ragged=False, state=True, gates="default"),
        # fp32 prompts of different lengths in one padded batch
        dict(name="scan_ragged_f32", op="scan", B=5, T=777, H=6, G=3, dk=64, dv=64, dtype="f32", dt="f32",
             ragged=True, state=True, gates="default"),
        # one token of 128 streams: the state's traffic
        dict(name="scan_token_batch", op="scan", B=128, T=1, H=32, G=1, dk=128, dv=64, dtype="bf16", dt="bf16",
             ragged=False, state=True, gates="default"),
        # one token of one stream: latency
        dict(name="scan_token", op="scan", B=1, T=1, H=16, G=16, dk=128, dv=128, dtype="f32", dt="f32",
             ragged=False, state=True, gates="default"),
        # q and k of the 480p clip on its frame / row / column grid
        dict(name="rotary_prompt", op="rotary", B=1, T=32760, Hq=12, Hk=12, d=128, rot=128, interleaved=True,
             axes=3, scaling="none", dtype="bf16", far=0),
        # long context: scaled positions past a million, half layout on part of the head, shared keys
        dict(name="rotary_far_f32", op="rotary", B=2, T=4099, Hq=24, Hk=4, d=128, rot=64, interleaved=False,
             axes=1, scaling="yarn", dtype="f32", far=1 << 20),
        # one token of 64 streams
        dict(name="rotary_token", op="rotary", B=64, T=1, Hq=32, Hk=8, d=128, rot=128, interleaved=False,
             axes=1, scaling="none", dtype="bf16", far=30000),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["conv", "scan", "scan", "rotary"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op == "conv":
        K = rng.choice([2, 3, 4])
        C = _log_int(rng, 64, 8192)
        if rng.random() < 0.7:
            C = (C + 7) // 8 * 8
        T = 1 if rng.random() < 0.25 else _log_int(rng, 2, 32768)
        B = _log_int(rng, 1, max(1, min(64, 150000000 // (T * C))))
        while B * T * C > 150000000:
            T = max(1, T // 2)
        return dict(op=op, B=B, T=T, C=C, K=K, dtype=dtype, silu=rng.random() < 0.7, bias=rng.random() < 0.7,
                    ragged=rng.random() < 0.4, state=rng.random() < 0.6, pad=rng.choice([0, 0, 8, 37]))
    if op == "scan":
        G = rng.choice([1, 1, 2, 4, 8])
        H = G * _log_int(rng, 1, max(1, 48 // G))
        dk, dv = rng.choice([64, 128, 128]), rng.choice([64, 64, 128])
        T = 1 if rng.random() < 0.3 else _log_int(rng, 2, 16384 if dtype == "bf16" else 2048)
        cap = 2000000 if dtype == "bf16" else 150000        # token-heads
        B = _log_int(rng, 1, max(1, min(128 if T == 1 else 8, cap // (T * H))))
        while B * T * H > cap:
            T = max(1, T // 2)
        return dict(op=op, B=B, T=T, H=H, G=G, dk=dk, dv=dv, dtype=dtype,
                    dt=dtype if rng.random() < 0.5 else "f32", ragged=rng.random() < 0.4,
                    state=rng.random() < 0.6, gates=rng.choice(["default", "default", "fast"]))
    d = rng.choice([64, 128])
    rot = rng.choice([d, d, d // 2])
    axes = rng.choice([1, 1, 3])
    Hk = rng.choice([1, 2, 4, 8, 12])
    Hq = Hk * rng.choice([1, 2, 4])
    T = 1 if rng.random() < 0.25 else _log_int(rng, 2, 32768)
    B = _log_int(rng, 1, max(1, min(64, 50000000 // (T * (Hq + Hk) * d))))
    while B * T * (Hq + Hk) * d > 100000000:
        T = max(1, T // 2)
    return dict(op=op, B=B, T=T, Hq=Hq, Hk=Hk, d=d, rot=rot, interleaved=rng.random() < 0.5, axes=axes,
                scaling="none" if axes > 1 else rng.choice(["none", "linear", "ntk", "yarn"]), dtype=dtype,
                far=rng.choice([0, 0, 30000, 1 << 20]))


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _lengths(case, g):
    """Lengths of a padded batch: empty, one token, full and between."""
    B, T = case["B"], case["T"]
    n = torch.randint(0, T + 1, (B,), generator=g, device=DEV)
    n[0] = T
    if B > 1:
        n[1] = 0
    if B > 2:
        n[2] = 1
    return n.to(torch.int32)


def _thetas(case):
    """Angle per position of each pair (float64), its axis, and the factor on
    the rotated values."""
    rot, axes = case["rot"], case["axes"]
    base, factor, length = 10000.0, 8.0, 4096
    scale = 1.0
    if axes > 1:
        pairs = rot // 2
        per = [pairs - 2 * (pairs // 3), pairs // 3, pairs // 3]
        th, ax = [], []
        for a, n in enumerate(per):
            th += [base ** (-i / n) for i in range(n)]
            ax += [a] * n
        return np.array(th), ax, scale, per
    j = np.arange(rot // 2, dtype=np.float64)
    s = case["scaling"]
    if s == "ntk":
        base = base * factor ** (rot / (rot - 2.0))
    th = base ** (-2.0 * j / rot)
    if s == "linear":
        th = th / factor
    if s == "yarn":
        turns = length * th / (2 * math.pi)
        ramp = np.clip((turns - 1.0) / (32.0 - 1.0), 0.0, 1.0)
        th = (1 - ramp) * th / factor + ramp * th
        scale = 0.1 * math.log(factor) + 1.0
    return th, [0] * (rot // 2), scale, None


def _rotary_plan(case):
    import gated_delta_rule_72_b200 as gdn
    kw = {}
    if case["axes"] > 1:
        kw["axes"] = [2 * n for n in _thetas(case)[3]]
    elif case["scaling"] != "none":
        kw = dict(scaling=case["scaling"], factor=8.0, original_len=4096)
    return gdn.rotary_freqs(case["rot"], base=10000.0, device=DEV, **kw)


def prepare(case, seed):
    g = torch.Generator(DEV).manual_seed(seed)
    td = DT[case["dtype"]]

    def rand(*shape):
        return torch.randn(*shape, generator=g, device=DEV)

    if case["op"] == "conv":
        B, T, C, K = case["B"], case["T"], case["C"], case["K"]
        wide = rand(B, T, C + case["pad"]).to(td)
        s = dict(case=case, x=wide[:, :, case["pad"]:], w=rand(C, K) / math.sqrt(K),
                 bias=rand(C) * 0.2 if case["bias"] else None,
                 state=rand(B, K - 1, C).to(td) if case["state"] else None,
                 lengths=_lengths(case, g) if case["ragged"] else None)
        if case["ragged"]:
            s["y"] = torch.zeros(B, T, C, dtype=td, device=DEV)   # rows behind a sequence stay zero
        return s
    if case["op"] == "scan":
        B, T, H, G, dk, dv = (case[n] for n in ("B", "T", "H", "G", "dk", "dv"))
        # q, k, v as the activated convolution leaves them, side by side in one tensor
        mixed = torch.nn.functional.silu(rand(B, T, H * dv + 2 * G * dk)).to(td)
        v = mixed[..., :H * dv].view(B, T, H, dv)
        k = mixed[..., H * dv:H * dv + G * dk].view(B, T, G, dk)
        q = mixed[..., H * dv + G * dk:].view(B, T, G, dk)
        lo, hi = (1e-3, 1e-1) if case["gates"] == "default" else (5e-2, 5e-1)
        u = torch.rand(H, generator=g, device=DEV)
        step = torch.exp(math.log(lo) + u * (math.log(hi) - math.log(lo)))
        s = dict(case=case, q=q, k=k, v=v, dt=(0.5 * rand(B, T, H)).to(DT[case["dt"]]),
                 A=-(1.0 + 15.0 * torch.rand(H, generator=g, device=DEV)), D=1.0 + 0.1 * rand(H),
                 dt_bias=step + torch.log(-torch.expm1(-step)),
                 state=0.3 * rand(B, H, dk, dv) if case["state"] else None,
                 state_out=torch.empty(B, H, dk, dv, device=DEV),
                 lengths=_lengths(case, g) if case["ragged"] else None)
        if case["ragged"]:
            s["y"] = torch.zeros(B, T, H, dv, dtype=td, device=DEV)
        return s
    B, T, d = case["B"], case["T"], case["d"]
    qkv = rand(B, T, case["Hq"] + case["Hk"], d).to(td)
    start = torch.randint(0, case["far"] + 1, (B, 1), generator=g, device=DEV) if case["far"] else 0
    t = torch.arange(T, device=DEV)[None] + start + torch.zeros(B, 1, dtype=torch.int64, device=DEV)
    if case["axes"] > 1:
        t = torch.stack([t // 1560, t % 1560 // 52, t % 52], dim=-1)
    s = dict(case=case, q=qkv[:, :, :case["Hq"]], k=qkv[:, :, case["Hq"]:], pos=t.contiguous())
    th, ax, s["scale"], _ = _thetas(case)
    s["theta"] = torch.tensor(th, dtype=torch.float64, device=DEV)
    s["axis"] = torch.tensor(ax, dtype=torch.int64, device=DEV)
    if own:
        s["plan"] = _rotary_plan(case)
    return s


# ---------------------------------------------------------------------------
# plain forms, 32 bits
# ---------------------------------------------------------------------------
def _last_inputs(xp, T, K, lengths):
    """The K-1 inputs before position `length` of each sequence; xp carries
    the K-1 inputs before token 0 in front."""
    B, _, C = xp.shape
    n = torch.full((B,), T, device=xp.device) if lengths is None else lengths.long()
    idx = n[:, None] + torch.arange(K - 1, device=xp.device)[None]
    return torch.gather(xp, 1, idx[:, :, None].expand(B, K - 1, C))


def _plain_conv(s):
    case, x = s["case"], s["x"]
    B, T, C, K = case["B"], case["T"], case["C"], case["K"]
    head = torch.zeros(B, K - 1, C, dtype=x.dtype, device=x.device) if s["state"] is None else s["state"]
    xp = torch.cat([head, x], dim=1)
    y = torch.zeros(B, T, C, device=x.device)
    for j in range(K):
        y = y + xp[:, j:j + T].float() * s["w"][:, j]
    if s["bias"] is not None:
        y = y + s["bias"]
    if case["silu"]:
        y = y * torch.sigmoid(y)
    if s["lengths"] is not None:
        keep = torch.arange(T, device=x.device)[None] < s["lengths"][:, None]
        y = torch.where(keep[:, :, None], y, torch.zeros_like(y))
    return y.to(x.dtype), _last_inputs(xp, T, K, s["lengths"])


def _steps(s):
    """softplus(dt + bias) in 32 bits, zero behind a sequence's end."""
    d = s["dt"].float() + s["dt_bias"]
    d = torch.clamp(d, min=0) + torch.log1p(torch.exp(-d.abs()))
    if s["lengths"] is not None:
        keep = torch.arange(d.shape[1], device=d.device)[None] < s["lengths"][:, None]
        d = torch.where(keep[:, :, None], d, torch.zeros_like(d))
    return d


def _plain_scan(s, Q=64):
    """Chunks of Q tokens: products within a chunk, a walk over the chunks'
    states."""
    case = s["case"]
    B, T, H, G, dk, dv = (case[n] for n in ("B", "T", "H", "G", "dk", "dv"))
    d = _steps(s)
    S = s["state"] if s["state"] is not None else torch.zeros(B, H, dk, dv, device=DEV)
    q, k, v = (s[n].float() for n in ("q", "k", "v"))
    if T == 1:
        kh, qh = (z[:, 0].repeat_interleave(H // G, dim=1) for z in (k, q))
        S = torch.exp(d[:, 0] * s["A"])[:, :, None, None] * S + \
            (d[:, 0, :, None] * kh)[..., None] * v[:, 0, :, None, :]
        y = (S * qh[..., None]).sum(2) + s["D"][:, None] * v[:, 0]
        y = y[:, None]
    else:
        n = (T + Q - 1) // Q
        pad = n * Q - T
        if pad:
            z = lambda t: torch.cat([t, t.new_zeros((B, pad) + t.shape[2:])], dim=1)
            q, k, v, d = z(q), z(k), z(v), z(d)
        q, k = (t.view(B, n, Q, G, dk).transpose(2, 3) for t in (q, k))            # B n G Q dk
        v = v.view(B, n, Q, H, dv).transpose(2, 3)                                 # B n H Q dv
        d = d.view(B, n, Q, H).transpose(2, 3)                                     # B n H Q
        c = torch.cumsum((d * s["A"][:, None]).double(), dim=-1)
        gap = (c[..., :, None] - c[..., None, :]).float()
        low = torch.ones(Q, Q, dtype=torch.bool, device=DEV).tril()
        mask = torch.where(low, torch.exp(torch.where(low, gap, torch.zeros_like(gap))),
                           torch.zeros_like(gap)) * d[..., None, :]
        scores = (q @ k.transpose(-1, -2))[:, :, :, None]                          # B n G 1 Q Q
        mask = (mask.view(B, n, G, H // G, Q, Q) * scores).view(B, n, H, Q, Q)
        y = mask @ v
        del mask, gap, scores
        wv = v * (torch.exp((c[..., -1:] - c).float()) * d)[..., None]
        add = (k.transpose(-1, -2)[:, :, :, None] @ wv.view(B, n, G, H // G, Q, dv)).view(B, n, H, dk, dv)
        del wv
        total = torch.exp(c[..., -1].float())[..., None, None]
        before = torch.empty_like(add)
        for i in range(n):
            before[:, i] = S
            S = total[:, i] * S + add[:, i]
        read = (q[:, :, :, None] @ before.view(B, n, G, H // G, dk, dv)).view(B, n, H, Q, dv)
        y = y + torch.exp(c.float())[..., None] * read + s["D"][:, None, None] * v
        y = y.transpose(2, 3).reshape(B, n * Q, H, dv)[:, :T]
    if s["lengths"] is not None:
        keep = torch.arange(T, device=DEV)[None] < s["lengths"][:, None]
        y = torch.where(keep[:, :, None, None], y, torch.zeros_like(y))
    return y.to(s["v"].dtype), S


def _plain_rotary(s):
    case = s["case"]
    pos = s["pos"] if case["axes"] > 1 else s["pos"][..., None]
    angle = pos[..., s["axis"]].double() * s["theta"]
    cos = (torch.cos(angle) * s["scale"]).float()[:, :, None]
    sin = (torch.sin(angle) * s["scale"]).float()[:, :, None]
    rot, outs = case["rot"], []
    for x in (s["q"], s["k"]):
        xf = x[..., :rot].float()
        if case["interleaved"]:
            a, b = xf[..., 0::2], xf[..., 1::2]
            r = torch.stack([a * cos - b * sin, a * sin + b * cos], dim=-1).flatten(-2)
        else:
            a, b = xf[..., :rot // 2], xf[..., rot // 2:]
            r = torch.cat([a * cos - b * sin, a * sin + b * cos], dim=-1)
        outs.append(torch.cat([r.to(x.dtype), x[..., rot:]], dim=-1))
    return tuple(outs)


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def run(state):
    s, case = state, state["case"]
    if not own:
        return {"conv": _plain_conv, "scan": _plain_scan, "rotary": _plain_rotary}[case["op"]](s)
    import gated_delta_rule_72_b200 as gdn
    if case["op"] == "conv":
        return gdn.short_conv(s["x"], s["w"], s["bias"], s["state"], silu=case["silu"], lengths=s["lengths"],
                              out=s.get("y"))
    if case["op"] == "scan":
        return gdn.ssm_scan(s["q"], s["k"], s["v"], s["dt"], s["A"], s["D"], s["dt_bias"], s["state"],
                            softplus=True, lengths=s["lengths"], out=s.get("y"), state_out=s["state_out"])
    if "plan" not in s:
        s["plan"] = _rotary_plan(case)
    freqs, scale = s["plan"]
    return gdn.rotary(s["q"], s["k"], s["pos"], freqs, interleaved=case["interleaved"], scale=scale)


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------
def work(case):
    e = 4 if case["dtype"] == "f32" else 2
    B, T = case["B"], case["T"]
    if case["op"] == "conv":
        C, K = case["C"], case["K"]
        n = B * T * C
        return {"bytes": 2 * n * e + (1 + case["state"]) * B * (K - 1) * C * e + 4 * C * (K + case["bias"]),
                "flops": 2 * K * n}
    if case["op"] == "scan":
        H, G, dk, dv = (case[n] for n in ("H", "G", "dk", "dv"))
        th = B * T * H
        de = 4 if case["dt"] == "f32" else 2
        return {"bytes": 2 * th * dv * e + 2 * B * T * G * dk * e + th * de +
                (1 + case["state"]) * B * H * dk * dv * 4, "flops": 5 * th * dk * dv}
    n = B * T * (case["Hq"] + case["Hk"]) * case["d"]
    return {"bytes": 2 * n * e + B * T * case["axes"] * 8, "flops": 3 * n}


# ---------------------------------------------------------------------------
# the definitions, 64 bits, token by token
# ---------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    B, T = case["B"], case["T"]
    n = s.get("lengths")
    n = [T] * B if n is None else n.tolist()
    if case["op"] == "conv":
        C, K = case["C"], case["K"]
        y = torch.zeros(B, T, C, dtype=torch.float64, device=DEV)
        last = torch.zeros(B, K - 1, C, dtype=torch.float64, device=DEV)
        for b in range(B):
            if s["state"] is not None:
                last[b] = s["state"][b].double()
            seq = torch.cat([last[b], s["x"][b, :n[b]].double()])
            if n[b]:
                r = (seq.unfold(0, K, 1) * s["w"].double()).sum(-1)         # windows: n C K
                r = r if s["bias"] is None else r + s["bias"].double()
                y[b, :n[b]] = r / (1 + torch.exp(-r)) if case["silu"] else r
            last[b] = seq[seq.shape[0] - (K - 1):]
        return y, last
    if case["op"] == "scan":
        H, G, dk, dv = (case[m] for m in ("H", "G", "dk", "dv"))
        S = torch.zeros(B, H, dk, dv, dtype=torch.float64, device=DEV)
        if s["state"] is not None:
            S += s["state"]
        y = torch.zeros(B, T, H, dv, dtype=torch.float64, device=DEV)
        step = torch.logaddexp(s["dt"].double() + s["dt_bias"].double(), torch.zeros((), dtype=torch.float64,
                                                                                     device=DEV))
        decay = torch.exp(step * s["A"].double())
        live = torch.tensor(n, device=DEV)
        Sg = S.view(B, G, H // G, dk, dv)
        full = min(n) == T
        for t in range(T):
            kt, qt = s["k"][:, t].double(), s["q"][:, t].double()
            vt = s["v"][:, t].double()
            u = (step[:, t, :, None] * vt).view(B, G, H // G, 1, dv)
            new = torch.addcmul(decay[:, t].view(B, G, H // G, 1, 1) * Sg, kt[:, :, None, :, None], u)
            if full:
                Sg = new
                y[:, t] = torch.matmul(qt[:, :, None, None], Sg).view(B, H, dv) + s["D"].double()[:, None] * vt
            else:
                on = (t < live)
                Sg = torch.where(on.view(B, 1, 1, 1, 1), new, Sg)
                o = torch.matmul(qt[:, :, None, None], Sg).view(B, H, dv) + s["D"].double()[:, None] * vt
                y[:, t] = torch.where(on.view(B, 1, 1), o, torch.zeros_like(o))
        return y, Sg.reshape(B, H, dk, dv)
    rot = case["rot"]
    pos = s["pos"].double()
    pos = pos if case["axes"] > 1 else pos[..., None]
    outs = []
    i = torch.arange(rot // 2, device=DEV)
    ia, ib = (2 * i, 2 * i + 1) if case["interleaved"] else (i, i + rot // 2)
    unit = torch.polar(torch.full_like(s["theta"], s["scale"]).expand(B, T, 1, -1),
                       (torch.index_select(pos, 2, s["axis"]) * s["theta"])[:, :, None])
    for x in (s["q"], s["k"]):
        r = x.double()
        z = torch.complex(r[..., ia], r[..., ib]) * unit
        r = r.clone()
        r[..., ia], r[..., ib] = z.real, z.imag
        outs.append(r)
    return tuple(outs)
