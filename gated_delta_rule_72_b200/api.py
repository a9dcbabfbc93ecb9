"""Torch-facing wrappers over the C-ABI (device memory and streams only).

`scan_causal`, `scan_bidir` and `step` take CUDA tensors, allocate the output
(and the workspace unless one is passed), and call the library on the
current torch stream.  No arithmetic of the scan happens here.
"""
from __future__ import annotations

import math
from fractions import Fraction

import torch

from . import _lib

_TWO_PI = 2 * Fraction("3.14159265358979323846264338327950288419716939937510")

_F32 = torch.float32
_DT = {torch.float32: _lib.GDN_F32, torch.bfloat16: _lib.GDN_BF16}


def _ptr(t):
    return None if t is None else t.data_ptr()


def _check(t, name, dtype=None, shape=None):
    if not t.is_cuda:
        raise ValueError("%s must be a CUDA tensor (the library has no CPU path)" % name)
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    if dtype is not None and t.dtype != dtype:
        raise ValueError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError("%s must have shape %s, got %s" % (name, tuple(shape), tuple(t.shape)))


def _dims(q, k, v, alpha, beta):
    if q.dtype not in _DT:
        raise ValueError("q must be float32 or bfloat16")
    B, T, H, dk = q.shape
    dv = v.shape[-1]
    _check(q, "q")
    _check(k, "k", q.dtype, (B, T, H, dk))
    _check(v, "v", q.dtype, (B, T, H, dv))
    _check(alpha, "alpha", torch.float32, (B, T, H))
    _check(beta, "beta", torch.float32, (B, T, H))
    return B, T, H, dk, dv, _DT[q.dtype]


def workspace_size(B, T, H, dk, dv, dtype=torch.bfloat16, bidir=False,
                   out_dtype=torch.float32) -> int:
    return int(_lib.gdn_workspace_size(B, T, H, dk, dv, _DT[dtype], _DT[out_dtype],
                                       int(bool(bidir))))


def _out(B, T, H, dv, device, out, out_dtype):
    if out is None:
        return torch.empty((B, T, H, dv), dtype=out_dtype, device=device), _DT[out_dtype]
    if out.dtype not in _DT:
        raise ValueError("out must be float32 or bfloat16")
    _check(out, "out", None, (B, T, H, dv))
    return out, _DT[out.dtype]


def _workspace(nbytes, device, workspace):
    if nbytes == 0:
        return None, 0
    if workspace is None:
        workspace = torch.empty(nbytes, dtype=torch.uint8, device=device)
    elif workspace.numel() * workspace.element_size() < nbytes:
        raise ValueError("workspace too small: %d < %d bytes" % (workspace.numel(), nbytes))
    return workspace, workspace.numel() * workspace.element_size()


def _raise(fn, st):
    if st != 0:
        raise _lib.GDNError(fn, st)


def scan_causal(q, k, v, alpha, beta, state=None, *, return_state=True, out=None,
                out_dtype=torch.float32, state_out=None, workspace=None):
    """Causal scan.  Returns (o, final_state) (final_state None if not asked).
    o is fp32 unless out_dtype (or the dtype of `out`) is bfloat16."""
    B, T, H, dk, dv, dt = _dims(q, k, v, alpha, beta)
    if state is not None:
        _check(state, "state", torch.float32, (B, H, dk, dv))
    o, odt = _out(B, T, H, dv, q.device, out, out_dtype)
    if return_state and state_out is None:
        state_out = torch.empty((B, H, dk, dv), dtype=torch.float32, device=q.device)
    ws, nbytes = _workspace(workspace_size(B, T, H, dk, dv, q.dtype, False, o.dtype), q.device,
                            workspace)
    stream = torch.cuda.current_stream(q.device).cuda_stream
    st = _lib.gdn_scan_causal(_ptr(q), _ptr(k), _ptr(v), _ptr(alpha), _ptr(beta), _ptr(state),
                              _ptr(state_out), _ptr(o), B, T, H, dk, dv, dt, odt, _ptr(ws), nbytes,
                              stream)
    _raise("gdn_scan_causal", st)
    return o, state_out


def scan_bidir(q, k, v, alpha, beta, *, out=None, out_dtype=torch.float32, workspace=None,
               state=None, state_bwd=None, return_states=False):
    """Bidirectional scan (causal + strict reverse readouts, summed in fp32).

    state / state_bwd: initial states ([B,H,dk,dv] fp32) of the causal scan
    (S_0) and of the reverse scan (R_{T+1}); None = zero.  Returns o, or with
    return_states=True (o, S_T, R_1)."""
    B, T, H, dk, dv, dt = _dims(q, k, v, alpha, beta)
    for t, name in ((state, "state"), (state_bwd, "state_bwd")):
        if t is not None:
            _check(t, name, torch.float32, (B, H, dk, dv))
    o, odt = _out(B, T, H, dv, q.device, out, out_dtype)
    ws, nbytes = _workspace(workspace_size(B, T, H, dk, dv, q.dtype, True, o.dtype), q.device,
                            workspace)
    stream = torch.cuda.current_stream(q.device).cuda_stream
    if state is None and state_bwd is None and not return_states:
        st = _lib.gdn_scan_bidir(_ptr(q), _ptr(k), _ptr(v), _ptr(alpha), _ptr(beta), _ptr(o),
                                 B, T, H, dk, dv, dt, odt, _ptr(ws), nbytes, stream)
        _raise("gdn_scan_bidir", st)
        return o
    s_out = s_out_b = None
    if return_states:
        s_out = torch.empty((B, H, dk, dv), dtype=torch.float32, device=q.device)
        s_out_b = torch.empty((B, H, dk, dv), dtype=torch.float32, device=q.device)
    st = _lib.gdn_scan_bidir_states(_ptr(q), _ptr(k), _ptr(v), _ptr(alpha), _ptr(beta), _ptr(state),
                                    _ptr(state_bwd), _ptr(s_out), _ptr(s_out_b), _ptr(o), B, T, H, dk,
                                    dv, dt, odt, _ptr(ws), nbytes, stream)
    _raise("gdn_scan_bidir_states", st)
    return (o, s_out, s_out_b) if return_states else o


def step(q, k, v, alpha, beta, state, *, out=None, out_dtype=torch.float32, workspace=None):
    """One streaming call; `state` ([B,H,dk,dv] fp32) is updated in place."""
    B, T, H, dk, dv, dt = _dims(q, k, v, alpha, beta)
    _check(state, "state", torch.float32, (B, H, dk, dv))
    o, odt = _out(B, T, H, dv, q.device, out, out_dtype)
    ws, nbytes = _workspace(workspace_size(B, T, H, dk, dv, q.dtype, False, o.dtype), q.device,
                            workspace)
    stream = torch.cuda.current_stream(q.device).cuda_stream
    st = _lib.gdn_step(_ptr(q), _ptr(k), _ptr(v), _ptr(alpha), _ptr(beta), _ptr(state), _ptr(o),
                       B, T, H, dk, dv, dt, odt, _ptr(ws), nbytes, stream)
    _raise("gdn_step", st)
    return o


def readout_gate(o, z, gamma=None, eps=1e-6, *, out=None, out_dtype=None):
    """Readout epilogue: y = o / sqrt(mean(o^2 over d_v) + eps) * gamma * sigmoid(z),
    per (b, t, h).  o, z: [B,T,H,dv] (fp32 or bf16); gamma: [dv] fp32 or None.
    y is `out` (may be o or z itself, same dtype) or a new tensor of
    out_dtype (default: o's dtype)."""
    _check(o, "o")
    if o.dtype not in _DT:
        raise ValueError("o must be float32 or bfloat16")
    B, T, H, dv = o.shape
    _check(z, "z", None, (B, T, H, dv))
    if z.dtype not in _DT:
        raise ValueError("z must be float32 or bfloat16")
    if gamma is not None:
        _check(gamma, "gamma", torch.float32, (dv,))
    if out is None:
        out = torch.empty((B, T, H, dv), dtype=out_dtype or o.dtype, device=o.device)
    else:
        _check(out, "out", None, (B, T, H, dv))
    if out.dtype not in _DT:
        raise ValueError("out must be float32 or bfloat16")
    stream = torch.cuda.current_stream(o.device).cuda_stream
    st = _lib.gdn_readout_gate(_ptr(o), _DT[o.dtype], _ptr(z), _DT[z.dtype], _ptr(gamma), float(eps),
                               _ptr(out), _DT[out.dtype], B, T, H, dv, stream)
    _raise("gdn_readout_gate", st)
    return out


def vda_scan(q, k, v, alpha_frame, beta, U, *, bidir=False, state=None, state_bwd=None, return_states=False,
             out=None, out_dtype=torch.float32, workspace=None):
    """Frame-wise delta operator over frames of U tokens (T = F * U):
    S_f = (I + K^T diag(beta) K)^{-1} (alpha_f S_{f-1} + K^T diag(beta) V), read by
    every token of frame f (bidir: plus the reverse scan, read strictly).
    alpha_frame: [B, F, H] fp32; beta: [B, T, H] fp32.  Returns o, or with
    return_states (o, S_F, R_1) (R_1 None unless bidir)."""
    if q.dtype not in _DT:
        raise ValueError("q must be float32 or bfloat16")
    B, T, H, dk = q.shape
    dv = v.shape[-1]
    if U < 1 or T % U != 0:
        raise ValueError("T (%d) must be a multiple of the frame length U (%d)" % (T, U))
    F = T // U
    _check(q, "q")
    _check(k, "k", q.dtype, (B, T, H, dk))
    _check(v, "v", q.dtype, (B, T, H, dv))
    _check(alpha_frame, "alpha_frame", torch.float32, (B, F, H))
    _check(beta, "beta", torch.float32, (B, T, H))
    for t, name in ((state, "state"), (state_bwd, "state_bwd")):
        if t is not None:
            _check(t, name, torch.float32, (B, H, dk, dv))
    o, odt = _out(B, T, H, dv, q.device, out, out_dtype)
    s_out = s_out_b = None
    if return_states:
        s_out = torch.empty((B, H, dk, dv), dtype=torch.float32, device=q.device)
        if bidir:
            s_out_b = torch.empty((B, H, dk, dv), dtype=torch.float32, device=q.device)
    ws, nbytes = _workspace(int(_lib.gdn_vda_workspace_size(B, F, U, H, dk, dv, int(bool(bidir)))), q.device,
                            workspace)
    stream = torch.cuda.current_stream(q.device).cuda_stream
    st = _lib.gdn_vda_scan(_ptr(q), _ptr(k), _ptr(v), _ptr(alpha_frame), _ptr(beta), _ptr(state),
                           _ptr(state_bwd), _ptr(s_out), _ptr(s_out_b), _ptr(o), B, F, U, H, dk, dv,
                           int(bool(bidir)), _DT[q.dtype], odt, _ptr(ws), nbytes, stream)
    _raise("gdn_vda_scan", st)
    return (o, s_out, s_out_b) if return_states else o


# ---------------------------------------------------------------------------
# Operators around the scan: inputs may be views (last dimension contiguous)
# ---------------------------------------------------------------------------
# The calls on single tokens are a few microseconds of device time, so what
# runs on the host before the launch is kept short: each tensor's checks are
# one expression, spelled out only when it fails.
def _view(t, name, dtype, shape, device):
    """`t` is on `device` (a CUDA device), of `dtype` and `shape`, its last
    dimension contiguous."""
    if t.device != device or t.dtype is not dtype or t.shape != shape or (t.stride()[-1] != 1 and shape[-1] > 1):
        _refuse(t, name, dtype, shape, device)


def _dense(t, name, dtype, shape, device):
    if t.device != device or t.dtype is not dtype or t.shape != shape or not t.is_contiguous():
        _refuse(t, name, dtype, shape, device)
        raise ValueError("%s must be contiguous" % name)


def _refuse(t, name, dtype, shape, device):
    if not t.is_cuda:
        raise ValueError("%s must be a CUDA tensor (the library has no CPU path)" % name)
    if t.device != device:
        raise ValueError("%s must be on %s, got %s" % (name, device, t.device))
    if t.dtype != dtype:
        raise ValueError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if tuple(t.shape) != tuple(shape):
        raise ValueError("%s must have shape %s, got %s" % (name, tuple(shape), tuple(t.shape)))
    if shape[-1] > 1 and t.stride(-1) != 1:
        raise ValueError("%s must be contiguous in its last dimension" % name)


def _rows(t, name):
    """The heads of a token are contiguous: [B, T, H, d] with any batch and token stride."""
    if t.shape[2] > 1 and t.stride()[2] != t.shape[3]:
        raise ValueError("%s must have the heads of a token contiguous" % name)


def _cuda(t, name):
    """The device of the call's first tensor, and its dtype's code."""
    if not t.is_cuda:
        raise ValueError("%s must be a CUDA tensor (the library has no CPU path)" % name)
    code = _DT.get(t.dtype)
    if code is None:
        raise ValueError("%s must be float32 or bfloat16" % name)
    return t.device, code


def _on(device, fn, *args):
    """fn(*args) with `device` current."""
    if device.index == torch._C._cuda_getDevice():
        return fn(*args)
    with torch.cuda.device(device):
        return fn(*args)


def _run(name, device, fn, *args):
    """fn(*args, stream) with `device` current, on its current stream."""
    if device.index == torch._C._cuda_getDevice():
        st = fn(*args, torch._C._cuda_getCurrentRawStream(device.index))
    else:
        with torch.cuda.device(device):
            st = fn(*args, torch.cuda.current_stream(device).cuda_stream)
    if st != 0:
        raise _lib.GDNError(name, st)


def _result(out, like, shape, lengths):
    """The output: `out`, or a new tensor, zero behind the sequences of a padded batch."""
    if out is None:
        return like.new_empty(shape) if lengths is None else like.new_zeros(shape)
    _dense(out, "out", like.dtype, shape, like.device)
    return out


def short_conv(x, w, bias=None, state=None, *, silu=True, lengths=None, return_state=True, out=None,
               state_out=None):
    """Short causal convolution over time, one filter per channel:
    y[b,t,c] = act(bias[c] + sum_j w[c,j] x[b,t-(K-1)+j,c]), act = silu or none.

    x: [B,T,C] (fp32 or bf16, any batch and token stride of at least C); w:
    [C,K] fp32, K in 2..4; bias: [C] fp32 or None; state: [B,K-1,C] of x's
    dtype, the inputs before token 0, oldest first (None = zero); lengths: [B]
    int32, tokens of each sequence of a padded batch.  Returns (y, last K-1
    inputs) (the state None if not asked).  A new y is zero behind a sequence's
    end (a fill of the whole of it before the call), a given `out` keeps what
    it held there."""
    dev, dtype = x.device, x.dtype
    code = _DT.get(dtype)
    if x.dim() != 3 or w.dim() != 2:
        raise ValueError("x must be [B, T, C] and w [C, K]")
    B, T, C = shape = x.shape
    K = w.shape[1]
    sshape = (B, K - 1, C)
    if not (code is not None and x.is_cuda and x.stride()[2] == 1 and 2 <= K <= 4 and
            w.device == dev and w.dtype is _F32 and w.shape[0] == C and w.is_contiguous() and
            (bias is None or bias.device == dev and bias.dtype is _F32 and bias.shape == (C,) and
             bias.is_contiguous()) and
            (state is None or state.device == dev and state.dtype is dtype and state.shape == sshape and
             state.is_contiguous())):
        _cuda(x, "x")
        _view(x, "x", dtype, shape, dev)
        _dense(w, "w", _F32, (C, K), dev)
        if not 2 <= K <= 4:
            raise ValueError("w must have 2 to 4 taps, got %d" % K)
        if bias is not None:
            _dense(bias, "bias", _F32, (C,), dev)
        if state is not None:
            _dense(state, "state", dtype, sshape, dev)
    if lengths is not None:
        _dense(lengths, "lengths", torch.int32, (B,), dev)
    y = _result(out, x, shape, lengths)
    if state_out is not None:
        if state_out is not state:
            _dense(state_out, "state_out", dtype, sshape, dev)
    elif return_state:
        state_out = x.new_empty(sshape) if state is None else torch.empty_like(state)
    xst = x.stride()
    _run("gdn_short_conv", dev, _lib.load().gdn_short_conv, x.data_ptr(), xst[0], xst[1], w.data_ptr(),
         None if bias is None else bias.data_ptr(), None if state is None else state.data_ptr(),
         None if state_out is None else state_out.data_ptr(), y.data_ptr(),
         None if lengths is None else lengths.data_ptr(), B, T, C, K, 1 if silu else 0, code)
    return y, state_out


def short_conv_step(x, w, bias, state, *, silu=True, lengths=None, out=None):
    """One streaming call of short_conv (usually T = 1): `state` ([B,K-1,C],
    x's dtype) is updated in place.  Returns y."""
    if state is None:
        raise ValueError("a step needs the state that it updates")
    return short_conv(x, w, bias, state, silu=silu, lengths=lengths, out=out, state_out=state)[0]


def rotary_freqs(rot_dim, *, base=10000.0, scaling="none", factor=1.0, original_len=None, beta_fast=32.0,
                 beta_slow=1.0, axes=None, device="cuda"):
    """Table of the angles of `rotary`: (freqs, scale).

    freqs: int64 [2, rot_dim/2] on `device`: each pair's angle per position as
    a 64-bit fraction of a turn, and the position axis that it follows; scale:
    the factor on the rotated channels (1 but for "yarn").
      theta_j = base^(-2j/rot_dim)
      scaling "linear": theta / factor;  "ntk": base * factor^(rot_dim/(rot_dim-2));
      "yarn" (Peng et al. 2023), factor >= 1: pairs that turn more than beta_fast
      times over original_len positions keep theta, those below beta_slow take
      theta / factor, between them the weight of theta rises linearly with the
      turns, as the paper has it (models trained with a ramp over the pairs'
      numbers differ in the pairs between and need a table of their own);
      scale = 0.1 ln(factor) + 1.
      axes: channels per position axis (even, summing to rot_dim), for instance
      (44, 42, 42) for frame, row and column; axis a of n_a channels has
      theta_j = base^(-2j/n_a)."""
    if rot_dim < 2 or rot_dim % 2:
        raise ValueError("rot_dim must be even and at least 2, got %d" % rot_dim)
    if scaling not in ("none", "linear", "ntk", "yarn"):
        raise ValueError("unknown scaling %r" % (scaling,))
    if not base > 0 or not factor > 0:
        raise ValueError("base and factor must be positive")
    dims = [rot_dim] if axes is None else list(axes)
    if sum(dims) != rot_dim or any(n < 2 or n % 2 for n in dims):
        raise ValueError("axes must be even and sum to rot_dim (%d), got %s" % (rot_dim, dims))
    scale = 1.0
    theta, axis = [], []
    for a, n in enumerate(dims):
        b = float(base)
        if scaling == "ntk":
            if n == 2:
                raise ValueError("ntk scaling needs more than one pair an axis")
            b *= factor ** (n / (n - 2.0))
        for j in range(n // 2):
            th = b ** (-2.0 * j / n)
            if scaling == "linear":
                th /= factor
            elif scaling == "yarn":
                if not factor >= 1:
                    raise ValueError("yarn scaling lengthens a context: factor must be at least 1, got %r" % (factor,))
                if original_len is None or not original_len > 0 or not beta_fast > beta_slow:
                    raise ValueError("yarn scaling needs original_len > 0 and beta_fast > beta_slow")
                ramp = (original_len * th / (2 * math.pi) - beta_slow) / (beta_fast - beta_slow)
                ramp = min(1.0, max(0.0, ramp))
                th = (1.0 - ramp) * th / factor + ramp * th
            theta.append(th)
            axis.append(a)
    if scaling == "yarn":
        scale = 0.1 * math.log(factor) + 1.0
    turns = []
    for th in theta:
        p = int(round(Fraction(th) / _TWO_PI * 2 ** 64)) % 2 ** 64
        turns.append(p - 2 ** 64 if p >= 2 ** 63 else p)
    return torch.tensor([turns, axis], dtype=torch.int64, device=device), scale


def rotary(q, k, pos, freqs, *, interleaved=False, scale=1.0, q_out=None, k_out=None):
    """Rotary positions of q [B,T,Hq,d] and k [B,T,Hk,d] (k may be None) in one
    pass: pair j of every head is turned by pos * theta_j.

    q, k: fp32 or bf16, any strides (last dimension contiguous); pos: [B,T] or
    [B,T,axes], int32 or int64, contiguous; freqs, scale: from rotary_freqs
    (2 * freqs.shape[1] <= d channels are turned, the others pass through);
    interleaved: pairs (2j, 2j+1), else (j, j + rot/2).  q_out / k_out: where
    the results go (q / k itself: in place); new contiguous tensors by default.
    Returns (q', k')."""
    dev, dtype = q.device, q.dtype
    code = _DT.get(dtype)
    if q.dim() != 4 or (k is not None and k.dim() != 4):
        raise ValueError("q and k must be [B, T, heads, d]")
    B, T, Hq, d = shape = q.shape
    kshape = None if k is None else (B, T, k.shape[2], d)
    pshape = pos.shape
    axes = pshape[2] if len(pshape) == 3 else 1
    bits = 64 if pos.dtype is torch.int64 else 32
    pairs = freqs.shape[-1]
    if not (code is not None and q.is_cuda and q.stride()[3] == 1 and
            (k is None or k.device == dev and k.dtype is dtype and k.shape == kshape and k.stride()[3] == 1) and
            pos.device == dev and (bits == 64 or pos.dtype is torch.int32) and pshape[:2] == (B, T) and
            len(pshape) <= 3 and pos.is_contiguous() and
            freqs.device == dev and freqs.dtype is torch.int64 and freqs.shape == (2, pairs) and
            freqs.is_contiguous() and 2 * pairs <= d):
        _cuda(q, "q")
        _view(q, "q", dtype, shape, dev)
        if k is not None:
            _view(k, "k", dtype, kshape, dev)
        if pos.dtype is not torch.int64 and pos.dtype is not torch.int32:
            raise ValueError("pos must be int32 or int64")
        _dense(pos, "pos", pos.dtype, (B, T, axes) if len(pshape) == 3 else (B, T), dev)
        _dense(freqs, "freqs", torch.int64, (2, pairs), dev)
        if 2 * pairs > d:
            raise ValueError("freqs turn %d channels, the heads have %d" % (2 * pairs, d))
    if q_out is None:
        q_out = q.new_empty(shape)
    elif q_out is not q:
        _view(q_out, "q_out", dtype, shape, dev)
    qst, qost = q.stride(), q_out.stride()
    if k is not None:
        if k_out is None:
            k_out = k.new_empty(kshape)
        elif k_out is not k:
            _view(k_out, "k_out", dtype, kshape, dev)
        kst, kost = k.stride(), k_out.stride()
        kargs = (k.data_ptr(), kst[0], kst[1], kst[2], k_out.data_ptr(), kost[0], kost[1], kost[2], kshape[2])
    elif k_out is not None:
        raise ValueError("k_out without k")
    else:
        kargs = (None, 0, 0, 0, None, 0, 0, 0, 0)
    _run("gdn_rotary", dev, _lib.load().gdn_rotary, q.data_ptr(), qst[0], qst[1], qst[2], q_out.data_ptr(),
         qost[0], qost[1], qost[2], Hq, *kargs,
         pos.data_ptr(), bits, axes, freqs.data_ptr(), scale, B, T, d, 2 * pairs, 1 if interleaved else 0, code)
    return q_out, k_out


def ssm_workspace_size(B, T, H, G, dk, dv, dtype=torch.bfloat16, device=None) -> int:
    """Bytes of workspace that ssm_scan needs for these sizes on `device` (a CUDA
    device; the current one by default: the plan goes by its number of SMs)."""
    args = (B, T, H, G, dk, dv, _DT[dtype])
    if device is None:
        return _lib.gdn_ssm_workspace_size(*args)
    device = torch.device(device)
    if device.type != "cuda":
        raise ValueError("device must be a CUDA device, got %s" % device)
    return _lib.gdn_ssm_workspace_size(*args) if device.index is None else \
        _on(device, _lib.gdn_ssm_workspace_size, *args)


def ssm_scan(q, k, v, dt, A, D=None, dt_bias=None, state=None, *, softplus=True, lengths=None, return_state=True,
             out=None, state_out=None, workspace=None):
    """Selective state space scan (the scan without the erase term):
    d_t = softplus(dt_t + dt_bias), S_t = exp(d_t A) S_{t-1} + d_t k_t v_t^T,
    o_t = S_t^T q_t + D v_t.

    q, k: [B,T,G,dk] (G groups, each shared by H/G heads), v: [B,T,H,dv], fp32
    or bf16, any batch and token stride of at least a row (multiples of 16
    bytes); dt: [B,T,H] fp32 or q's dtype, any batch and token stride of at
    least H; A (<= 0, -inf too), D, dt_bias: [H] fp32; state: [B,H,dk,dv] fp32
    (None = zero); lengths: [B] int32, tokens of each sequence of a padded
    batch.  Returns (o, final state) (the state None if not asked), o in q's
    dtype.  A new o is zero behind a sequence's end (a fill of the whole of it
    before the scan), a given `out` keeps what it held there.

    Calls of more than 32 tokens go in chunks (128 tokens of bf16, 64 of fp32,
    where that is faster): there an infinite or NaN value in v reaches earlier
    outputs of its head and chunk too, in single tokens and short calls later
    ones only."""
    dev, dtype = q.device, q.dtype
    code = _DT.get(dtype)
    if q.dim() != 4 or v.dim() != 4 or dt.dim() != 3:
        raise ValueError("q, k must be [B, T, G, dk], v [B, T, H, dv], dt [B, T, H]")
    B, T, G, dk = gshape = q.shape
    H, dv = v.shape[2], v.shape[3]
    oshape, sshape, hshape = (B, T, H, dv), (B, H, dk, dv), (H,)
    qst, kst, vst = q.stride(), k.stride(), v.stride()
    if not (code is not None and q.is_cuda and k.device == dev and v.device == dev and dt.device == dev and
            k.dtype is dtype and v.dtype is dtype and (dt.dtype is _F32 or dt.dtype is dtype) and
            k.shape == gshape and v.shape == oshape and dt.shape == (B, T, H) and G > 0 and H % G == 0 and
            qst[2:] == (dk, 1) and kst[2:] == (dk, 1) and vst[2:] == (dv, 1) and dt.stride()[2] == 1 and
            A.device == dev and A.dtype is _F32 and A.shape == hshape and A.is_contiguous() and
            (D is None or D.device == dev and D.dtype is _F32 and D.shape == hshape and D.is_contiguous()) and
            (dt_bias is None or dt_bias.device == dev and dt_bias.dtype is _F32 and dt_bias.shape == hshape and
             dt_bias.is_contiguous()) and
            (state is None or state.device == dev and state.dtype is _F32 and state.shape == sshape and
             state.is_contiguous())):
        _cuda(q, "q")
        for t, name, shape in ((q, "q", gshape), (k, "k", gshape), (v, "v", oshape)):
            _view(t, name, dtype, shape, dev)
            _rows(t, name)
        if dt.dtype is not _F32 and dt.dtype is not dtype:
            raise ValueError("dt must be float32 or q's dtype")
        _view(dt, "dt", dt.dtype, (B, T, H), dev)
        if G < 1 or H % G:
            raise ValueError("the %d heads of v must be a multiple of the %d groups of q and k" % (H, G))
        for t, name in ((A, "A"), (D, "D"), (dt_bias, "dt_bias")):
            if t is not None:
                _dense(t, name, _F32, hshape, dev)
        if state is not None:
            _dense(state, "state", _F32, sshape, dev)
    if lengths is not None:
        _dense(lengths, "lengths", torch.int32, (B,), dev)
    o = _result(out, q, oshape, lengths)
    if state_out is not None:
        if state_out is not state:
            _dense(state_out, "state_out", _F32, sshape, dev)
    elif return_state:
        state_out = A.new_empty(sshape)
    lib = _lib.load()
    nbytes = _on(dev, lib.gdn_ssm_workspace_size, B, T, H, G, dk, dv, code)
    ws = None
    if nbytes:
        if workspace is not None and (workspace.device != dev or not workspace.is_contiguous()):
            raise ValueError("workspace must be contiguous and on %s" % dev)
        ws, nbytes = _workspace(nbytes, dev, workspace)
        ws = ws.data_ptr()
    dst = dt.stride()
    _run("gdn_ssm_scan", dev, lib.gdn_ssm_scan, q.data_ptr(), qst[0], qst[1], k.data_ptr(), kst[0], kst[1],
         v.data_ptr(), vst[0], vst[1], dt.data_ptr(), dst[0], dst[1], A.data_ptr(),
         None if D is None else D.data_ptr(), None if dt_bias is None else dt_bias.data_ptr(),
         None if state is None else state.data_ptr(), None if state_out is None else state_out.data_ptr(),
         o.data_ptr(), None if lengths is None else lengths.data_ptr(), B, T, H, G, dk, dv, 1 if softplus else 0, code,
         _DT[dt.dtype], ws, nbytes)
    return o, state_out


def ssm_step(q, k, v, dt, A, state, D=None, dt_bias=None, *, softplus=True, lengths=None, out=None,
             workspace=None):
    """One streaming call of ssm_scan (usually T = 1): `state` ([B,H,dk,dv]
    fp32) is updated in place.  Returns o."""
    if state is None:
        raise ValueError("a step needs the state that it updates")
    return ssm_scan(q, k, v, dt, A, D, dt_bias, state, softplus=softplus, lengths=lengths, out=out, state_out=state,
                    workspace=workspace)[0]
