"""The scan's paths on the GPU: long walks cut into segments, fp32 in chunks and
walked, calls that the library is given in odd places of memory or twice at
once."""
import pytest
import torch

import gated_delta_rule_72_b200 as gdn
from tests import mixer_ref as ref
from tests.test_mixer_gpu import BF16, F32, _check_ssm, _conv_case, _gen, _randn, _ssm_case

pytestmark = pytest.mark.gpu


def _kernels(call):
    """Names of the kernels a call launches."""
    gdn.gdn_set_kernel_timing(1)
    gdn.gdn_read_kernel_timing()
    try:
        out = call()
        torch.cuda.synchronize()
        return out, set(gdn.gdn_read_kernel_timing())
    finally:
        gdn.gdn_set_kernel_timing(0)


@pytest.mark.parametrize("H,G,dk,dv", [(4, 1, 128, 64), (3, 1, 64, 64), (2, 2, 128, 128), (4, 2, 64, 128)])
@pytest.mark.parametrize("T", [768, 1000, 1537])
def test_segments(T, H, G, dk, dv):
    """Walks cut into segments: heads that forget within a chunk, heads that
    remember the initial state to the end, and ones between."""
    B = 2
    c = _ssm_case(B, T, H, G, dk, dv, BF16, T + H)
    c["A"] = -torch.tensor([8.0, 1e-4, 0.05, 0.0][:H], device="cuda")
    (o, s), names = _kernels(lambda: gdn.ssm_scan(**c))
    assert names == {"ssm_tail", "ssm_walk"}, names
    _check_ssm(c, o, s)
    # in place: every segment starts from the state as it was
    state = c["state"].clone()
    o2 = gdn.ssm_step(c["q"], c["k"], c["v"], c["dt"], c["A"], state, c["D"], c["dt_bias"])
    assert torch.equal(o2, o) and torch.equal(state, s)


def test_segments_of_a_padded_batch():
    """Sequences that end in the first, a middle and the last segment, at and
    beside the borders of chunks, and one without tokens."""
    T = 1600
    n = [0, 1, 127, 128, 129, 512, 513, 1023, 1599, 1600]
    c = _ssm_case(len(n), T, 2, 1, 128, 64, BF16, 77)
    c = {m: t.clone() for m, t in c.items()}
    for b, k in enumerate(n):
        for m in ("q", "k", "v", "dt"):
            c[m][b, k:] = float("nan")
    lengths = torch.tensor(n, dtype=torch.int32, device="cuda")
    out = torch.full((len(n), T, 2, 64), 7.0, dtype=BF16, device="cuda")
    state = c["state"].clone()
    (o, s), names = _kernels(lambda: gdn.ssm_scan(**dict(c, state=state), lengths=lengths, out=out, state_out=state))
    assert "ssm_tail" in names
    for b, k in enumerate(n):
        assert (o[b, k:] == 7).all()
        o[b, k:] = 0
    clean = {m: (torch.nan_to_num(t) if m in ("q", "k", "v", "dt") else t) for m, t in c.items()}
    _check_ssm(clean, o, s, lengths=lengths)
    assert torch.equal(s[0], c["state"][0])


@pytest.mark.parametrize("B,H,T,path", [(1, 4, 1000, "chunk"), (8, 48, 100, "cols"), (2, 3, 33, "cols"),
                                        (1, 1, 2000, "chunk")])
@pytest.mark.parametrize("dk,dv", [(64, 64), (128, 128), (128, 64), (64, 128)])
def test_fp32_paths(B, H, T, path, dk, dv):
    c = _ssm_case(B, T, H, 1, dk, dv, F32, T + dk)
    c["A"][0] = 0.0                                   # a head that never forgets
    (o, s), names = _kernels(lambda: gdn.ssm_scan(**c))
    assert all(m.startswith("ssm_" + path) for m in names), names
    _check_ssm(c, o, s)


def test_fp32_chunks_of_a_padded_batch():
    T = 700
    n = [0, 1, 63, 64, 65, 699, 700]
    c = _ssm_case(len(n), T, 2, 2, 64, 128, F32, 78)
    c = {m: t.clone() for m, t in c.items()}
    for b, k in enumerate(n):
        for m in ("q", "k", "v", "dt"):
            c[m][b, k:] = float("nan")
    lengths = torch.tensor(n, dtype=torch.int32, device="cuda")
    state = c["state"].clone()
    (o, s), names = _kernels(lambda: gdn.ssm_scan(**dict(c, state=state), lengths=lengths, state_out=state))
    assert "ssm_chunk_out" in names
    clean = {m: (torch.nan_to_num(t) if m in ("q", "k", "v", "dt") else t) for m, t in c.items()}
    _check_ssm(clean, o, s, lengths=lengths)


@pytest.mark.parametrize("T", [1, 20, 200, 900])
def test_outputs_at_16_byte_offsets(T):
    """Outputs, states and inputs that start 16 bytes into an allocation."""
    B, H, dk, dv = 2, 2, 128, 64
    c = _ssm_case(B, T, H, 1, dk, dv, BF16, T)
    want, ws = gdn.ssm_scan(**c)

    def shifted(t, fill=None):
        k = 16 // t.element_size()
        flat = torch.empty(t.numel() + k, dtype=t.dtype, device="cuda")
        v = flat[k:].view(t.shape)
        return v.copy_(t) if fill is None else v.fill_(fill)

    d = {m: shifted(t.contiguous()) if m in ("q", "k", "v", "state") else t for m, t in c.items()}
    o, s = gdn.ssm_scan(**d, out=shifted(want, 7.0), state_out=shifted(ws, 7.0))
    assert torch.equal(o, want) and torch.equal(s, ws)
    x, w, bias, state = _conv_case(B, T, 64, 4, BF16, T)
    yw, lw = gdn.short_conv(x, w, bias, state)
    y, last = gdn.short_conv(shifted(x.contiguous()), w, bias, shifted(state), out=shifted(yw, 7.0))
    assert torch.equal(y, yw) and torch.equal(last, lw)


def test_two_calls_at_once():
    """The same call on two streams, and one graph's calls replayed beside
    eager ones, each with its own workspace."""
    c = _ssm_case(1, 1600, 8, 1, 128, 64, BF16, 5)
    f = _ssm_case(1, 700, 4, 1, 64, 64, F32, 6)
    want, fw = gdn.ssm_scan(**c), gdn.ssm_scan(**f)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        g = gdn.ssm_scan(**c), gdn.ssm_scan(**f)
    streams = [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    outs = []
    for _ in range(4):
        for st in streams[:2]:
            with torch.cuda.stream(st):
                outs.append((gdn.ssm_scan(**c), gdn.ssm_scan(**f)))
        with torch.cuda.stream(streams[2]):
            graph.replay()
    torch.cuda.synchronize()
    for a, b in outs + [g]:
        assert torch.equal(a[0], want[0]) and torch.equal(a[1], want[1])
        assert torch.equal(b[0], fw[0]) and torch.equal(b[1], fw[1])


def test_results_do_not_change_from_run_to_run():
    c = _ssm_case(2, 1500, 6, 2, 128, 64, BF16, 9)
    o, s = gdn.ssm_scan(**c)
    for _ in range(5):
        o2, s2 = gdn.ssm_scan(**c)
        assert torch.equal(o, o2) and torch.equal(s, s2)


def test_workspace_given_by_the_caller():
    c = _ssm_case(1, 900, 4, 1, 128, 64, BF16, 10)
    need = gdn.ssm_workspace_size(1, 900, 4, 1, 128, 64)
    assert need > 0
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    o, s = gdn.ssm_scan(**c, workspace=ws)
    _check_ssm(c, o, s)
    with pytest.raises(ValueError):
        gdn.ssm_scan(**c, workspace=ws[:-1])
    with pytest.raises(ValueError):
        gdn.ssm_scan(**c, workspace=torch.empty(need, dtype=torch.uint8))
    with pytest.raises(gdn.GDNError):
        gdn.ssm_scan(**c, workspace=torch.empty(need + 16, dtype=torch.uint8, device="cuda")[16:])


def test_large_values_stay_in_range():
    """Values, keys and queries far outside 16-bit floating point's other
    format: nothing saturates before the products do."""
    c = _ssm_case(1, 300, 2, 1, 128, 64, BF16, 11)
    c["k"] = c["k"] * 1e6
    c["v"] = c["v"] * 1e6
    c["q"] = c["q"] * 1e-6
    o, s = gdn.ssm_scan(**c)
    _check_ssm(c, o, s)


def test_heads_shared_by_a_group_match_heads_of_their_own():
    """q and k of a group given once, or repeated for each of its heads."""
    c = _ssm_case(2, 500, 6, 2, 64, 64, F32, 12)
    a = gdn.ssm_scan(**c)
    own = dict(c, q=c["q"].repeat_interleave(3, 2), k=c["k"].repeat_interleave(3, 2))
    b = gdn.ssm_scan(**own)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("B,T,H", [(1, 385, 1), (3, 512, 2), (1, 513, 4), (1, 5001, 1)])
def test_segments_of_one_and_of_few_chunks(B, T, H):
    """The shortest walks that are cut, and one head's long one, whose segments
    remember every segment before them."""
    c = _ssm_case(B, T, H, 1, 128, 128, BF16, T)
    c["A"] = -torch.tensor([1e-4, 8.0, 0.0, 0.05][:H], device="cuda")
    (o, s), names = _kernels(lambda: gdn.ssm_scan(**c))
    assert names == {"ssm_tail", "ssm_walk"}, names
    _check_ssm(c, o, s)
