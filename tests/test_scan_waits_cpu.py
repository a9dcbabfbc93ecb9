"""Order of the waits in the tensor-core scan's kernels, without a GPU.

A wait on an mbarrier names a phase by its parity, so it is only sound where
the phase after the awaited one cannot complete before the waiter has looked:
else the barrier seems not to have moved and the wait runs out.  The roles of
each kernel are written below as the lists of their waits, arrivals, loads
and commits, in C expressions that the kernel's source has to hold in the same order;
each role is then held back at each of its steps while the others run as far as
they can (what can run never stops what else can, so that state is unique), and
no phase may go by."""
import os
import re
from collections import Counter

import pytest

SRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "gated_delta_rule_72_b200", "csrc",
                   "ssm_tc.cuh")

# An operation: (kind, barrier, phase or None, condition or None).  kinds: wait,
# arrive, load (arrives when the copy has landed), commit (when the products before have).
# A "loop" holds operations repeated over a range.
def _w(bar, phase, cond=None):
    return ("wait", bar, phase, cond)


def _a(bar, cond=None):
    return ("arrive", bar, None, cond)


def _l(bar, arg, cond=None):
    return ("load", bar, arg, cond)


def _c(bar, cond=None):
    return ("commit", bar, None, cond)


WALK = {
    "loads": [_w("r_done", "c", "c + 1 < nch"), _l("q_full", "c + 1", "c + 1 < nch"),
              _w("k_free[c & 1]", "c >> 1", "c + 2 < nch"), _l("k_full", "c + 2", "c + 2 < nch"),
              _w("y_staged[c & 1]", "c >> 1"), _l("x_full", "c + 2", "c + 2 < nch")],
    "mma": [_w("q_full", "c"), _w("k_full[c & 1]", "c >> 1"), _w("fixed", "0", "partial"),
            _w("y_full", "c - 1", "c > 0"), _c("g_full"), _w("ds_free", "c"),
            ("loop", "q", 4, [_w("y_free", "c - 1", "q == 1 and c > 0"), _w("s_ready", "c", "q == 1"),
                              _c("r_done", "q == 1"),
                              _w("wx_ready[q & 1]", "wph >> 1"), _c("wx_free[q & 1]")]),
            _c("s_full"), _c("k_free[c & 1]"), _w("m_ready", "c"), _c("y_full")],
    "tables": [_w("tab_free[c & 1]", "(c >> 1) - 1", "c >= 2"), _a("tab_full[c & 1]")],
    "output": [_w("tab_full[c & 1]", "c >> 1"), _w("g_full", "c"), _a("tab_free[c & 1]"), _w("r_done", "c"),
               _a("m_ready"), _w("y_full", "c"), _a("y_free"), _a("y_staged[c & 1]")],
    "weights": [_w("tab_full[c & 1]", "c >> 1"), _w("x_full[c & 1]", "c >> 1"), _w("k_full[c & 1]", "c >> 1", "partial"),
                _a("fixed", "partial"), _w("fixed", "0", "partial"),
                ("loop", "q", 4, [_w("wx_free[q & 1]", "use - 1", "use >= 1"), _a("wx_ready[q & 1]")]),
                _a("tab_free[c & 1]")],
    "state": [_w("s_full", "c - 1", "c > 0"), _a("ds_free"), _w("r_done", "c - 1", "c > 0"), _a("s_ready"),
              _w("tab_full[c & 1]", "c >> 1"), _a("tab_free[c & 1]")],
}
# members of each role, as far as they tell apart: two stand for more
WALK_ROLES = {"loads": 1, "mma": 1, "tables": 2, "output": 2, "weights": 2, "state": 2}
WALK_SECTIONS = ["loads and stores", "MMA issue", "decay tables", "M and the output", "weighted values", "the state"]

TAIL = {
    "loads": [_w("freed[i % kTailStages]", "i / kTailStages - 1", "i >= kTailStages"), _l("full", "i")],
    "mma": [_w("full[st]", "i / kTailStages"), _w("wx_ready[i & 1]", "i >> 1"),
            _w("s_free", "i - 1", "i > 0"), _c("freed[st]"), _c("wx_free[i & 1]"), _c("s_full")],
    "gates": [_w("w_free[i & 1]", "(i >> 1) - 1", "i >= 2"), _a("w_full[i & 1]")],
    # (goes one step further than the others)
    "weights": [_w("w_full[i & 1]", "i >> 1", "i < steps"), _w("full[st]", "i / kTailStages", "i < steps"),
                _a("w_free[i & 1]", "i < steps"), _w("wx_free[i & 1]", "(i >> 1) - 1", "2 <= i < steps"),
                _a("wx_ready[i & 1]", "i < steps"), _w("s_full", "i - 1", "i > 0"), _a("s_free", "i > 0")],
}
TAIL_ROLES = {"loads": 1, "mma": 1, "gates": 2, "weights": 2}


def _flat(ops):
    for op in ops:
        if op[0] == "loop":
            yield from _flat(op[3])
        else:
            yield op


def _norm(s):
    return re.sub(r"\s+", "", s)


def _source_ops(text):
    """(kind, barrier, phase) of every operation, in the order of the source."""
    names = {"load_q": "q_full", "load_k": "k_full", "load_x": "x_full", "load": "full"}
    out = []
    for m in re.finditer(r"\b(wait|mbar_arrive|mma_commit|load_[qkx]|load)\(&?(\w+(?:\[[^\]]*\])?[^,;{]*?)"
                         r"(?:, ((?:[^()]|\([^()]*\))*?))?\)(?=[;)\s|&])", text):
        kind, a, b = m.groups()
        if kind in names:
            out.append(("load", names[kind], _norm(a)))
        else:
            out.append((dict(wait="wait", mbar_arrive="arrive", mma_commit="commit")[kind], _norm(a),
                        _norm(b) if b else None))
    return out


def _kernel(name):
    with open(SRC) as f:
        text = re.sub(r"//[^\n]*", lambda m: m.group(0) if "====" in m.group(0) else "", f.read())
    start = text.index("\n" + name + "(")
    return text[start:text.index("\ntemplate", start) if "\ntemplate" in text[start:] else len(text)]


def _model_ops(ops):
    return [(k, _norm(b), _norm(p) if p else None) for k, b, p, _ in _flat(ops)]


def test_walk_source_has_the_modelled_order():
    text = _kernel("walk_kernel")
    heads = [text.index("= " + s + " =") for s in WALK_SECTIONS] + [text.index("if (last && p.a.state_out && nch > 0")]
    for (role, ops), a, b in zip(WALK.items(), heads, heads[1:]):
        assert _source_ops(text[a:b]) == _model_ops(ops), role


def test_tail_source_has_the_modelled_order():
    text = _kernel("tail_kernel")
    cuts = [text.index(s) for s in ("if (warp == 16)", "else if (warp == 17)", "else if (warp >= 18)",
                                    "const int q = warp >> 2, xcol")] + [text.index("if (ok && v < W)")]
    for (role, ops), a, b in zip(TAIL.items(), cuts, cuts[1:]):
        assert _source_ops(text[a:b]) == _model_ops(ops), role


class _Run:
    """Programs of flat operations over barriers, run in any order."""

    def __init__(self, programs, counts, started):
        self.programs, self.counts = programs, counts
        self.pc = {r: 0 for r in programs}
        self.done = Counter()             # completed phases of a barrier
        self.pending = Counter()
        for bar in started:
            self._arrive(bar)

    def _arrive(self, bar):
        self.pending[bar] += 1
        if self.pending[bar] == self.counts.get(bar, 1):
            self.pending[bar] = 0
            self.done[bar] += 1

    def step(self, role):
        ops, i = self.programs[role], self.pc[role]
        if i == len(ops):
            return False
        kind, bar, phase = ops[i]
        if kind == "wait":
            if self.done[bar] <= phase:
                return False
        else:
            self._arrive(bar)             # (copies and products land at once: the latest a waiter can be, the worst)
        self.pc[role] += 1
        return True

    def settle(self, held=None):
        while any([self.step(r) for r in self.programs if r != held]):
            pass

    def missed(self, role):
        """A phase that `role` still has to see and that another one has followed."""
        seen = set()
        for kind, bar, phase in self.programs[role][self.pc[role]:]:
            if kind == "wait" and bar not in seen:
                seen.add(bar)
                if self.done[bar] > phase + 1:
                    return bar, phase
        return None


def _programs(model, roles, n, partial, consts):
    def expand(ops, env):
        for op in ops:
            if op[0] == "loop":
                for q in range(op[2]):
                    c = env["c"]
                    yield from expand(op[3], dict(env, q=q, wph=4 * c + q, use=2 * c + (q >> 1)))
                continue
            kind, bar, phase, cond = op
            if cond and not eval(cond, {}, env):
                continue
            m = re.match(r"(\w+)\[(.*)\]$", bar)
            at = (m[1], eval(m[2], {}, env)) if m else (bar, 0)
            if kind == "load":
                v = eval(phase, {}, env)
                yield kind, (bar, v % consts["slots"].get(bar, 1)), None
            else:
                yield kind, at, None if phase is None else eval(phase.replace("/", "//"), {}, env)

    out = {}
    for role, count in roles.items():
        for i in range(count):
            ops = []
            for c in range(n + consts.get("further", {}).get(role, 0)):
                env = dict(c=c, i=c, nch=n, steps=n, partial=partial and c == n - 1, kTailStages=3, st=c % 3)
                ops += expand([o for o in model[role] if not (o[0] == "load" and o[1] == "full" and c == 0)], env)
            out[role, i] = ops
    return out


def _walk(n, partial, model=WALK):
    slots = dict(x_full=2, k_full=2)
    programs = _programs(model, WALK_ROLES, n, partial, dict(slots=slots))
    two = {("m_ready", 0): 2, ("y_free", 0): 2, ("s_ready", 0): 2, ("ds_free", 0): 2,
           ("fixed", 0): 2}
    for s in (0, 1):
        two.update({("y_staged", s): 2, ("wx_ready", s): 2, ("tab_full", s): 2, ("tab_free", s): 6})
    started = [("k_full", 0), ("q_full", 0), ("x_full", 0)] + ([("k_full", 1), ("x_full", 1)] if n > 1 else [])
    return lambda: _Run(programs, two, started)


def _tail(n, model=TAIL):
    programs = _programs(model, TAIL_ROLES, n, False, dict(slots=dict(full=3), further=dict(weights=1)))
    two = {("s_free", 0): 2}
    for s in (0, 1):
        two.update({("w_full", s): 2, ("w_free", s): 2, ("wx_ready", s): 2})
    return lambda: _Run(programs, two, [("full", 0)])


def _faults(make):
    """Phases that go by while one member of a role is held at one of its steps."""
    run = make()
    run.settle()
    stuck = {r: run.programs[r][run.pc[r]] for r in run.programs if run.pc[r] < len(run.programs[r])}
    assert not stuck, stuck
    bad = []
    for role, ops in run.programs.items():
        for stop in range(len(ops)):
            r = make()
            while r.pc[role] < stop:      # the role is never ahead of where it is held
                if not r.step(role):
                    for other in r.programs:
                        if other != role:
                            r.step(other)
            r.settle(held=role)
            if r.missed(role):
                bad.append((role, stop, r.missed(role)))
    return bad


@pytest.mark.parametrize("partial", [False, True])
@pytest.mark.parametrize("n", [1, 2, 3, 4, 7])
def test_walk_waits_see_every_phase(n, partial):
    assert not _faults(_walk(n, partial))


@pytest.mark.parametrize("n", [1, 2, 3, 5, 8])
def test_tail_waits_see_every_phase(n):
    assert not _faults(_tail(n))


def test_one_barrier_for_both_output_tiles_would_not_do():
    """The check finds what it is for: with one barrier for the output tiles of
    both slots, chunk c + 1 can finish before the storing warp looks at chunk c's."""
    one = dict(WALK)
    one["loads"] = [_w("y_staged", "c") if op[1].startswith("y_staged") else op for op in WALK["loads"]]
    one["output"] = [_a("y_staged") if op[1].startswith("y_staged") else op for op in WALK["output"]]
    programs = _programs(one, WALK_ROLES, 4, False, dict(slots=dict(x_full=2, k_full=2)))
    base = _walk(4, False)()
    counts = dict(base.counts)
    counts["y_staged", 0] = 2
    started = [("k_full", 0), ("q_full", 0), ("x_full", 0), ("k_full", 1), ("x_full", 1)]
    bad = _faults(lambda: _Run(programs, counts, started))
    assert {b[2][0][0] for b in bad} == {"y_staged"} and {b[0][0] for b in bad} == {"loads"}, bad


# ---- a kernel that gives up: what is in flight lands before it returns
def _drains(text):
    """(barrier, uses) of every wait of a kernel's way out."""
    return re.findall(r"mbar_drain\(&?(\w+(?:\[s\]| \+ i)?), ((?:[^()]|\([^()]*\))*)\);", text)


def _cols_source():
    with open(os.path.join(os.path.dirname(SRC), "ssm_cols.cuh")) as f:
        return f.read()


def _uses(drains, bar, **env):
    expr = dict(drains)[bar].replace("/", "//")
    return eval(expr, {}, env)


def test_no_wait_of_the_way_out_names_a_fixed_phase():
    """The phase of a copy in flight depends on how many there were before it."""
    for text in (_kernel("walk_kernel"), _kernel("tail_kernel"), _cols_source()):
        assert not re.findall(r"\bmbar_wait(?:_ns)?\([^;]*?, 0, ", text)
        assert _drains(text)


def test_the_way_out_waits_for_the_last_load_of_every_slot():
    walk, tail, cols = _drains(_kernel("walk_kernel")), _drains(_kernel("tail_kernel")), _drains(_cols_source())
    assert {b for b, _ in walk} == {"q_full", "k_full[s]", "x_full[s]"}
    assert "if (*abort_s) drain_products(drained);" in _kernel("walk_kernel")
    assert "if (*abort_s) drain_products(drained);" in _kernel("tail_kernel")
    assert {b for b, _ in tail} == {"full[s]"} and {b for b, _ in cols} == {"full + i"}
    for n in range(12):
        assert _uses(walk, "q_full", nq=n) == n
        for s in range(2):
            want = len([c for c in range(n) if c % 2 == s])
            assert _uses(walk, "k_full[s]", nk=n, s=s) == want and _uses(walk, "x_full[s]", nx=n, s=s) == want
        for s in range(3):
            assert _uses(tail, "full[s]", issued=n, kTailStages=3, s=s) == len([c for c in range(n) if c % 3 == s])
        for s in range(4):
            assert _uses(cols, "full + i", issued=n, kStages=4, i=s) == len([c for c in range(n) if c % 4 == s])


def test_threads_of_a_block_agree_that_a_wait_gave_up():
    """What each thread's wait came to is joined by the barrier itself: a flag
    read behind it could be raised by a thread that is a step ahead."""
    assert "__syncthreads_or" in _cols_source()
