"""Where a NaN or an infinity in one operand of the gated scan or of its gradients may go:
what it may not reach is bitwise that of the call without it, on both schedules and for all
kinds of gates and inputs.  Every value stands in a channel of its own, at the first and last
tokens of sequences and around the edges of waves and tiles (28 to 240 tokens).  With 64 empty
sequences behind the others the bounds are searched in memory, and one pass takes its small
workgroups."""
import pytest
import torch

import gated_delta_rule_short_amd as kda
from tests._scan_common import BF, DEV, F32, KINDS, make_scan

pytestmark = pytest.mark.gpu
LENGTHS = [250, 0, 37, 481, 1]
STARTS = [0, 250, 250, 287, 768]
EDGES = [0, 1, 3, 4, 7, 8, 15, 16, 27, 28, 41, 42, 55, 56, 59, 60, 89, 90, 111, 112, 119, 120, 149, 150, 179, 180, 209,
         210, 239, 240, 249]
SPOTS = [t for t in EDGES] + [250, 250 + 15, 250 + 16, 286, 287, 287 + 239, 287 + 240, 287 + 480, 768]
C = 136
VALUES = [float("nan"), float("inf"), float("-inf")]
FORMS = [("one_pass", 0), ("one_pass", 64), ("chained", 0), ("chained", 64)]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    kda.load_library()


def _sequence(t):
    """(first token, end) of the sequence that holds token t."""
    return next((s, s + n) for s, n in zip(STARTS, LENGTHS) if s <= t < s + n)


def _number(first):
    """The sequence with tokens that begins at token `first`."""
    return next(n for n, (s, L) in enumerate(zip(STARTS, LENGTHS)) if s == first and L)


def _channels(i):
    """Channels of spot i: one for each value, spread over both groups of 128."""
    return [(3 * i + k) % C for k in range(3)]


def _planted(t, values):
    """A copy of [T, C] with every value at its spot."""
    t = t.clone()
    for i, at in enumerate(SPOTS):
        for k, c in enumerate(_channels(i)):
            if values[k] is not None:
                t[at, c] = values[k]
    return t


def _planted_state(t, values):
    """A copy of [N, C] with values in channels 8 n .. of sequence n."""
    t = t.clone()
    for n in range(len(LENGTHS)):  # (the empty ones behind them stay)
        for k, v in enumerate(values):
            t[n, 8 * n + k] = v
    return t


def _agree(got, clean, reach, nan, what):
    """Equal outside `reach`, not finite in it (of a NaN: NaN), which `nan` names."""
    assert torch.equal(got[~reach], clean[~reach]), what
    assert not torch.isfinite(got[reach]).any(), what
    assert torch.isnan(got[nan]).all(), what


def _inputs(dtype, gate, empty):
    inp = make_scan(LENGTHS + [0] * empty, C, dtype, gate, seed=31, device=DEV)
    if gate == "log":  # (no gate at which a or b is 0)
        inp["gate"].clamp_(min=-4.0, max=-2.0 ** -8)
    assert len(SPOTS) * 3 <= C and torch.isfinite(inp["x"]).all()
    return inp


def _mask(shape):
    return torch.zeros(shape, dtype=torch.bool, device=DEV), torch.zeros(shape, dtype=torch.bool, device=DEV)


@pytest.mark.parametrize("gate,inputs", KINDS)
@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("schedule,empty", FORMS)
def test_forward(gate, inputs, dtype, schedule, empty):
    inp = _inputs(dtype, gate, empty)

    def call(**kw):
        t = dict(inp, **kw)
        return kda.kda_gated_scan_prefill(t["x"], t["gate"], gate_kind=gate, input_kind=inputs, cu_seqlens=inp["cu"],
                                          state_in=t["state"], state_out=True, schedule=schedule)
    clean = call()
    for name in ("x", "gate", "state"):
        values = [VALUES[0], None, None] if name == "gate" else VALUES  # (an infinite gate is a gate)
        (ro, no), (rs, ns) = _mask((769, C)), _mask((5 + empty, C))
        if name == "state":
            got = call(state=_planted_state(inp["state"], values))
            for n, (s, L) in enumerate(zip(STARTS, LENGTHS)):
                ro[s:s + L, 8 * n:8 * n + 3] = rs[n, 8 * n:8 * n + 3] = True
                no[s:s + L, 8 * n] = ns[n, 8 * n] = True
        else:
            got = call(**{name: _planted(inp[name], values)})
            for i, at in enumerate(SPOTS):
                s, end = _sequence(at)
                for k, c in enumerate(_channels(i)):
                    if values[k] is not None:
                        ro[at:end, c] = rs[_number(s), c] = True
                        if k == 0:
                            no[at:end, c] = ns[_number(s), c] = True
        _agree(got[0], clean[0], ro, no, "o of %s" % name)
        _agree(got[1], clean[1], rs, ns, "state of %s" % name)


@pytest.mark.parametrize("gate,inputs", KINDS)
@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("schedule,empty", FORMS)
def test_backward(gate, inputs, dtype, schedule, empty):
    """d_o and the gate reach their own token and those before it, x the gate's gradient of
    its own token, o that of the token behind it, a state that of its sequence's first one, and
    the final state's gradient the whole sequence."""
    inp = _inputs(dtype, gate, empty)
    gen = torch.Generator().manual_seed(32)
    base = dict(inp, d_o=torch.randn(769, C, generator=gen).to(dtype).to(DEV),
                o=torch.randn(769, C, generator=gen).to(dtype).to(DEV), dstate=torch.randn(5 + empty, C, generator=gen).to(DEV))

    def call(**kw):
        t = dict(base, **kw)
        return kda.kda_gated_scan_backward(
            t["d_o"], t["gate"], t["o"], None if inputs == "plain" else t["x"], gate_kind=gate, input_kind=inputs,
            cu_seqlens=inp["cu"], state_in=t["state"], dstate_out=t["dstate"], dstate_in=True, schedule=schedule)
    clean = call()
    for name in ("d_o", "gate", "o", "x", "state", "dstate"):
        if name == "x" and inputs == "plain":
            continue
        values = [VALUES[0], None, None] if name == "gate" else VALUES
        (rx, nx), (rg, ng), (rs, ns) = _mask((769, C)), _mask((769, C)), _mask((5 + empty, C))

        def mark(reach, nan, rows, c, k):
            reach[rows, c] = True
            if k == 0:
                nan[rows, c] = True
        if name in ("state", "dstate"):
            got = call(**{name: _planted_state(base[name], values)})
            for n, (s, L) in enumerate(zip(STARTS, LENGTHS)):
                for k in range(3):
                    if name == "dstate":
                        mark(rs, ns, n, 8 * n + k, k)
                        mark(rx, nx, slice(s, s + L), 8 * n + k, k)
                    mark(rg, ng, slice(s, s + (L if name == "dstate" else min(L, 1))), 8 * n + k, k)
        else:
            got = call(**{name: _planted(base[name], values)})
            for i, at in enumerate(SPOTS):
                s, end = _sequence(at)
                for k, c in enumerate(_channels(i)):
                    if values[k] is None:
                        continue
                    if name in ("d_o", "gate"):
                        mark(rs, ns, _number(s), c, k)
                        mark(rx, nx, slice(s, at + (name == "d_o")), c, k)
                        if name == "gate" and inputs != "plain":
                            mark(rx, nx, at, c, k)
                        mark(rg, ng, slice(s, at + 1), c, k)
                    elif name == "x":
                        mark(rg, ng, at, c, k)
                    elif at + 1 < end:
                        mark(rg, ng, at + 1, c, k)
        for x, y, reach, nan, what in zip(got, clean, (rx, rg, rs), (nx, ng, ns), ("dx", "dgate", "dstate_in")):
            _agree(x, y, reach, nan, "%s of %s" % (what, name))
