"""Long memories of the gated scan: steady gates over tens of thousands of tokens, forward,
backward and in single steps, within bounds that a rounded decay would break (shown on the
CPU in test_scan_precision_host).  Bounds: _scan_memory."""
import pytest
import torch

import gated_delta_rule_short_amd as kda
from tests._scan_common import BF, DEV, F32, KINDS, U32, check, half_step, make_scan
from tests._scan_memory import GATES, TOKENS, filled, input_factor, slack, steady, step_slack

pytestmark = pytest.mark.gpu
C = 136  # two groups of channels, the second not full


@pytest.fixture(scope="module", autouse=True)
def _lib():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    kda.load_library()


@pytest.mark.parametrize("gate,inputs", KINDS)
@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("schedule", ["one_pass", "chained"])
def test_steady_gates_forward(gate, inputs, dtype, schedule):
    g = torch.full((TOKENS, C), GATES[gate], dtype=dtype, device=DEV)
    x = torch.ones(TOKENS, C, dtype=dtype, device=DEV)
    assert float(g[0, 0]) == GATES[gate]
    o, state = kda.kda_gated_scan_prefill(x, g, gate_kind=gate, input_kind=inputs, state_out=True, schedule=schedule)
    _, a, c = steady(gate)
    at = torch.tensor([0, 1, 100, 5000, 20000, TOKENS - 1])
    want = (input_factor(a, c, inputs) * filled(gate, at + 1))[:, None].expand(-1, C)
    check(o[at], want, (slack(gate, False) + half_step(dtype)) * want, "o")
    check(state, want[-1:], slack(gate, False) * want[-1:], "state")


@pytest.mark.parametrize("gate,inputs", KINDS)
@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("schedule", ["one_pass", "chained"])
def test_steady_gates_backward(gate, inputs, dtype, schedule):
    """d_o of ones: dh_t = 1 + a + .. over the tokens behind t; with 2 for every state
    dgate = dh a' (2 - q), q = -db/da."""
    fill = lambda v: torch.full((TOKENS, C), v, dtype=dtype, device=DEV)
    x = None if inputs == "plain" else fill(1.0)
    dx, dg, ds = kda.kda_gated_scan_backward(
        fill(1.0), fill(GATES[gate]), fill(2.0), x, gate_kind=gate, input_kind=inputs,
        state_in=torch.full((1, C), 2.0, device=DEV), dstate_in=True, schedule=schedule)
    _, a, c = steady(gate)
    b = input_factor(a, c, inputs)
    q = {"plain": 0.0, "complement": 1.0, "norm": float(a / b)}[inputs]
    slope = float(a if gate == "log" else a * c)
    at = torch.tensor([0, 1, 20000, TOKENS - 5000, TOKENS - 100, TOKENS - 1])
    dh = filled(gate, TOKENS - at)[:, None].expand(-1, C)
    tol = slack(gate, True)
    check(dx[at], b * dh, (tol + half_step(dtype)) * b * dh, "dx")
    want = dh * slope * (2.0 - q)
    check(dg[at], want, half_step(dtype) * want.abs() + tol * dh * slope * (2.0 + q), "dgate")
    check(ds, a * dh[:1], tol * a * dh[:1], "dstate_in")


@pytest.mark.parametrize("gate", ["log", "sigmoid"])
def test_steady_gates_in_single_steps(gate):
    """400 tokens without an input, states of random digits: the mean decay is the gate's own
    and not that of its fp32 rounding, which would be off by 200 u32."""
    steps, gen = 400, torch.Generator().manual_seed(1)
    h = (1.0 + torch.rand(4, 8192, generator=gen)).to(DEV)
    first = h.double()
    x, g = torch.zeros(4, 8192, device=DEV), torch.full((4, 8192), GATES[gate], device=DEV)
    for _ in range(steps):
        kda.kda_gated_scan_decode(x, g, h, gate_kind=gate)
    drift = float((h.double() / first).mean() * torch.exp(-steps * steady(gate)[0]) - 1.0)
    assert abs(drift) <= step_slack(gate, steps, h.numel()), drift


@pytest.mark.parametrize("gate,inputs", KINDS)
def test_long_chains_repeat(gate, inputs):
    """Bitwise the same from run to run, and a sequence of a batch as on its own."""
    inp = make_scan([9000, 3, 1000], 264, F32, gate, seed=18, device=DEV)
    kw = dict(gate_kind=gate, input_kind=inputs, schedule="chained")
    o, state = kda.kda_gated_scan_prefill(inp["x"], inp["gate"], cu_seqlens=inp["cu"], state_in=inp["state"],
                                          state_out=True, **kw)
    for _ in range(3):
        o2, state2 = kda.kda_gated_scan_prefill(inp["x"], inp["gate"], cu_seqlens=inp["cu"], state_in=inp["state"],
                                                state_out=True, **kw)
        assert torch.equal(o, o2) and torch.equal(state, state2)
    o3, state3 = kda.kda_gated_scan_prefill(inp["x"][:9000], inp["gate"][:9000], state_in=inp["state"][:1].contiguous(),
                                            state_out=True, **kw)
    assert torch.equal(o3, o[:9000]) and torch.equal(state3, state[:1])


def test_a_bf16_state_is_rounded_at_every_step():
    """Steps of less than half a bf16 step leave the state, which the same steps in one
    prompt, rounded once, move; steps of more than half a step move it."""
    for gate, moves in ((-2.0 ** -10, False), (-2.0 ** -7, True)):
        g, x = torch.full((64, 8), gate, device=DEV), torch.zeros(64, 8, device=DEV)
        h = torch.ones(1, 8, dtype=BF, device=DEV)
        for t in range(64):
            kda.kda_gated_scan_decode(x[t:t + 1], g[t:t + 1], h)
        assert (h != 1.0).all() if moves else (h == 1.0).all()
        _, once = kda.kda_gated_scan_prefill(x, g, state_in=torch.ones(1, 8, dtype=BF, device=DEV), state_out=True)
        want = torch.exp(torch.tensor(64.0 * gate, dtype=torch.float64)).expand(1, 8)
        check(once, want, (half_step(BF) + 200 * U32) * want, "one prompt")
