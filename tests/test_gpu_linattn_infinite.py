"""Infinities in the linear attention's returned states: what the recurrence keeps as an
infinity (or turns into NaN) comes back as such from prompts, from segments and from
single tokens alike, and every other element keeps its bound.  Decays are mild here:
behind a decay that rounds to zero an infinity becomes NaN."""
import pytest
import torch

import gated_delta_rule_short_amd as kda
from tests._linattn_common import DEV, U16, U32, TINY, check, check_linattn, half_step, linattn_ref, make_linattn

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
INF = float("inf")


@pytest.fixture(scope="module", autouse=True)
def _lib():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    kda.load_library()


def _inputs(lengths, H, Hk, dk, dv, dtype, state_dtype=F32):
    inp = make_linattn(lengths, H, Hk, dk, dv, dtype, state_dtype, seed=sum(lengths) + dk, device=DEV)
    inp["log_decay"] = inp["log_decay"] * (0.02 / 8)  # at most 0.02 a token
    cu = inp["cu_host"].tolist()
    last = [b - 1 for a, b in zip(cu, cu[1:]) if b > a]
    first = [a for a, b in zip(cu, cu[1:]) if b > a]
    # the last token of one sequence (ends inside a chunk), the first of another, one between
    inp["v"][last[0], 0, 3] = INF
    inp["k"][last[1], 0, 5] = -INF
    inp["v"][first[2], H - 1, dv - 1] = -INF
    inp["k"][(first[2] + last[2]) // 2, Hk - 1, dk - 1] = INF
    inp["v"][(first[0] + last[0]) // 2, 1, 0] = INF
    inp["v"][(first[0] + last[0]) // 2 + 1, 1, 0] = INF  # of both signs in the state: NaN where they meet
    if inp["state"] is not None:
        inp["state"][1, 0, 7, 9] = -INF
    return inp


def _check_states(st, inp, what):
    ref, rs, _, sa = linattn_ref(inp)
    st = st.cpu()
    assert torch.equal(torch.isnan(st), torch.isnan(rs)), what + ": NaN"
    assert torch.equal(torch.isposinf(st), torch.isposinf(rs)), what + ": +inf"
    assert torch.equal(torch.isneginf(st), torch.isneginf(rs)), what + ": -inf"
    assert torch.isinf(rs).any()
    fin = torch.isfinite(rs)
    n = (320 + max(inp["lengths"])) * U32
    bound = half_step(st.dtype) * rs.abs() + (n + U16 * U16) * sa * 1.01 + TINY
    check(st[fin], rs[fin], bound[fin], what)


CASES = [([90, 33, 130], 4, 2, "one_pass"),                           # 32 columns to a workgroup
         ([90, 33, 130, 0, 64], 4, 2, "two_pass"),                    # segments of 64 tokens
         ([1, 20, 75] + [9 + i % 60 for i in range(70)], 4, 2, "one_pass"),   # many short sequences
         ([250, 120, 201] + [130 + i for i in range(14)], 16, 8, "one_pass")]  # many pairs


@pytest.mark.parametrize("dk,dv", [(64, 64), (64, 128), (128, 64), (128, 128)])
@pytest.mark.parametrize("case", range(len(CASES)))
@pytest.mark.parametrize("dtype,state_dtype", [(BF, F32), (BF, BF), (F32, F32)])
def test_prefill_states_keep_infinities(case, dk, dv, dtype, state_dtype):
    lengths, H, Hk, schedule = CASES[case]
    if case == 3 and state_dtype == BF:
        pytest.skip("the type of the states is covered by the smaller cases")
    inp = _inputs(lengths, H, Hk, dk, dv, dtype, state_dtype)
    _, st = kda.kda_linattn_prefill(inp["q"], inp["k"], inp["v"], inp["log_decay"], cu_seqlens=inp["cu"],
                                    cu_seqlens_host=inp["cu_host"], state_in=inp["state"], state_out=True,
                                    schedule=schedule)
    _check_states(st, inp, "%s %d" % (schedule, case))


@pytest.mark.parametrize("dtype,state_dtype", [(BF, F32), (BF, BF), (F32, F32)])
def test_decode_states_keep_infinities(dtype, state_dtype):
    inp = _inputs([1, 2, 3], 4, 2, 128, 128, dtype, state_dtype)
    state = inp["state"].clone()
    start = inp["cu_host"].tolist()
    for t in range(3):
        rows = [n for n in range(3) if inp["lengths"][n] > t]
        at = torch.tensor([start[n] + t for n in rows], device=DEV)
        kda.kda_linattn_decode(inp["q"][at], inp["k"][at], inp["v"][at], inp["log_decay"][at], state,
                               state_slots=torch.tensor(rows, dtype=torch.int32, device=DEV))
    if state_dtype == BF:  # rounded once a token
        ref = linattn_ref(inp)[1]
        assert torch.equal(torch.isinf(state.cpu()), torch.isinf(ref)) and torch.equal(torch.isnan(state.cpu()), torch.isnan(ref))
    else:
        _check_states(state, inp, "decode")


@pytest.mark.parametrize("schedule", ["one_pass", "two_pass"])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_products_that_underflow_stay_numbers(schedule, dtype):
    """Tiny values of both signs under decays of every size, zeros of both signs, and a
    whole sequence of such: their products round to zero and change nothing else."""
    inp = make_linattn([200, 64, 1], 3, 3, 128, 128, dtype, seed=77, device=DEV)
    g = torch.Generator().manual_seed(78)
    power = torch.randint(-126, 0, (265, 3, 128), generator=g).to(DEV)
    tiny = torch.exp2(power.float()) * torch.where(inp["v"].float() < 0, -1.0, 1.0)
    pick = torch.rand(265, 3, 128, generator=g).to(DEV)
    v = torch.where(pick < 0.4, tiny, torch.where(pick < 0.5, 0.0, torch.where(pick < 0.6, -0.0, inp["v"].float())))
    v[200:264, 1] = tiny[200:264, 1]
    inp["v"] = v.to(dtype)
    inp["log_decay"][:, 0] = -2.0  # e^-128 over a chunk
    inp["log_decay"][::9, 1] = -60.0
    o, st = kda.kda_linattn_prefill(inp["q"], inp["k"], inp["v"], inp["log_decay"], cu_seqlens=inp["cu"],
                                    cu_seqlens_host=inp["cu_host"], state_in=inp["state"], state_out=True,
                                    schedule=schedule)
    check_linattn(o, st, inp, True)
