"""Forms of the linear attention that the other GPU tests leave out: batches without
tokens, whole states of 64 columns, the returned states' precision, segments over every
kind of input, decays and tokens that are not finite in single steps, captured segments,
and which kernel runs where."""
import os
import re
import subprocess
import sys

import pytest
import torch

import gated_delta_rule_short_amd as kda
from tests._linattn_common import DEV, U32, check, check_linattn, linattn_ref, make_linattn

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _lib():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    kda.load_library()


@pytest.mark.parametrize("schedule", ["auto", "one_pass", "two_pass"])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_an_empty_batch_passes_its_states_through(schedule, dtype):
    inp = make_linattn([0, 0, 0], 4, 2, 64, 128, dtype, seed=1, device=DEV)
    o, st = kda.kda_linattn_prefill(inp["q"], inp["k"], inp["v"], inp["log_decay"], cu_seqlens=inp["cu"],
                                    cu_seqlens_host=inp["cu_host"], state_in=inp["state"], state_out=True,
                                    schedule=schedule)
    assert o.shape == (0, 4, 128) and torch.equal(st, inp["state"])


def _prefill(inp, state_out=True, **kw):
    return kda.kda_linattn_prefill(inp["q"], inp["k"], inp["v"], inp["log_decay"], cu_seqlens=inp["cu"],
                                   cu_seqlens_host=inp["cu_host"], state_in=inp["state"], state_out=state_out,
                                   state_slots=inp["slots"], **kw)


# ------------------------------------------------------------------ whole states of 64 columns
MANY = [(83 * i) % 401 for i in range(17)]  # 0 .. 400 tokens, more than 128 on average


@pytest.mark.parametrize("dk", [64, 128])
@pytest.mark.parametrize("dtype,state_dtype", [(BF, F32), (BF, BF), (F32, F32)])
def test_many_pairs_of_64_columns(dk, dtype, state_dtype):
    inp = make_linattn(MANY, 16, 8, dk, 64, dtype, state_dtype, seed=dk, packed=True, device=DEV)
    o, st = _prefill(inp, schedule="one_pass")
    check_linattn(o, st, inp, True)
    cu = inp["cu_host"].tolist()
    n = 4  # 332 tokens
    at, end = cu[n] + 150, cu[n + 1]
    assert end - at > 64
    inp["v"][at, 3, 5] = float("nan")
    o1, st1 = _prefill(inp, schedule="one_pass")
    keep = torch.ones(o.shape[:2], dtype=torch.bool, device=DEV)
    keep[at:end, 3] = False
    assert torch.equal(o[keep], o1[keep]) and not torch.isfinite(o1[at:end, 3].float()).all(-1).any()
    rows = torch.ones(st.shape[:2], dtype=torch.bool, device=DEV)
    rows[n, 3] = False
    assert torch.equal(st[rows], st1[rows]) and not torch.isfinite(st1[n, 3].float()).all()


# ------------------------------------------------------------------ precision of the states
@pytest.mark.parametrize("dk,dv", [(64, 64), (64, 128), (128, 64), (128, 128)])
@pytest.mark.parametrize("L,t,schedule", [(1, 0, "one_pass"), (64, 10, "one_pass"), (64, 63, "one_pass"),
                                          (300, 70, "one_pass"), (300, 5, "one_pass"), (300, 5, "two_pass"),
                                          (300, 140, "two_pass"), (1500, 1100, "two_pass")])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_the_state_of_one_token_is_good_to_fp32(L, t, schedule, dk, dv, dtype):
    """v is zero but at token t, so the state is k_t v_t^T times its decay and nothing
    hides its roundings, in units of 2^-24: the exponent's argument (at most 64 tokens of
    0.07 in base 2, half a step of at most 4: 3), the exponential (2), its product with v
    (1) and one addition for each of the operand's three parts (2 each where the matrix
    cores truncate) or the fp32 product and its addition (3); behind that, 7 for each chunk
    (32 tokens at least, its factor 5 as above, the product 1) and for each segment that a
    join passes.  Zeros add nothing.  A write in two parts would be off by up to 2^-15."""
    H = 3
    inp = make_linattn([L], H, H, dk, dv, dtype, seed=L + t + dk, initial=False, device=DEV)
    inp["log_decay"] = inp["log_decay"].clamp(min=-0.05)
    one = inp["v"][t].clone()
    inp["v"].zero_()
    inp["v"][t] = one
    _, st = _prefill(inp, schedule=schedule)
    g = inp["log_decay"].cpu().double()[t + 1:].sum(0)
    ref = inp["k"][t].cpu().double()[:, :, None] * one.cpu().double()[:, None, :] * g.exp()[:, None, None]
    n = 12 + 7 * ((L - t + 31) // 32) + 7 * ((L - t + 63) // 64 if schedule == "two_pass" else 0)
    assert n < 250  # of about 512 for a part of 2^-15 left out
    check(st[0], ref, n * U32 * ref.abs(), "state")


# ------------------------------------------------------------------ segments over every kind of input
@pytest.mark.parametrize("dk,dv", [(64, 64), (64, 128), (128, 64), (128, 128)])
@pytest.mark.parametrize("dtype,state_dtype,decay,initial,pool", [
    (BF, BF, "head", True, 0), (BF, BF, "token", True, 7), (BF, F32, "head", False, 0), (BF, F32, "head", True, 7),
    (F32, BF, "head", True, 7), (F32, F32, "token", False, 0)])
def test_two_passes_over_packed_tokens_and_every_state(dk, dv, dtype, state_dtype, decay, initial, pool):
    lengths = [300, 0, 65, 130, 1]
    inp = make_linattn(lengths, 6, 2, dk, dv, dtype, state_dtype, decay, initial, pool, packed=True, seed=dk + dv + 7,
                       device=DEV)
    if decay == "head":
        inp["log_decay"][1] = float("-inf")  # every token clears this head's state
    ref = dict(inp, state=inp["state"].clone() if initial else None)
    out = inp["state"] if pool else torch.empty(5, 6, dk, dv, dtype=state_dtype, device=DEV)
    o, st = _prefill(inp, state_out=out, schedule="two_pass")
    rows = inp["slots"].long() if pool else torch.arange(5, device=DEV)
    check_linattn(o, st[rows], ref, True)
    if pool:
        rest = [i for i in range(pool) if i not in rows.tolist()]
        assert torch.equal(st[rest], ref["state"][rest])


@pytest.mark.parametrize("lengths", [[100, 640, 70], [100, 1500, 70]])  # joined by the outputs, by a scan
@pytest.mark.parametrize("where", ["q", "k", "v", "log_decay"])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_two_passes_keep_non_finite_values_to_later_tokens(lengths, where, value, dtype):
    if where == "log_decay" and value > 0:
        value = 3.0  # a positive decay counts as 0
    inp = make_linattn(lengths, 3, 3, 128, 128, dtype, seed=lengths[1], device=DEV)
    at, end = 100 + lengths[1] // 2 + 5, 100 + lengths[1]
    if value == 3.0:
        inp["log_decay"][at, 1] = 0.0
    o0, s0 = _prefill(inp, schedule="two_pass")
    if where == "log_decay":
        inp[where][at, 1] = value
    else:
        inp[where][at, 1, 11] = value
    o1, s1 = _prefill(inp, schedule="two_pass")
    if value == 3.0:
        assert torch.equal(o0, o1) and torch.equal(s0, s1)
        return
    keep = torch.ones(o0.shape[:2], dtype=torch.bool, device=DEV)
    keep[at:at + 1 if where == "q" else end, 1] = False
    assert torch.equal(o0[keep], o1[keep])
    assert not torch.isfinite(o1[~keep].float()).all(-1).any()
    rows = torch.ones(s0.shape[:2], dtype=torch.bool, device=DEV)
    rows[1, 1] = where == "q"
    assert torch.equal(s0[rows], s1[rows])
    if where != "q":
        assert not torch.isfinite(s1[1, 1]).all()


@pytest.mark.parametrize("dtype", [BF, F32])
def test_two_passes_captured_and_replayed(dtype):
    """Segments with either join and a decode step in one graph, replayed with eager work
    between; the workspaces are the graph's own."""
    inp = make_linattn([700, 90], 3, 1, 128, 128, dtype, seed=15, device=DEV)
    far = make_linattn([2000], 3, 3, 128, 64, dtype, seed=16, device=DEV)
    state = torch.empty(2, 3, 128, 128, device=DEV)

    def step():
        o, _ = _prefill(inp, state_out=state, schedule="two_pass")
        d = kda.kda_linattn_decode(inp["q"][:2], inp["k"][:2], inp["v"][:2], inp["log_decay"][:2], state)
        f, s = _prefill(far, schedule="two_pass")
        return o, d, f, s

    eager = [x.clone() for x in step()] + [state.clone()]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for i in range(4):
        for x in list(out) + [state]:
            x.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for x, y in zip(list(out) + [state], eager):
            assert torch.equal(x, y), i
        o, s = _prefill(far, schedule="two_pass")  # eager, with a workspace of its own
        assert torch.equal(o, eager[2]) and torch.equal(s, eager[3])


# ------------------------------------------------------------------ single steps
@pytest.mark.parametrize("N,dv", [(5, 64), (5, 128), (130, 128)])
@pytest.mark.parametrize("dtype,state_dtype", [(BF, F32), (BF, BF), (F32, F32), (F32, BF)])
def test_decode_extreme_decays(N, dv, dtype, state_dtype):
    """-inf and huge negative decays clear the state, positive ones count as 0."""
    inp = make_linattn([1] * N, 4, 2, 128, dv, dtype, state_dtype, seed=N, device=DEV)
    ld = inp["log_decay"]
    ld[0, 0] = float("-inf")
    ld[1, 1], ld[2, 1] = -1e30, -3e38
    ld[:, 2] = 5.0
    ld[3, 3], ld[4, 3] = float("inf"), -200.0
    ref = dict(inp, state=inp["state"].clone())
    o = kda.kda_linattn_decode(inp["q"], inp["k"], inp["v"], ld, inp["state"])
    check_linattn(o, inp["state"], ref, False)


@pytest.mark.parametrize("where", ["q", "k", "v", "log_decay", "state"])
@pytest.mark.parametrize("N,dtype,state_dtype", [(3, BF, F32), (130, BF, BF), (3, F32, BF), (130, F32, F32)])
def test_decode_non_finite_values_stay_with_their_head(where, N, dtype, state_dtype):
    inp = make_linattn([1] * N, 4, 4, 128, 128, dtype, state_dtype, seed=N + 1, device=DEV)

    def step():
        state = inp["state"].clone()
        return kda.kda_linattn_decode(inp["q"], inp["k"], inp["v"], inp["log_decay"], state), state

    o0, s0 = step()
    if where == "log_decay":
        inp[where][1, 2] = float("nan")
    elif where == "state":
        inp[where][1, 2, 9, 11] = float("nan")
    else:
        inp[where][1, 2, 11] = float("nan")
    o1, s1 = step()
    keep = torch.ones(N, 4, dtype=torch.bool, device=DEV)
    keep[1, 2] = False
    assert torch.equal(o0[keep], o1[keep]) and torch.equal(s0[keep], s1[keep])
    if where in ("v", "state"):  # one column
        col = torch.arange(128, device=DEV) != 11
        assert torch.equal(o0[1, 2, col], o1[1, 2, col]) and torch.equal(s0[1, 2][:, col], s1[1, 2][:, col])
        assert torch.isnan(o1[1, 2, 11])
    else:
        assert torch.isnan(o1[1, 2]).all()
    assert torch.equal(s0, s1) if where == "q" else not torch.isfinite(s1[1, 2].float()).all()


# ------------------------------------------------------------------ which kernel runs where
DISPATCH = r"""
import sys
import torch
import gated_delta_rule_short_amd as kda
from tests._linattn_common import DEV, make_linattn
from tests.test_gpu_linattn_forms import MANY
BF, F32 = torch.bfloat16, torch.float32

def prefill(name, lengths, H, Hk, dk, dv, dtype, schedule):
    inp = make_linattn(lengths, H, Hk, dk, dv, dtype, seed=1, device=DEV)
    print("== " + name, file=sys.stderr, flush=True)
    kda.kda_linattn_prefill(inp["q"], inp["k"], inp["v"], inp["log_decay"], cu_seqlens=inp["cu"],
                            cu_seqlens_host=inp["cu_host"], state_in=inp["state"], state_out=True, schedule=schedule)

for dk in (64, 128):
    prefill("many64 %d" % dk, MANY, 16, 8, dk, 64, BF, "one_pass")
    prefill("short64 %d" % dk, [9 + i % 60 for i in range(73)], 4, 2, dk, 64, BF, "one_pass")
    prefill("few64 %d" % dk, [90, 33, 130], 4, 2, dk, 64, BF, "one_pass")
    prefill("many128 %d" % dk, MANY, 16, 8, dk, 128, BF, "one_pass")
    prefill("manyf32 %d" % dk, MANY, 16, 8, dk, 64, F32, "one_pass")
    prefill("fewf32 %d" % dk, [90, 33, 130], 4, 2, dk, 64, F32, "one_pass")
    for dv in (64, 128):
        prefill("segments %d %d" % (dk, dv), [640], 3, 3, dk, dv, BF, "two_pass")
        prefill("scan %d %d" % (dk, dv), [1500], 3, 3, dk, dv, BF, "two_pass")
torch.cuda.synchronize()
"""


def test_the_kernels_of_each_shape():
    """The launch log of calls of the tests above: a moved threshold must not drop a
    kernel out of them."""
    r = subprocess.run([sys.executable, "-c", DISPATCH], capture_output=True, text=True, timeout=300, cwd=ROOT,
                       env=dict(os.environ, KDA_TRACE="1", PYTHONPATH=ROOT))
    assert r.returncode == 0, r.stderr[-2000:]
    ran, name = {}, None
    for line in r.stderr.splitlines():
        if line.startswith("== "):
            name = line[3:]
            ran[name] = []
        elif line.startswith("[kda] ") and name:
            m = re.match(r"\[kda\] (\w+)(?:<([^>]*)>)?", line)
            ran[name].append(m.group(1) + ("<%s>" % m.group(2) if m.group(2) else ""))
    want = {}
    for dk in (64, 128):
        want["many64 %d" % dk] = ["chunk_kernel<%s, 1>" % ("64, 64, 1, 3" if dk == 64 else "128, 64, 2, 2")]
        want["short64 %d" % dk] = ["chunk_kernel<%d, 64, 1, 1, 1>" % dk]
        want["few64 %d" % dk] = ["chunk_kernel<%d, 32, 2, 3, 1>" % dk]
        want["many128 %d" % dk] = ["chunk_kernel<%d, 128, 1, 3, 1>" % dk]
        want["manyf32 %d" % dk] = ["chunk_f32_kernel<%d, 64, 1>" % dk]
        want["fewf32 %d" % dk] = ["chunk_f32_kernel<%d, 32, 1>" % dk]
        for dv in (64, 128):
            first, out = ("2, 0", "1, 1") if dv == 64 else ("4, 0", "3, 1")
            seg = ["chunk_kernel<%d, %d, 1, %s>" % (dk, dv, x) for x in (first, out)]
            want["segments %d %d" % (dk, dv)] = seg
            want["scan %d %d" % (dk, dv)] = [seg[0], "segment_scan_kernel", seg[1]]
    assert ran == want
