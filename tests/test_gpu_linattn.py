"""Linear attention with one decay per head (kda_linattn_prefill, kda_linattn_decode)
against the token-by-token recurrence in 64 bits, at the sizes, strides, decays and
masks where it can go wrong.  The bounds are derived in _linattn_common."""
import pytest
import torch

import gated_delta_rule_short_amd as kda
from tests._linattn_common import DEV, check, check_linattn, linattn_ref, make_linattn

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _lib():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    kda.load_library()


def _prefill(inp, state_out=True, **kw):
    return kda.kda_linattn_prefill(inp["q"], inp["k"], inp["v"], inp["log_decay"], cu_seqlens=inp["cu"],
                                   cu_seqlens_host=inp["cu_host"], state_in=inp["state"], state_out=state_out,
                                   state_slots=inp["slots"], **kw)


@pytest.mark.parametrize("lengths", [[1], [2], [16], [63], [64], [65], [0, 5, 0], [1, 130, 0, 64, 17], [300]])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_prefill_lengths(lengths, dtype):
    inp = make_linattn(lengths, 3, 3, 128, 128, dtype, seed=len(lengths) + lengths[0], device=DEV)
    o, st = _prefill(inp)
    check_linattn(o, st, inp, True)


@pytest.mark.parametrize("dk,dv", [(64, 64), (64, 128), (128, 64), (128, 128)])
@pytest.mark.parametrize("dtype,state_dtype", [(BF, F32), (BF, BF), (F32, F32), (F32, BF)])
def test_prefill_head_dims_and_types(dk, dv, dtype, state_dtype):
    inp = make_linattn([70, 1, 100], 4, 2, dk, dv, dtype, state_dtype, seed=dk + dv, packed=True, device=DEV)
    o, st = _prefill(inp)
    assert st.dtype == state_dtype
    check_linattn(o, st, inp, True)


@pytest.mark.parametrize("dk,dv", [(64, 64), (64, 128), (128, 64), (128, 128)])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_prefill_many_pairs(dk, dv, dtype):
    """Enough (sequence, head) pairs to fill the GPU without splitting states."""
    lengths = [(37 * i) % 150 for i in range(17)] + [0, 1, 64, 128, 200]
    inp = make_linattn(lengths, 16, 8, dk, dv, dtype, seed=40, device=DEV)
    o, st = _prefill(inp)
    check_linattn(o, st, inp, True)
    inp["v"][60, 3, 5] = float("nan")
    o1, _ = _prefill(inp)
    keep = torch.ones(o.shape[:2], dtype=torch.bool, device=DEV)
    assert lengths[0] == 0 and lengths[1] == 37 and lengths[2] == 74
    keep[60:111, 3] = False  # the third sequence: tokens 37..110
    assert torch.equal(o[keep], o1[keep]) and not torch.isfinite(o1[60:111, 3].float()).all(-1).any()


@pytest.mark.parametrize("dk,dv", [(64, 64), (64, 128), (128, 64), (128, 128)])
@pytest.mark.parametrize("lengths,pool", [([700], 0), ([0, 1, 64, 65, 300, 0, 129], 9), ([5] * 130 + [400], 0),
                                          ([250, 200, 64, 1], 6)])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_prefill_two_passes(dk, dv, lengths, pool, dtype):
    """Segments of 64 tokens: one, none and many to a sequence, in place in a pool too, with
    decays that clear the state, and a workspace that held something else."""
    inp = make_linattn(lengths, 4, 2, dk, dv, dtype, seed=50 + len(lengths), pool=pool, device=DEV)
    inp["log_decay"][-100, 1] = float("-inf")
    n = len(lengths)
    args = [inp[x] for x in ("q", "k", "v", "log_decay")]
    ws = torch.full((1 << 27,), 255, dtype=torch.uint8, device=DEV)  # NaN everywhere
    kw = dict(cu_seqlens=inp["cu"], state_slots=inp["slots"], schedule="two_pass", workspace=ws)
    ref = dict(inp, state=inp["state"].clone())
    out = inp["state"] if pool else torch.empty(n, 4, dk, dv, device=DEV)
    o, st = kda.kda_linattn_prefill(*args, state_in=inp["state"], state_out=out, **kw)
    rows = inp["slots"].long() if pool else torch.arange(n, device=DEV)
    check_linattn(o, st[rows], ref, True)
    o1, st1 = kda.kda_linattn_prefill(*args, state_in=ref["state"], state_out=torch.empty_like(out), **kw)
    assert torch.equal(o, o1) and torch.equal(st[rows], st1[rows])


@pytest.mark.parametrize("lengths,host,dk,dv", [([1500], True, 128, 128), ([3800, 3, 1300], False, 64, 128),
                                                ([2100, 0, 70], True, 128, 64)])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_prefill_two_passes_of_many_segments(lengths, host, dk, dv, dtype):
    """Segments joined by the launch that makes the outputs, or by one of their own, over
    enough heads that a workgroup takes more columns; a cleared state among them."""
    inp = make_linattn(lengths, 12, 4, dk, dv, dtype, seed=90 + len(lengths), device=DEV)
    inp["log_decay"][len(inp["q"]) // 2, 5] = float("-inf")
    ref = dict(inp, state=inp["state"].clone())
    o, st = kda.kda_linattn_prefill(inp["q"], inp["k"], inp["v"], inp["log_decay"], cu_seqlens=inp["cu"],
                                    cu_seqlens_host=inp["cu_host"] if host else None, state_in=inp["state"],
                                    state_out=inp["state"], schedule="two_pass")
    check_linattn(o, st, ref, True)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_prefill_automatic_segments(dtype):
    """A long lone sequence takes two passes by itself; the outputs agree with one pass
    within both bounds."""
    inp = make_linattn([6000], 2, 1, 128, 128, dtype, seed=60, device=DEV)
    o, st = _prefill(inp)
    o1, st1 = _prefill(inp, schedule="one_pass")
    assert not torch.equal(o, o1)  # other roundings: the two schedules were run
    check_linattn(o, st, inp, True)
    check_linattn(o1, st1, inp, True)


@pytest.mark.parametrize("H,Hk", [(1, 1), (6, 1), (6, 3), (8, 8), (33, 11)])
@pytest.mark.parametrize("decay", ["token", "head"])
def test_prefill_shared_key_heads_and_fixed_decays(H, Hk, decay):
    inp = make_linattn([90, 33], H, Hk, 128, 64, seed=H, decay=decay, initial=False, device=DEV)
    o, st = _prefill(inp)
    check_linattn(o, st, inp, True)


def test_prefill_equal_sequences_without_cu_seqlens():
    inp = make_linattn([77, 77, 77], 2, 1, 128, 128, seed=5, device=DEV)
    o, st = kda.kda_linattn_prefill(inp["q"], inp["k"], inp["v"], inp["log_decay"], num_seqs=3,
                                    state_in=inp["state"], state_out=True)
    check_linattn(o, st, inp, True)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_prefill_extreme_decays(dtype):
    """-inf and huge negative decays clear the state, positive ones count as 0, and the
    pairs after a clear are as exact as any."""
    inp = make_linattn([150, 64, 40], 4, 4, 128, 128, dtype, seed=9, device=DEV)
    ld = inp["log_decay"]
    ld[3, 0] = float("-inf")
    ld[70:75, 0] = float("-inf")
    ld[:, 1] = -1e30
    ld[::7, 2] = 5.0
    ld[20, 3], ld[21, 3], ld[63, 3] = -3e38, -200.0, -1e4
    ld[150, :] = float("-inf")  # a sequence's first token: its initial state is gone
    o, st = _prefill(inp)
    check_linattn(o, st, inp, True)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("where", ["q", "k", "v", "log_decay"])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_prefill_non_finite_inputs_touch_only_later_tokens(dtype, where, value):
    if where == "log_decay" and value > 0:
        pytest.skip("a positive decay counts as 0")
    inp = make_linattn([100, 90], 2, 2, 128, 128, dtype, seed=3, device=DEV)
    o0, s0 = _prefill(inp)
    if where == "log_decay":
        inp[where][37, 1] = value
    else:
        inp[where][37, 1, 11] = value
    o1, s1 = _prefill(inp)
    keep = torch.ones(190, 2, dtype=torch.bool)
    keep[37:100, 1] = False
    assert torch.equal(o0.cpu()[keep], o1.cpu()[keep])
    assert torch.equal(s0[1], s1[1]) and torch.equal(s0[0, 0], s1[0, 0])
    assert not torch.isfinite(o1[37, 1].float()).all()
    if where == "q":
        assert torch.equal(o0[38:], o1[38:]) and torch.equal(s0, s1)
    else:
        assert not torch.isfinite(s1[0, 1]).all()


def test_prefill_pool_slots_in_place_and_out_of_range():
    inp = make_linattn([50, 3, 70], 2, 2, 128, 128, seed=21, pool=7, device=DEV)
    ref_o, ref_s, _, _ = linattn_ref(inp)
    before = inp["state"].clone()
    pool = inp["state"]
    bad = inp["slots"].clone()
    bad[1] = 7  # outside the pool: that sequence is skipped
    o = torch.full((123, 2, 128), 7.0, dtype=BF, device=DEV)
    _, out = kda.kda_linattn_prefill(inp["q"], inp["k"], inp["v"], inp["log_decay"], cu_seqlens=inp["cu"],
                                     state_in=pool, state_out=pool, state_slots=bad, o=o)
    assert out is pool
    assert (o[50:53] == 7.0).all()
    rows = [int(bad[0]), int(bad[2])]
    for i in range(7):
        if i not in rows:
            assert torch.equal(pool[i], before[i])
    inp["state"] = before
    _, _, oa, sa = linattn_ref(inp)
    for n, r in ((0, rows[0]), (2, rows[1])):
        check(pool[r], ref_s[n], 1e-4 * sa[n], "pool row")
    bad[1] = -1
    o.fill_(7.0)
    kda.kda_linattn_prefill(inp["q"], inp["k"], inp["v"], inp["log_decay"], cu_seqlens=inp["cu"],
                            state_in=before, state_out=pool, state_slots=bad, o=o)
    assert (o[50:53] == 7.0).all()


def test_prefill_leaves_rows_behind_the_last_sequence():
    inp = make_linattn([40, 25, 30], 2, 2, 128, 128, seed=22, device=DEV)
    o0, _ = _prefill(inp)
    cu = inp["cu"].clone()
    cu[3] = 80  # the last sequence holds 15 tokens; 15 rows lie behind it
    o = torch.full((95, 2, 128), 5.0, dtype=BF, device=DEV)
    inp["v"][80:] = float("nan")
    kda.kda_linattn_prefill(inp["q"], inp["k"], inp["v"], inp["log_decay"], cu_seqlens=cu,
                            state_in=inp["state"], o=o)
    assert (o[80:] == 5.0).all() and torch.equal(o[:80], o0[:80])


def test_prefill_without_states_and_without_tokens():
    inp = make_linattn([30], 2, 2, 64, 64, seed=1, initial=False, device=DEV)
    o, st = _prefill(inp, state_out=None)
    assert st is None
    check_linattn(o, None, inp, True)
    e = make_linattn([0, 0], 2, 2, 64, 64, seed=2, device=DEV)
    o, st = _prefill(e)
    assert o.shape == (0, 2, 64) and torch.equal(st, e["state"])
    e["state"] = None
    _, st = _prefill(e)
    assert (st == 0).all()


@pytest.mark.parametrize("dtype", [BF, F32])
def test_prefill_continues_and_decode_follows(dtype):
    """One prompt at once, in two parts, and one token at a time: the states agree within
    twice the bound of each."""
    inp = make_linattn([140], 3, 1, 128, 128, dtype, seed=8, device=DEV)
    o, st = _prefill(inp)
    check_linattn(o, st, inp, True)
    parts, state = [], inp["state"].clone()
    for a, b in ((0, 75), (75, 130)):
        p, _ = kda.kda_linattn_prefill(inp["q"][a:b], inp["k"][a:b], inp["v"][a:b], inp["log_decay"][a:b],
                                       state_in=state, state_out=state)
        parts.append(p)
    for t in range(130, 140):
        parts.append(kda.kda_linattn_decode(inp["q"][t:t + 1], inp["k"][t:t + 1], inp["v"][t:t + 1],
                                            inp["log_decay"][t:t + 1], state))
    check_linattn(torch.cat(parts), state, inp, True)


@pytest.mark.parametrize("N,H,Hk", [(1, 1, 1), (1, 64, 64), (3, 6, 2), (40, 16, 4)])
@pytest.mark.parametrize("dk,dv", [(64, 64), (128, 128), (64, 128), (128, 64)])
@pytest.mark.parametrize("dtype,state_dtype", [(BF, F32), (BF, BF), (F32, F32), (F32, BF)])
def test_decode(N, H, Hk, dk, dv, dtype, state_dtype):
    inp = make_linattn([1] * N, H, Hk, dk, dv, dtype, state_dtype, pool=N + 3 if N > 1 else 0, packed=N == 3,
                       decay="head" if N == 40 else "token", seed=N + dk, device=DEV)
    ref = dict(inp, state=inp["state"].clone())
    o = kda.kda_linattn_decode(inp["q"], inp["k"], inp["v"], inp["log_decay"], inp["state"],
                               state_slots=inp["slots"])
    rows = inp["slots"].long() if inp["slots"] is not None else torch.arange(N, device=DEV)
    check_linattn(o, inp["state"][rows], ref, False)
    rest = [i for i in range(inp["state"].shape[0]) if i not in rows.tolist()]
    assert torch.equal(inp["state"][rest], ref["state"][rest])


@pytest.mark.parametrize("dk,dtype,state_dtype", [(64, BF, F32), (128, BF, F32), (64, F32, BF), (128, BF, BF), (128, F32, F32)])
def test_decode_many_states(dk, dtype, state_dtype):
    """Enough (sequence, head) pairs for 128 columns to a workgroup, in a pool, out of order."""
    inp = make_linattn([1] * 65, 8, 2, dk, 128, dtype, state_dtype, seed=110 + dk, pool=70, device=DEV)
    ref = dict(inp, state=inp["state"].clone())
    o = kda.kda_linattn_decode(inp["q"], inp["k"], inp["v"], inp["log_decay"], inp["state"],
                               state_slots=inp["slots"])
    rows = inp["slots"].long()
    check_linattn(o, inp["state"][rows], ref, False)
    rest = [i for i in range(70) if i not in rows.tolist()]
    assert torch.equal(inp["state"][rest], ref["state"][rest])


def test_decode_skips_slots_outside_the_pool():
    inp = make_linattn([1] * 4, 2, 2, 128, 128, seed=4, pool=6, device=DEV)
    before = inp["state"].clone()
    slots = inp["slots"].clone()
    slots[0], slots[2] = 6, -5
    o = torch.full((4, 2, 128), 3.0, dtype=BF, device=DEV)
    kda.kda_linattn_decode(inp["q"], inp["k"], inp["v"], inp["log_decay"], inp["state"], state_slots=slots, o=o)
    assert (o[0] == 3.0).all() and (o[2] == 3.0).all()
    changed = [i for i in range(6) if not torch.equal(inp["state"][i], before[i])]
    assert changed == sorted([int(slots[1]), int(slots[3])])


def test_decode_pool_beyond_32_bit_offsets():
    """A pool of more than 2^32 elements: its last rows are reached."""
    rows, H = 4200, 64
    pool = torch.empty(rows, H, 128, 128, dtype=BF, device=DEV)
    inp = make_linattn([1, 1], H, H, 128, 128, BF, BF, seed=6, device=DEV)
    slots = torch.tensor([rows - 1, 2099], dtype=torch.int32, device=DEV)
    pool[slots.long()] = inp["state"]
    o = kda.kda_linattn_decode(inp["q"], inp["k"], inp["v"], inp["log_decay"], pool, state_slots=slots)
    check_linattn(o, pool[slots.long()], inp, False)


def test_prefill_token_offsets_beyond_32_bits():
    """q, k and v as views of rows 2^20 elements wide: 2^32 elements from first to last."""
    T, W = 4200, 1 << 20
    wide = torch.empty(T, W, dtype=BF, device=DEV)
    inp = make_linattn([4000, 200], 1, 1, 64, 64, seed=13, device=DEV)
    q, k, v = wide[:, :64], wide[:, 64:128], wide[:, 128:192]
    for view, name in ((q, "q"), (k, "k"), (v, "v")):
        view.copy_(inp[name][:, 0])
    args = [x.unflatten(1, (1, 64)) for x in (q, k, v)] + [inp["log_decay"]]
    o, st = kda.kda_linattn_prefill(*args, cu_seqlens=inp["cu"], state_in=inp["state"], state_out=True)
    o1, st1 = _prefill(inp)
    assert torch.equal(o, o1) and torch.equal(st, st1)


def test_other_stream_and_repeated_calls_are_bit_identical():
    inp = make_linattn([500, 20, 131], 4, 2, 128, 128, seed=14, device=DEV)
    o0, s0 = _prefill(inp)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(3):
        o1, s1 = _prefill(inp, stream=side)
        side.synchronize()
        assert torch.equal(o0, o1) and torch.equal(s0, s1)


def test_captured_steps_replay():
    """A prefill and a decode step in one graph, replayed with eager work between."""
    inp = make_linattn([90, 40], 4, 2, 128, 128, seed=15, device=DEV)
    dec = make_linattn([1, 1], 4, 2, 128, 128, seed=16, initial=False, device=DEV)
    state = torch.empty(2, 4, 128, 128, device=DEV)

    def step():
        o, _ = _prefill(inp, state_out=state)
        d = kda.kda_linattn_decode(dec["q"], dec["k"], dec["v"], dec["log_decay"], state)
        return o, d

    eager = [x.clone() for x in step()] + [state.clone()]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for i in range(4):
        for x in out:
            x.zero_()
        state.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for x, y in zip(list(out) + [state], eager):
            assert torch.equal(x, y), i
        torch.randn(1000, 1000, device=DEV).sum().item()
