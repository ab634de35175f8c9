"""kda_gated_scan_prefill, _decode and _backward against the recurrence and its gradients
in 64 bits.  The bounds are derived in _scan_common."""
import pytest
import torch

import gated_delta_rule_short_amd as kda
from tests._scan_common import (BF, DEV, F32, KINDS, U32, backward_ref, check, check_backward, check_scan, factors,
                                make_scan, scan_ref)

pytestmark = pytest.mark.gpu
SHAPES = [([1], 8), ([0, 1, 2], 120), ([15, 16, 17, 0], 128), ([127, 128, 129, 1], 136), ([300, 0, 700, 64], 264),
          ([239, 240, 241, 480], 72), ([149, 150, 151, 179, 180, 181], 40)]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    kda.load_library()


def _prefill(inp, gate, inputs, **kw):
    kw.setdefault("state_in", inp["state"])
    kw.setdefault("state_out", True)
    kw.setdefault("cu_seqlens", inp["cu"])
    return kda.kda_gated_scan_prefill(inp["x"], inp["gate"], gate_kind=gate, input_kind=inputs, **kw)


def _grads(inp, gate, inputs, dtype, seed=50, dstate=True, **kw):
    """(d_o, o, dstate_out, results) of a backward call on the forward call's output."""
    o, _ = _prefill(inp, gate, inputs)
    gen = torch.Generator().manual_seed(seed)
    d_o = torch.randn(*o.shape, generator=gen).to(dtype).to(DEV)
    ds = torch.randn(len(inp["lengths"]), o.shape[1], generator=gen).to(DEV) if dstate else None
    got = kda.kda_gated_scan_backward(d_o, inp["gate"], o, None if inputs == "plain" else inp["x"], gate_kind=gate,
                                      input_kind=inputs, cu_seqlens=inp["cu"], state_in=inp["state"], dstate_out=ds,
                                      dstate_in=True, **kw)
    return d_o, o, ds, got


@pytest.mark.parametrize("lengths,C", SHAPES)
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("schedule", ["one_pass", "chained"])
def test_prefill_shapes(lengths, C, dtype, schedule):
    for i, (gate, inputs) in enumerate(KINDS):
        inp = make_scan(lengths, C, dtype, gate, seed=i, initial=i % 2 == 0, device=DEV)
        o, state = _prefill(inp, gate, inputs, schedule=schedule)
        check_scan(o, state, inp, gate, inputs, "%s %s" % (gate, inputs))


@pytest.mark.parametrize("lengths,C", SHAPES)
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("schedule", ["one_pass", "chained"])
def test_backward_shapes(lengths, C, dtype, schedule):
    for i, (gate, inputs) in enumerate(KINDS):
        inp = make_scan(lengths, C, dtype, gate, seed=i, initial=i % 2 == 0, device=DEV)
        d_o, o, ds, got = _grads(inp, gate, inputs, dtype, dstate=i % 3 != 0, schedule=schedule)
        check_backward(got, inp, d_o, o, ds, gate, inputs, "%s %s" % (gate, inputs))


@pytest.mark.parametrize("gate,inputs", KINDS)
@pytest.mark.parametrize("dtype,state_dtype", [(BF, BF), (BF, F32), (F32, BF)])
def test_pool_and_packed_projections(gate, inputs, dtype, state_dtype):
    """Rows of a pool, tokens inside a wider projection, in place: other rows stay."""
    inp = make_scan([40, 0, 200, 1], 144, dtype, gate, state_dtype, pool=9, packed=True, seed=3, device=DEV)
    before = inp["state"].clone()
    out = torch.full((241, 400), 7.0, dtype=dtype, device=DEV)
    o = out[:, 128:272]
    got, state = kda.kda_gated_scan_prefill(inp["x"], inp["gate"], gate_kind=gate, input_kind=inputs,
                                            cu_seqlens=inp["cu"], cu_seqlens_host=inp["cu_host"], state_in=inp["state"],
                                            state_out=inp["state"], state_slots=inp["slots"], o=o)
    assert got is o and state is inp["state"]
    used = inp["slots"].long()
    check_scan(o, state[used], dict(inp, state=before), gate, inputs)
    rest = torch.ones(9, dtype=torch.bool, device=DEV)
    rest[used] = False
    assert torch.equal(state[rest], before[rest])
    assert (out[:, :128] == 7.0).all() and (out[:, 272:] == 7.0).all()


@pytest.mark.parametrize("schedule", ["one_pass", "chained"])
def test_slots_outside_the_pool_are_skipped(schedule):
    inp = make_scan([150, 30, 260], 136, F32, "log", pool=5, seed=4, device=DEV)
    good = inp["slots"].clone()
    for bad in (-1, 5, 2147483647):
        slots = good.clone()
        slots[1] = bad
        pool, o = inp["state"].clone(), torch.full_like(inp["x"], 3.0)
        kda.kda_gated_scan_prefill(inp["x"], inp["gate"], cu_seqlens=inp["cu"], state_in=pool, state_out=pool,
                                   state_slots=slots, o=o, schedule=schedule)
        ro, rs, eo, es = scan_ref(inp, "log", "plain")
        keep = torch.tensor([0, 2])
        check(pool[good.long()][keep], rs[keep], U32 * rs[keep].abs() + es[keep], "state")
        assert torch.equal(pool[good[1].long()], inp["state"][good[1].long()])
        assert (o[150:180] == 3.0).all()
        check(o[:150], ro[:150], U32 * ro[:150].abs() + eo[:150], "o")
        one = torch.full((3, 136), 3.0, device=DEV)
        pool = inp["state"].clone()
        kda.kda_gated_scan_decode(inp["x"][:3], inp["gate"][:3], pool, state_slots=slots, o=one)
        assert (one[1] == 3.0).all() and torch.equal(pool[good[1].long()], inp["state"][good[1].long()])


@pytest.mark.parametrize("schedule", ["one_pass", "chained"])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_equal_sequences_without_bounds(schedule, dtype):
    inp = make_scan([190, 190, 190], 72, dtype, "sigmoid", seed=5, device=DEV)
    o, state = _prefill(inp, "sigmoid", "complement", cu_seqlens=None, num_seqs=3, schedule=schedule)
    check_scan(o, state, inp, "sigmoid", "complement")


@pytest.mark.parametrize("schedule", ["one_pass", "chained"])
def test_rows_behind_the_last_sequence_stay(schedule):
    """Device bounds that end before T: the rows behind them are neither read nor written."""
    inp = make_scan([200, 90], 136, F32, "log", seed=6, device=DEV)
    pad = torch.full((70, 136), float("nan"), device=DEV)
    x, g = torch.cat([inp["x"], pad]), torch.cat([inp["gate"], pad])
    o = torch.full_like(x, 5.0)
    _, state = kda.kda_gated_scan_prefill(x, g, cu_seqlens=inp["cu"], state_in=inp["state"], state_out=True, o=o,
                                          schedule=schedule)
    check_scan(o[:290], state, inp, "log", "plain")
    assert (o[290:] == 5.0).all()
    d, dx, dg = torch.cat([inp["x"], pad]), torch.full_like(x, 5.0), torch.full_like(x, 6.0)
    _, _, ds = kda.kda_gated_scan_backward(d, g, o, cu_seqlens=inp["cu"], state_in=inp["state"], dx=dx, dgate=dg,
                                           dstate_in=True, schedule=schedule)
    check_backward((dx[:290], dg[:290], ds), inp, d[:290], o[:290], None, "log", "plain")
    assert (dx[290:] == 5.0).all() and (dg[290:] == 6.0).all()


@pytest.mark.parametrize("count", [63, 64, 65, 4100])
@pytest.mark.parametrize("schedule", ["one_pass", "chained"])
def test_many_sequences(count, schedule):
    """More sequences than a wave has lanes, and than two steps of its search tell apart."""
    gen = torch.Generator().manual_seed(count)
    lengths = torch.randint(0, 4, (count,), generator=gen).tolist()
    lengths[count // 2] = 500
    inp = make_scan(lengths, 16, F32, "log", pool=count + 3, seed=count, device=DEV)
    before = inp["state"].clone()
    o, pool = kda.kda_gated_scan_prefill(inp["x"], inp["gate"], cu_seqlens=inp["cu"], state_in=inp["state"],
                                         state_out=inp["state"], state_slots=inp["slots"], schedule=schedule)
    check_scan(o, pool[inp["slots"].long()], dict(inp, state=before), "log", "plain")
    dense = dict(inp, state=before[inp["slots"].long()].contiguous(), slots=None)
    d_o, o, ds, got = _grads(dense, "log", "plain", F32, schedule=schedule)
    check_backward(got, dense, d_o, o, ds, "log", "plain")


def test_many_tiles_and_repeatability():
    """A long chain beside short ones: bitwise the same from run to run, and the sequences
    of a ragged batch as on their own."""
    inp = make_scan([9000, 3, 1000], 264, F32, "log", seed=7, device=DEV)
    o, state = _prefill(inp, "log", "plain", schedule="chained")
    check_scan(o, state, inp, "log", "plain")
    for _ in range(5):
        o2, state2 = _prefill(inp, "log", "plain", schedule="chained")
        assert torch.equal(o, o2) and torch.equal(state, state2)
    first = {k: inp[k][:9000] for k in ("x", "gate")}
    o3, state3 = kda.kda_gated_scan_prefill(first["x"], first["gate"], state_in=inp["state"][:1].contiguous(),
                                            state_out=True, schedule="chained")
    assert torch.equal(o3, o[:9000]) and torch.equal(state3, state[:1])
    d_o, o, ds, got = _grads(inp, "log", "plain", F32, schedule="chained")
    check_backward(got, inp, d_o, o, ds, "log", "plain")
    for _ in range(3):
        again = kda.kda_gated_scan_backward(d_o, inp["gate"], o, cu_seqlens=inp["cu"], state_in=inp["state"],
                                            dstate_out=ds, dstate_in=True, schedule="chained")
        assert all(torch.equal(a, b) for a, b in zip(got, again))


@pytest.mark.parametrize("schedule", ["one_pass", "chained"])
def test_long_memories_keep_their_length(schedule):
    """A steady gate 1 - 1e-4 over 60,000 tokens of ones: the state is that of the gate as it
    is, not of its fp32 rounding (which would be off by 3e-4)."""
    T, C = 60000, 16
    g = torch.full((T, C), -1.0001e-4, device=DEV)
    x = torch.ones(T, C, device=DEV)
    o, state = kda.kda_gated_scan_prefill(x, g, state_out=True, schedule=schedule)
    z = g[0, 0].double().cpu()
    want = -torch.expm1(z * torch.arange(1, T + 1, dtype=torch.float64)) / -torch.expm1(z)
    at = torch.tensor([0, 100, 5000, 30000, 59999])
    # one rounding of the exponential (1 ulp = 2 u32) and of the step (u32) for each tile, of
    # 56 tokens or more, over the 10,000 tokens that count, and those of a tile's sums
    bound = 3 * (10000 / 56 + 32) * U32 * want[at][:, None]
    check(o[at], want[at][:, None].expand(-1, C), bound.expand(-1, C), "o")
    check(state, want[-1].expand(1, C), float(bound[-1]), "state")
    h = torch.zeros(1, C, device=DEV)
    for _ in range(300):
        kda.kda_gated_scan_decode(x[:1], g[:1], h)
    check(h, want[299].expand(1, C), float(300 * U32 * want[299]), "decode")


@pytest.mark.parametrize("gate,inputs", KINDS)
@pytest.mark.parametrize("dtype,state_dtype", [(BF, F32), (F32, F32), (BF, BF)])
def test_decode_steps(gate, inputs, dtype, state_dtype):
    for N, C in ((1, 8), (3, 4096), (37, 1000)):
        inp = make_scan([1] * N, C, dtype, gate, state_dtype, pool=N + 3, packed=True, seed=N, device=DEV)
        pool = inp["state"].clone()
        o = kda.kda_gated_scan_decode(inp["x"], inp["gate"], pool, gate_kind=gate, input_kind=inputs,
                                      state_slots=inp["slots"])
        check_scan(o, pool[inp["slots"].long()], inp, gate, inputs)
        dense = inp["state"][inp["slots"].long()].contiguous()
        o2 = kda.kda_gated_scan_decode(inp["x"], inp["gate"], dense, gate_kind=gate, input_kind=inputs)
        assert torch.equal(o, o2) and torch.equal(dense, pool[inp["slots"].long()])


@pytest.mark.parametrize("schedule", ["one_pass", "chained"])
@pytest.mark.parametrize("gate", ["log", "sigmoid"])
def test_extreme_gates(schedule, gate):
    """Gates that clear, that hold, above 0, and far out on both sides."""
    inp = make_scan([260, 5], 40, F32, gate, seed=8, device=DEV)
    vals = [0.0, -0.0, 1.0, 40.0, -40.0, -1e30, float("-inf"), float("inf"), -1e-30, 3.0]
    for i, v in enumerate(vals):
        inp["gate"][:, i] = v
        inp["gate"][100 + i, 10:40] = v
    for inputs in ("plain", "complement", "norm"):
        o, state = _prefill(inp, gate, inputs, schedule=schedule)
        ref = dict(inp, gate=inp["gate"].clamp(-1e4, 1e4))  # the bounds' |z| |l| of infinities
        check_scan(o, state, ref, gate, inputs, inputs)
        d_o, o, ds, got = _grads(inp, gate, inputs, F32, schedule=schedule)
        fin = torch.isfinite(inp["gate"])
        assert all(torch.isfinite(t).all() for t in got), inputs
        check_backward(got, ref, d_o, o, ds, gate, inputs, inputs)
        if gate == "log":
            assert (got[1][inp["gate"] > 0] == 0).all()
        assert fin.any()


@pytest.mark.parametrize("schedule", ["one_pass", "chained"])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), float("-inf")])
def test_non_finite_values_stay_in_their_channel(schedule, value):
    inp = make_scan([500, 400], 136, BF, "log", seed=9, device=DEV)
    inp["gate"].clamp_(min=-0.05)  # decays that an infinity outlives
    clean, cstate = _prefill(inp, "log", "plain", schedule=schedule)
    x = inp["x"].clone()
    x[333, 17] = value
    x[20, 135] = value
    o, state = _prefill(dict(inp, x=x), "log", "plain", schedule=schedule)
    hit = torch.zeros_like(x, dtype=torch.bool)
    hit[333:500, 17] = hit[20:500, 135] = True
    assert torch.equal(o[~hit], clean[~hit])
    assert torch.equal(state[1], cstate[1])
    bad = torch.isnan(o[hit]) if value != value else o[hit] == value
    assert bad.all()
    keep = torch.ones(136, dtype=torch.bool, device=DEV)
    keep[[17, 135]] = False
    assert torch.equal(state[0, keep], cstate[0, keep]) and not torch.isfinite(state[0, [17, 135]]).any()
    s0 = inp["state"].clone()
    s0[0, 5] = value
    o, _ = _prefill(inp, "log", "plain", schedule=schedule, state_in=s0)
    assert torch.equal(o[500:], clean[500:]) and not torch.isfinite(o[:500, 5]).any()
    h = torch.tensor([[value] * 8], device=DEV)
    one = kda.kda_gated_scan_decode(torch.ones(1, 8, device=DEV), torch.full((1, 8), -0.01, device=DEV), h)
    assert (torch.isnan(one) if value != value else one == value).all()


def test_backward_against_autograd_and_differences():
    """The gradients of a scalar of o and the final state, by autograd through the
    recurrence in 64 bits and by central differences of it."""
    for gate, inputs in KINDS:
        inp = make_scan([33, 20], 8, F32, gate, seed=10, device=DEV)
        d_o, o, ds, got = _grads(inp, gate, inputs, F32)
        leaves = [inp[k].cpu().double().requires_grad_(True) for k in ("x", "gate", "state")]

        def scalar(x, z, s):
            a, b = factors(z, gate, inputs)[:2]
            h, total, t = list(s.unbind(0)), 0.0, 0
            for n, L in enumerate(inp["lengths"]):
                for t in range(t, t + L):
                    h[n] = a[t] * h[n] + b[t] * x[t]
                    total = total + (h[n] * d_o[t].cpu().double()).sum()
                t += 1
            return total + (torch.stack(h) * ds.cpu().double()).sum()
        grads = torch.autograd.grad(scalar(*leaves), leaves)
        refs, errs = backward_ref(inp, d_o, o, ds, gate, inputs)
        for g, ref, err, x in zip(grads, refs, errs, got):
            # o itself, and with it dgate, carries the forward pass's fp32 error
            slack = 64 * U32 * ref.abs() + 300 * U32 * (1.0 + ref.abs().max())
            check(x, g, err + slack, "%s %s" % (gate, inputs))
        with torch.no_grad():
            for leaf, g in zip(leaves, grads):
                for i in (0, leaf.numel() // 2, leaf.numel() - 1):
                    old, eps = leaf.view(-1)[i].item(), 1e-5
                    leaf.view(-1)[i] = old + eps
                    up = scalar(*leaves)
                    leaf.view(-1)[i] = old - eps
                    down = scalar(*leaves)
                    leaf.view(-1)[i] = old
                    num = float((up - down) / (2 * eps))
                    # eps^2 / 6 of the third derivative and 1e-16 of the scalar over eps
                    assert abs(num - float(g.view(-1)[i])) < 1e-6 * (1.0 + abs(num)) * 20


def test_backward_strides_and_shared_buffers():
    inp = make_scan([210, 40], 136, BF, "sigmoid", packed=True, seed=11, device=DEV)
    o, _ = _prefill(inp, "sigmoid", "norm")
    gen = torch.Generator().manual_seed(1)
    d_o = torch.randn(250, 136, generator=gen).to(BF).to(DEV)
    ds = torch.randn(2, 136, generator=gen).to(DEV)
    args = dict(gate_kind="sigmoid", input_kind="norm", cu_seqlens=inp["cu"], state_in=inp["state"])
    want = kda.kda_gated_scan_backward(d_o, inp["gate"], o, inp["x"], dstate_out=ds, dstate_in=True, **args)
    check_backward(want, inp, d_o, o, ds, "sigmoid", "norm")
    grads = torch.full((250, 2 * 136 + 16), 9.0, dtype=BF, device=DEV)
    dx, dg = grads[:, :136], grads[:, 144:280]
    same = ds.clone()
    got = kda.kda_gated_scan_backward(d_o, inp["gate"], o, inp["x"], dstate_out=same, dstate_in=same, dx=dx, dgate=dg, **args)
    assert got[2] is same and all(torch.equal(a, b) for a, b in zip(want, got))
    assert (grads[:, 136:144] == 9.0).all() and (grads[:, 280:] == 9.0).all()


def test_a_wait_that_gives_up_ends_the_call():
    """With one poll allowed a tile may give up on the state before it: then NaN follows, and
    what is not NaN is right; the bound restored, the next call is whole."""
    inp = make_scan([6000], 264, F32, "log", seed=12, device=DEV)
    want, _ = _prefill(inp, "log", "plain", schedule="chained")
    old = kda.set_spin_limit(1)
    try:
        got, _ = _prefill(inp, "log", "plain", schedule="chained")
        torch.cuda.synchronize()
    finally:
        kda.set_spin_limit(0)
    assert old > 1
    ok = ~torch.isnan(got)
    assert torch.equal(got[ok], want[ok]) and ok[:56].all()
    got, _ = _prefill(inp, "log", "plain", schedule="chained")
    assert torch.equal(got, want)


def test_captured_calls_replay():
    """Two graphs with a workspace each, forward and backward, replayed in turn between eager
    calls on changing inputs."""
    inp = make_scan([700, 300], 264, BF, "sigmoid", seed=13, device=DEV)
    args = dict(gate_kind="sigmoid", input_kind="complement", cu_seqlens=inp["cu"], cu_seqlens_host=inp["cu_host"])
    d_o = torch.randn(1000, 264, device=DEV).to(BF)
    x, o, st = inp["x"].clone(), torch.empty_like(inp["x"]), inp["state"].clone()
    dx, dg = torch.empty_like(x), torch.empty_like(x)
    ws = [torch.empty(1 << 20, dtype=torch.uint8, device=DEV) for _ in range(2)]

    def forward():
        kda.kda_gated_scan_prefill(x, inp["gate"], o=o, state_in=inp["state"], state_out=st, workspace=ws[0], **args)

    def backward():
        kda.kda_gated_scan_backward(d_o, inp["gate"], o, x, dx=dx, dgate=dg, state_in=inp["state"], workspace=ws[1], **args)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        forward()
        backward()
    torch.cuda.current_stream().wait_stream(side)
    graphs = []
    for f in (forward, backward):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            f()
        graphs.append(g)
    for i in range(4):
        x.copy_(torch.randn(1000, 264, generator=torch.Generator().manual_seed(i)).to(BF).to(DEV))
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (o, st, dx, dg)]
        w = kda.kda_gated_scan_prefill(x, inp["gate"], state_in=inp["state"], state_out=True, **args)
        b = kda.kda_gated_scan_backward(d_o, inp["gate"], w[0], x, state_in=inp["state"], **args)
        assert all(torch.equal(p, q) for p, q in zip(got, (w[0], w[1], b[0], b[1]))), i


def test_captured_decode_advances_a_pool():
    """Every replay is one more token of the sequences' slots, between eager steps of others."""
    inp = make_scan([1] * 5, 264, BF, "log", BF, pool=9, seed=16, device=DEV)
    x, pool, slots = inp["x"].clone(), inp["state"].clone(), inp["slots"]
    o = torch.empty_like(x)
    step = lambda p, out=None: kda.kda_gated_scan_decode(x, inp["gate"], p, input_kind="norm", o=out, state_slots=slots)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(pool.clone(), o)
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step(pool, o)
    want = inp["state"].clone()
    for i in range(4):
        x.copy_(torch.randn(5, 264, generator=torch.Generator().manual_seed(i)).to(BF).to(DEV))
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(step(want), o) and torch.equal(want, pool), i


@pytest.mark.parametrize("count", [5, 70])
@pytest.mark.parametrize("schedule", ["one_pass", "chained"])
def test_states_of_a_pool_in_place(count, schedule):
    """state_out is state_in: the first tile of a sequence reads the row that the last one
    writes; rows of the pool that no sequence has stay."""
    lengths = [(97 * i * i + 13 * i) % 700 for i in range(count)]
    inp = make_scan(lengths, 136, F32, "sigmoid", pool=count + 6, seed=17, device=DEV)
    pool = inp["state"].clone()
    kw = dict(state_slots=inp["slots"], schedule=schedule)
    o, out = _prefill(inp, "sigmoid", "complement", state_in=pool, state_out=pool, **kw)
    assert out is pool
    other = inp["state"].clone()
    o2, _ = _prefill(inp, "sigmoid", "complement", state_out=other, **kw)
    assert torch.equal(o, o2) and torch.equal(pool, other)
    check_scan(o, pool[inp["slots"].long()], inp, "sigmoid", "complement")
    rest = torch.ones(count + 6, dtype=torch.bool, device=DEV)
    rest[inp["slots"].long()] = False
    assert torch.equal(pool[rest], inp["state"][rest])


def test_two_streams_at_once():
    """Calls that overlap on streams of their own, a workspace each."""
    a = make_scan([5000], 264, F32, "log", seed=14, device=DEV)
    b = make_scan([2500, 2500], 264, F32, "log", seed=15, device=DEV)
    want = [_prefill(i, "log", "plain", schedule="chained") for i in (a, b)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(8):
        for k, i in enumerate((a, b)):
            got[k].append(_prefill(i, "log", "plain", schedule="chained", stream=streams[k]))
    torch.cuda.synchronize()
    for k in range(2):
        for o, s in got[k]:
            assert torch.equal(o, want[k][0]) and torch.equal(s, want[k][1])


def test_automatic_schedule_and_no_workspace():
    inp = make_scan([300, 5], 136, F32, "log", seed=16, device=DEV)
    whole = _prefill(inp, "log", "plain", schedule="one_pass")
    for kw in ({"workspace": None}, {"workspace": False}, {"workspace": None, "cu_seqlens_host": inp["cu_host"]}):
        got = _prefill(inp, "log", "plain", **kw)
        assert all(torch.equal(p, q) for p, q in zip(whole, got))
    check_scan(*_prefill(inp, "log", "plain", cu_seqlens_host=[0, 300, 305]), inp, "log", "plain")


def test_tensors_past_32_bits():
    """More than 2^31 elements in each tensor, and tokens 2 MB apart over 10 GB: the last rows
    against the recurrence over the tokens that still count."""
    T, C = 270000, 8192
    x = torch.randn(T, C, device=DEV, dtype=BF)
    g = torch.full((T, C), -1.0, device=DEV, dtype=BF)
    assert x.numel() > 1 << 31
    for schedule in ("chained", "one_pass"):
        o, state = kda.kda_gated_scan_prefill(x, g, state_out=True, schedule=schedule)
        cols = torch.tensor([0, 5, 4097, 8191], device=DEV)
        tail = {"x": x[-150:, cols], "gate": g[-150:, cols], "state": None, "slots": None, "lengths": [150]}
        ro, rs, eo, es = scan_ref(tail, "log", "plain")  # e^-150 of what stands before
        check(o[-40:, cols], ro[-40:], 2.0 ** -8 * ro[-40:].abs() + eo[-40:] + 1e-30, schedule + " o")
        check(state[:, cols], rs, U32 * rs.abs() + es + 1e-30, schedule + " state")
        dx, dg, _ = kda.kda_gated_scan_backward(x, g, o, schedule=schedule)
        (rx, rg, _), (ex, eg, _) = backward_ref(tail, x[-150:, cols], o[-150:, cols], None, "log", "plain")
        check(dx[-100:, cols], rx[-100:], 2.0 ** -8 * rx[-100:].abs() + ex[-100:] + 1e-30, schedule + " dx")
        check(dg[-100:, cols], rg[-100:], 2.0 ** -8 * rg[-100:].abs() + eg[-100:] + 1e-30, schedule + " dgate")
        del o, dx, dg
    del x, g
    wide = torch.empty(5000, 1 << 20, dtype=BF, device=DEV)
    inp = make_scan([5000], 120, BF, "log", seed=17, device=DEV)
    x, g, o = wide[:, :120], wide[:, 500000:500120], wide[:, 1000000:1000120]
    x.copy_(inp["x"])
    g.copy_(inp["gate"])
    _, state = kda.kda_gated_scan_prefill(x, g, state_in=inp["state"], state_out=True, o=o)
    want = kda.kda_gated_scan_prefill(inp["x"], inp["gate"], state_in=inp["state"], state_out=True)
    assert torch.equal(o, want[0]) and torch.equal(state, want[1])


def test_empty_batches():
    for dtype in (BF, F32):
        x = torch.empty(0, 16, dtype=dtype, device=DEV)
        s = torch.randn(2, 16, device=DEV)
        cu = torch.zeros(3, dtype=torch.int32, device=DEV)
        for kw in ({}, {"schedule": "chained"}):
            o, st = kda.kda_gated_scan_prefill(x, x.clone(), cu_seqlens=cu, state_in=s, state_out=True, **kw)
            assert o.shape == (0, 16) and torch.equal(st, s)
            _, st = kda.kda_gated_scan_prefill(x, x.clone(), cu_seqlens=cu, state_out=True, **kw)
            assert (st == 0).all()
            dx, dg, ds = kda.kda_gated_scan_backward(x, x.clone(), o, cu_seqlens=cu, dstate_out=s, dstate_in=True, **kw)
            assert torch.equal(ds, s) and dx.shape == (0, 16)
