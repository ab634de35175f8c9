"""kda_add_norm and kda_add_norm_backward against their formulas in 64 bits, and the runs
of the norm, the conv, the gated scan and the output norm as a layer uses them.  The bounds
are derived in _scan_common."""
import pytest
import torch

import gated_delta_rule_short_amd as kda
from tests._linattn_common import gated_ref
from tests._scan_common import (BF, DEV, F32, U16, U32, check, check_backward, check_scan, half_step, make_scan,
                                norm_backward_ref, norm_ref)

pytestmark = pytest.mark.gpu
E4 = torch.float8_e4m3fn
SIZES = [(1, 8), (5, 72), (37, 1000), (3, 4096), (2, 4104), (2, 16384), (2100, 520), (2050, 4096)]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    kda.load_library()


def _rand(shape, seed, dtype=F32, size=1.0):
    return (size * torch.randn(shape, generator=torch.Generator().manual_seed(seed))).to(dtype).to(DEV)


def check_quant(y, scale, ref, bound, group):
    """Codes and scales of y against the unrounded values: the scale is the largest modulus
    over 448, off by the bound there and two roundings; a value is then off by its bound and
    half an e4m3 step of itself (2^-4), or of the smallest normal value (2^-6, spacing 2^-9)."""
    T, C = ref.shape
    g = C if group == "token" else 128
    rb, bb = ref.reshape(T, -1, g), bound.reshape(T, -1, g)
    top = rb.abs().amax(-1)
    want = torch.where(top > 0, (top / 448).clamp(min=2.0 ** -126), 1.0)
    check(scale.reshape(T, -1), want, bb.amax(-1) / 448 * (top > 0) + 4 * U32 * want, "scale")
    sc = scale.cpu().double().reshape(T, -1, 1)
    got = y.cpu().float().double().reshape(T, -1, g)
    v = rb / sc
    check(got, v, (v.abs() * 2.0 ** -4).clamp(min=2.0 ** -10) * (1 + 1e-6) + bb / sc * 1.1 + 4 * U32 * v.abs(), "codes")


@pytest.mark.parametrize("T,C", SIZES)
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("quant", ["none", "token", "group"])
def test_add_norm(T, C, dtype, quant):
    if quant == "group":
        C = (C + 127) // 128 * 128
    for residual, weight in ((True, True), (False, True), (True, False)):
        x, r = _rand((T, C), T, dtype, 3.0), _rand((T, C), T + 1, dtype) if residual else None
        w = 1.0 + 0.2 * _rand((C,), 2) if weight else None
        y, scale, s = kda.kda_add_norm(x, r, w, quant=quant, eps=1e-5)
        ref_s, ref, bound = norm_ref(x, r, w, 1e-5)
        if residual:
            check(s, ref_s, half_step(dtype) * ref_s.abs(), "s")
        else:
            assert s is None
        if quant == "none":
            assert scale is None and y.dtype == dtype
            check(y, ref, half_step(dtype) * ref.abs() + bound, "y")
        else:
            assert y.dtype == E4
            check_quant(y, scale, ref, bound, quant)


@pytest.mark.parametrize("quant", ["none", "token", "group"])
def test_strides_and_in_place(quant):
    T, C = 70, 384
    wide = _rand((T, 3 * C + 8), 4, BF)
    x, r = wide[:, 8:C + 8], wide[:, C + 8:2 * C + 8]
    rest = torch.cat([wide[:, :8], wide[:, 2 * C + 8:]], 1)
    y, scale, s = kda.kda_add_norm(x.contiguous(), r.contiguous(), quant=quant)
    for target in ("r", "x"):
        again = wide.clone()
        xa, ra = again[:, 8:C + 8], again[:, C + 8:2 * C + 8]
        out = ra if target == "r" else xa
        ybuf = torch.zeros(T, C + 40, dtype=y.dtype, device=DEV)[:, 8:8 + C]
        y2, scale2, s2 = kda.kda_add_norm(xa, ra, quant=quant, residual_out=out, y=ybuf)
        assert s2 is out and y2 is ybuf and torch.equal(s2, s) and torch.equal(y2.float(), y.float())
        assert scale is None or torch.equal(scale, scale2)
        assert torch.equal(torch.cat([again[:, :8], again[:, 2 * C + 8:]], 1), rest)
    y3, _, s3 = kda.kda_add_norm(x, r, quant=quant, residual_out=False)
    assert s3 is None and torch.equal(y3.float(), y.float())


@pytest.mark.parametrize("quant", ["none", "token", "group"])
def test_zero_huge_tiny_and_non_finite_rows(quant):
    x = _rand((6, 256), 5)
    x[0] = 0.0
    x[1] *= 1e16
    x[2] *= 1e-25
    x[3, 128:] = 0.0
    w = 1.0 + 0.1 * _rand((256,), 6)
    y, scale, _ = kda.kda_add_norm(x, None, w, quant=quant)
    _, ref, bound = norm_ref(x, None, w, 1e-6)
    if quant == "none":
        check(y, ref, (1 + 0) * U32 * ref.abs() + bound + 1e-36, "y")
    else:
        check_quant(y[:4], scale[:4], ref[:4], bound[:4], quant)
        assert (scale[0] == 1.0).all() and (y[0].float() == 0).all()
    clean = y.float().clone()
    x[4, 7] = float("nan")
    x[5, 200] = float("inf")
    y, scale, _ = kda.kda_add_norm(x, None, w, quant=quant)
    assert torch.equal(y[:4].float(), clean[:4]) and torch.isnan(y[4].float()).all()
    out = y.float() if scale is None else y.float() * (scale[:, None] if scale.dim() == 1 else scale.repeat_interleave(128, 1))
    if quant == "token":
        assert torch.isnan(out[4:]).all() and torch.isnan(scale[4:]).all()
    else:  # an infinite row: zeros, and NaN at the infinity (its 128 channels)
        nan = torch.isnan(out[5])
        assert nan[200] and (out[5][~nan] == 0).all() and int(nan.sum()) == (1 if quant == "none" else 128)


def test_tiny_weights_keep_a_normal_scale():
    x = _rand((3, 128), 7)
    w = torch.full((128,), 1e-37, device=DEV)
    y, scale, _ = kda.kda_add_norm(x, None, w, quant="token")
    assert (scale == 2.0 ** -126).all()
    _, ref, bound = norm_ref(x, None, w, 1e-6)
    check(y.float(), ref * 2.0 ** 126, (ref.abs() * 2.0 ** 126 * 2.0 ** -4).clamp(min=2.0 ** -10) * 1.001 + bound * 2.0 ** 126 + 0.05, "codes")


@pytest.mark.parametrize("T,C", SIZES + [(600, 128)])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_add_norm_backward(T, C, dtype):
    for weight, stream, dweight in ((True, True, True), (False, False, True), (True, False, False)):
        dy, s = _rand((T, C), T, dtype), _rand((T, C), T + 1, dtype, 2.0)
        w = 1.0 + 0.2 * _rand((C,), 2) if weight else None
        dr = _rand((T, C), T + 2, dtype) if stream else None
        dx, dw = kda.kda_add_norm_backward(dy, s, w, eps=1e-5, dresidual=dr, dweight=dweight)
        rx, rw, ex, ew = norm_backward_ref(dy, s, w, 1e-5, dr)
        check(dx, rx, half_step(dtype) * rx.abs() + ex, "dx")
        if dweight:
            check(dw, rw, U32 * rw.abs() + ew, "dweight")
            again = kda.kda_add_norm_backward(dy, s, w, eps=1e-5, dresidual=dr)[1]
            assert torch.equal(dw, again)
        else:
            assert dw is None


def test_rows_past_one_launch_and_past_32_bits():
    """More rows than one launch has workgroups, and more elements than 2^31, sampled."""
    for T, C in ((1048576 + 77, 64), (280000, 8192)):
        x = torch.randn(T, C, device=DEV, dtype=BF)
        at = torch.tensor([0, 1, T // 2, T - 78, T - 2, T - 1], device=DEV)
        y, scale, s = kda.kda_add_norm(x, x, quant="token")
        rs, ref, bound = norm_ref(x[at], x[at], None, 1e-6)
        check(s[at], rs, U16 * rs.abs(), "s")
        check_quant(y[at], scale[at], ref, bound, "token")
        dx, _ = kda.kda_add_norm_backward(x, s, dweight=False)
        rx, _, ex, _ = norm_backward_ref(x[at], s[at], None, 1e-6, None)
        check(dx[at], rx, U16 * rx.abs() + ex, "dx")
        del x, y, s, dx


def test_add_norm_backward_in_place_strided_and_empty():
    T, C = 40, 264
    wide = _rand((T, 3 * C + 16), 8, BF)
    dy, s, dr = (wide[:, i * C:(i + 1) * C] for i in range(3))
    want, dw = kda.kda_add_norm_backward(dy.contiguous(), s.contiguous(), dresidual=dr.contiguous())
    for i in range(3):
        again = wide.clone()
        parts = [again[:, k * C:(k + 1) * C] for k in range(3)]
        dx, dw2 = kda.kda_add_norm_backward(parts[0], parts[1], dresidual=parts[2], dx=parts[i])
        assert dx is parts[i] and torch.equal(dx, want) and torch.equal(dw, dw2)
        assert torch.equal(again[:, 3 * C:], wide[:, 3 * C:])
    e = torch.empty(0, C, device=DEV)
    dx, dw = kda.kda_add_norm_backward(e, e.clone())
    assert dx.shape == (0, C) and (dw == 0).all()
    y, scale, s = kda.kda_add_norm(e, e.clone(), quant="token")
    assert y.shape == (0, C) and scale.shape == (0,) and s.shape == (0, C)


def test_backward_against_differences():
    """dx and dweight against autograd and central differences of the 64-bit formula."""
    T, C = 3, 16
    dy, s, dr = _rand((T, C), 20), _rand((T, C), 21), _rand((T, C), 22)
    w = 1.0 + 0.2 * _rand((C,), 23)
    dx, dw = kda.kda_add_norm_backward(dy, s, w, dresidual=dr)
    S, W = s.cpu().double().requires_grad_(True), w.cpu().double().requires_grad_(True)

    def scalar(a, b):
        y = a / (a.square().mean(-1, keepdim=True) + 1e-6).sqrt() * b
        return (y * dy.cpu().double()).sum() + (a * dr.cpu().double()).sum()
    gs, gw = torch.autograd.grad(scalar(S, W), (S, W))
    _, _, ex, ew = norm_backward_ref(dy, s, w, 1e-6, dr)
    check(dx, gs, ex + U32 * gs.abs(), "dx")
    check(dw, gw, ew + U32 * gw.abs(), "dweight")
    with torch.no_grad():
        for leaf, g in ((S, gs), (W, gw)):
            for i in range(0, leaf.numel(), 5):
                old, eps = leaf.view(-1)[i].item(), 1e-5
                leaf.view(-1)[i] = old + eps
                up = scalar(S, W)
                leaf.view(-1)[i] = old - eps
                down = scalar(S, W)
                leaf.view(-1)[i] = old
                assert abs(float((up - down) / (2 * eps)) - float(g.view(-1)[i])) < 1e-7 * 100


def test_captured_norms_replay():
    T, C = 300, 1000
    x, r, w = _rand((T, C), 24, BF), _rand((T, C), 25, BF), 1.0 + 0.1 * _rand((C,), 26)
    y, scale = torch.empty(T, C, dtype=E4, device=DEV), torch.empty(T, device=DEV)
    s, dx, dw = torch.empty_like(x), torch.empty_like(x), torch.empty(C, device=DEV)
    ws = torch.empty(4 << 20, dtype=torch.uint8, device=DEV)

    def step():
        kda.kda_add_norm(x, r, w, quant="token", residual_out=s, y=y, scale=scale)
        kda.kda_add_norm_backward(r, s, w, dx=dx, dweight=dw, workspace=ws)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for i in range(4):
        x.copy_(_rand((T, C), 30 + i, BF))
        g.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (y.float(), scale, s, dx, dw)]
        y2, sc2, s2 = kda.kda_add_norm(x, r, w, quant="token")
        b = kda.kda_add_norm_backward(r, s2, w)
        assert all(torch.equal(p, q) for p, q in zip(got, (y2.float(), sc2, s2) + b)), i


def test_layer_run_prompts_then_tokens_and_gradients():
    """Residual norm in 8 bits -> in-projection -> conv -> gated scan -> per-head output norm,
    two prompts and then three decode steps, and the gradients of scan and norm: each stage
    against 64 bits on its own inputs."""
    C, H, lengths = 256, 2, [140, 33]
    T, N = sum(lengths), 2
    w = 1.0 + 0.1 * _rand((C,), 40)
    proj = _rand((C, 3 * C), 41, F32, C ** -0.5)
    taps = _rand((C, 4), 42, F32, 0.5)
    cu = torch.tensor([0, 140, 173], dtype=torch.int32, device=DEV)
    state, conv_state = torch.zeros(N, C, device=DEV), torch.zeros(N, 3, C, dtype=BF, device=DEV)
    stream = _rand((T, C), 43, BF)
    for step in range(4):
        n = T if step == 0 else N
        x = _rand((n, C), 44 + step, BF)
        if step:
            stream = _rand((n, C), 50 + step, BF)
        y, scale, s = kda.kda_add_norm(x, stream, w, quant="group")
        rs, ref, bound = norm_ref(x, stream, w, 1e-6)
        check(s, rs, U16 * rs.abs(), "s at step %d" % step)
        check_quant(y, scale, ref, bound, "group")
        p = ((y.float() * scale.repeat_interleave(128, 1)) @ proj).to(BF)
        u, gate, z = p[:, :C], p[:, C:2 * C], p[:, 2 * C:]
        bounds = cu if step == 0 else torch.arange(N + 1, dtype=torch.int32, device=DEV)
        u, conv_state = kda.kda_short_conv(u.contiguous(), taps, cu_seqlens=bounds, conv_state_in=conv_state,
                                           conv_state_out=conv_state)
        s0 = state.clone()
        if step == 0:
            o, state = kda.kda_gated_scan_prefill(u, gate, gate_kind="sigmoid", input_kind="complement", cu_seqlens=cu,
                                                  state_in=state, state_out=state)
        else:
            o = kda.kda_gated_scan_decode(u, gate, state, gate_kind="sigmoid", input_kind="complement")
        inp = {"x": u, "gate": gate, "state": s0, "slots": None, "lengths": lengths if step == 0 else [1, 1]}
        check_scan(o, state, inp, "sigmoid", "complement", "step %d" % step)
        out = kda.kda_gated_norm(o.unflatten(1, (H, 128)), z.unflatten(1, (H, 128)), act="silu")
        gref, gb = gated_ref(o.unflatten(1, (H, 128)), z.unflatten(1, (H, 128)), None, "silu", 1e-6)
        check(out, gref, gb, "out at step %d" % step)
        if step == 0:
            d_o, ds = _rand((T, C), 60, BF), _rand((N, C), 61)
            got = kda.kda_gated_scan_backward(d_o, gate, o, u, gate_kind="sigmoid", input_kind="complement",
                                              cu_seqlens=cu, state_in=s0, dstate_out=ds, dstate_in=True)
            check_backward(got, inp, d_o, o, ds, "sigmoid", "complement")
            dy = (torch.cat([got[0], got[1], torch.zeros_like(d_o)], 1).float() @ proj.t()).to(BF)
            dx, dw = kda.kda_add_norm_backward(dy, s, w, dresidual=d_o)
            rx, rw, ex, ew = norm_backward_ref(dy, s, w, 1e-6, d_o)
            check(dx, rx, U16 * rx.abs() + ex, "dx")
            check(dw, rw, U32 * rw.abs() + ew, "dweight")
