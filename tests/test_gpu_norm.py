"""kda_qk_norm_rope and kda_gated_norm against their formulas in 64 bits, and the run
of norms, linear attention and output norm as a layer uses them.  The bounds are
derived in _linattn_common."""
import pytest
import torch

import gated_delta_rule_short_amd as kda
from tests._linattn_common import DEV, U16, check, gated_ref, linattn_ref, make_linattn, rope_ref

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _lib():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    kda.load_library()


def _rand(shape, seed, dtype=F32):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).to(dtype).to(DEV)


def _freq(R):
    return (1e6 ** (-2.0 * torch.arange(R // 2, dtype=torch.float64) / R)).float().to(DEV)


@pytest.mark.parametrize("T,Hq,Hk", [(1, 1, 1), (1, 64, 64), (5, 7, 3), (130, 16, 4), (33, 40, 8)])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("norm", ["rms", "l2", "none"])
def test_qk_norm_rope(T, Hq, Hk, D, dtype, norm):
    q, k = _rand((T, Hq, D), T, dtype), _rand((T, Hk, D), T + 1, dtype)
    w = (_rand((D,), 2), None) if norm == "rms" else (None, None)
    pos = torch.randint(0, 1 << 20, (T,), generator=torch.Generator().manual_seed(3)).to(torch.int32).to(DEV)
    pos[0] = 2147483647 if T > 1 else 0
    fr = _freq(D)
    qo, ko = kda.kda_qk_norm_rope(q, k, norm=norm, q_weight=w[0], k_weight=w[1], positions=pos, inv_freq=fr)
    for x, y, wt in ((q, qo, w[0]), (k, ko, w[1])):
        ref, bound = rope_ref(x, wt, norm, 1e-6, pos, fr, False)
        check(y, ref, bound, norm)


@pytest.mark.parametrize("D,R", [(64, 16), (64, 48), (128, 16), (128, 64), (128, 96), (128, 112), (128, 0)])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_partial_rotations(D, R, interleaved, dtype):
    q, k = _rand((9, 5, D), 1, dtype), _rand((9, 2, D), 2, dtype)
    pos = torch.arange(9, dtype=torch.int32, device=DEV) * 7777 - 20000 if R else None
    fr = _freq(R) if R else None
    qo, ko = kda.kda_qk_norm_rope(q, k, norm="l2", positions=pos, inv_freq=fr, interleaved=interleaved)
    for x, y in ((q, qo), (k, ko)):
        ref, bound = rope_ref(x, None, "l2", 1e-6, pos, fr, interleaved)
        check(y, ref, bound, "R=%d" % R)


def test_qk_norm_rope_packed_in_place_and_alone():
    """q and k inside a packed projection, written where they lie; the values beside them
    stay; q alone gives the same."""
    T, H, Hk, D = 37, 6, 2, 128
    x = _rand((T, (H + 2 * Hk) * D), 4, BF)
    before = x.clone()
    q = x[:, :H * D].unflatten(1, (H, D))
    k = x[:, H * D:(H + Hk) * D].unflatten(1, (Hk, D))
    pos, fr = torch.arange(T, dtype=torch.int32, device=DEV), _freq(D)
    qo, ko = kda.kda_qk_norm_rope(q.clone(), k.clone(), positions=pos, inv_freq=fr)
    only, none = kda.kda_qk_norm_rope(q, positions=pos, inv_freq=fr)
    assert none is None and torch.equal(only, qo)
    a, b = kda.kda_qk_norm_rope(q, k, positions=pos, inv_freq=fr, q_out=q, k_out=k)
    assert a is q and b is k and torch.equal(q, qo) and torch.equal(k, ko)
    assert torch.equal(x[:, (H + Hk) * D:], before[:, (H + Hk) * D:])


def test_norms_of_zero_huge_and_non_finite_rows():
    q = _rand((4, 3, 128), 5)
    q[0, 1] = 0.0
    q[1, 2] = q[1, 2] * 1e18
    q[2, 0] = q[2, 0] * 1e-18
    clean, _ = kda.kda_qk_norm_rope(q)
    ref, bound = rope_ref(q, None, "rms", 1e-6, None, None, False)
    check(clean, ref, bound, "rows")
    q[3, 1, 5] = float("nan")
    y, _ = kda.kda_qk_norm_rope(q)
    keep = torch.ones(4, 3, dtype=torch.bool, device=DEV)
    keep[3, 1] = False
    assert torch.equal(y[keep], clean[keep]) and torch.isnan(y[3, 1]).all()
    z = kda.kda_gated_norm(q, torch.full_like(q, -200.0))
    assert (z[keep] == 0).all()


@pytest.mark.parametrize("T,H", [(0, 3), (1, 1), (1, 64), (5, 7), (301, 16)])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("act,weight", [("sigmoid", "shared"), ("silu", "head"), ("none", "none"), ("silu", "none")])
def test_gated_norm(T, H, D, dtype, act, weight):
    x = _rand((T, H, D), T, dtype)
    z = None if act == "none" else (3 * _rand((T, H, D), T + 1)).to(dtype)
    w = None if weight == "none" else _rand((H, D) if weight == "head" else (D,), 2)
    y = kda.kda_gated_norm(x, z, w, act="sigmoid" if act == "none" else act, eps=1e-5)
    ref, bound = gated_ref(x, z, w, act, 1e-5)
    check(y, ref, bound, "y")


def test_gated_norm_strided_and_in_place():
    T, H, D = 50, 4, 128
    wide = _rand((T, 3 * H * D + 8), 6, BF)
    x, z = wide[:, :H * D].unflatten(1, (H, D)), wide[:, H * D:2 * H * D].unflatten(1, (H, D))
    rest = wide[:, 2 * H * D:].clone()
    y = kda.kda_gated_norm(x.contiguous(), z)
    assert torch.equal(kda.kda_gated_norm(x, z), y)
    x2 = x.contiguous()
    assert kda.kda_gated_norm(x2, z, y=x2) is x2 and torch.equal(x2, y)
    assert torch.equal(kda.kda_gated_norm(x, z, y=z), y)
    assert torch.equal(wide[:, 2 * H * D:], rest)


def test_many_rows():
    """More rows than one launch's workgroups hold side by side, sampled."""
    T, H, D = 40000, 16, 64
    x, z = torch.randn(T, H, D, device=DEV).to(BF), torch.randn(T, H, D, device=DEV).to(BF)
    y = kda.kda_gated_norm(x, z)
    pos = torch.randint(0, 1 << 20, (T,), device=DEV, dtype=torch.int32)
    q, _ = kda.kda_qk_norm_rope(x, positions=pos, inv_freq=_freq(64))
    at = torch.tensor([0, 1, 777, 19999, 39998, 39999], device=DEV)
    ref, bound = gated_ref(x[at], z[at], None, "sigmoid", 1e-6)
    check(y[at], ref, bound, "y")
    ref, bound = rope_ref(x[at], None, "rms", 1e-6, pos[at], _freq(64), False)
    check(q[at], ref, bound, "q")


def _layer(x, H, Hk, D, pos, fr, ld, state, cu=None, decode=False, o_w=None):
    q, k, v, z = x.split([H * D, Hk * D, H * D, H * D], dim=1)
    q, k = kda.kda_qk_norm_rope(q.unflatten(1, (H, D)), k.unflatten(1, (Hk, D)), positions=pos, inv_freq=fr)
    # every query head has its own decay; keys are shared by its group
    k = k.repeat_interleave(H // Hk, 1)
    v = v.unflatten(1, (H, D))
    if decode:
        o = kda.kda_linattn_decode(q, k, v, ld, state)
    else:
        o, _ = kda.kda_linattn_prefill(q, k, v, ld, cu_seqlens=cu, state_in=state, state_out=state)
    return kda.kda_gated_norm(o, z.unflatten(1, (H, D)), o_w), (q, k, v, o)


def test_layer_run_prompts_then_tokens():
    """Packed projections -> q/k norm and rotation -> linear attention -> gated norm: two
    prompts, then three decode steps, each stage against 64 bits on its own inputs."""
    H, Hk, D, lengths = 4, 2, 128, [70, 33]
    T, N = sum(lengths), 2
    fr, w = _freq(D), _rand((D,), 30)
    ld = -torch.rand(T, H, generator=torch.Generator().manual_seed(31)).to(DEV)
    cu = torch.tensor([0, 70, 103], dtype=torch.int32, device=DEV)
    state = _rand((N, H, D, D), 32)
    pos = torch.cat([torch.arange(n) for n in lengths]).to(torch.int32).to(DEV)
    length = list(lengths)
    for step in range(4):
        x = _rand(((T if step == 0 else N), (3 * H + Hk) * D), 40 + step, BF)
        g = ld if step == 0 else ld[:N]
        s0 = state.clone()
        y, (q, k, v, o) = _layer(x, H, Hk, D, pos, fr, g, state, cu, step > 0, w)
        raw_q, raw_k, _, z = x.split([H * D, Hk * D, H * D, H * D], dim=1)
        for a, b in ((raw_q.unflatten(1, (H, D)), q), (raw_k.unflatten(1, (Hk, D)), k[:, ::H // Hk])):
            ref, bound = rope_ref(a, None, "rms", 1e-6, pos, fr, False)
            check(b, ref, bound, "q/k at step %d" % step)
        inp = {"q": q, "k": k, "v": v, "log_decay": g, "state": s0, "slots": None,
               "lengths": lengths if step == 0 else [1, 1]}
        ref, rs, oa, sa = linattn_ref(inp)
        check(o, ref, U16 * ref.abs() + 1.05 * U16 * oa, "o at step %d" % step)
        check(state, rs, 4e-5 * sa, "state at step %d" % step)
        ref, bound = gated_ref(o, z.unflatten(1, (H, D)), w, "sigmoid", 1e-6)
        check(y, ref, bound, "y at step %d" % step)
        pos = torch.tensor(length, dtype=torch.int32, device=DEV)
        length = [n + 1 for n in length]
