"""Inputs, the plain 64-bit forms and the error bounds of the linear-attention and
per-head norm tests.

Bounds are element by element and follow from the arithmetic.  u32 = 2^-24 is half a
step of fp32 and u16 = 2^-8 (finfo(bf16).eps / 2) half a step of bf16.  The recurrence
over absolute values (every q, k, v and state replaced by its modulus) gives
o_abs >= sum of |terms of o| and s_abs >= sum of |terms of S|, so
  * fp32 arithmetic errs by at most n u32 of those sums, n counting the roundings a
    term can meet: a sum over dk = 128 keys and one over a chunk of 64 tokens, the
    decays (exp with an argument of up to 88 rounded once, a few units of its own), and
    one more for each token the state has been carried over: n = 320 + T;
  * where a matrix-core product takes operands rounded to bf16 (the decayed scores, the
    state under q), each term errs by at most u16 more: o by u16 o_abs;
  * the write k (decay v)^T splits its rounded operand into two bf16 parts, which leaves
    u16^2 = 2^-16 of s_abs;
  * a bf16 output or state is rounded once: u16 of its value, and of nothing else."""
import torch

U32 = 2.0 ** -24
U16 = torch.finfo(torch.bfloat16).eps / 2
TINY = 1e-37  # results below fp32's normal range may be flushed
DEV = torch.device("cuda:0")


def half_step(dtype):
    return U16 if dtype == torch.bfloat16 else 0.0  # fp32 rounding is in n


def make_linattn(lengths, H, Hk, dk, dv, dtype=torch.bfloat16, state_dtype=torch.float32, decay="token",
                 initial=True, pool=0, packed=False, seed=0, device="cpu"):
    """Inputs drawn on the host, moved to `device`.  Heads forget within a token up to
    hundreds of tokens."""
    g = torch.Generator().manual_seed(seed)
    T, N = sum(lengths), len(lengths)
    widths = [Hk * dk, Hk * dk, H * dv]
    if packed:
        x = torch.randn(T, sum(widths) + 16, generator=g).to(dtype).to(device)
        q, k, v, _ = x.split(widths + [16], dim=1)
    else:
        q, k, v = (torch.randn(T, w, generator=g).to(dtype).to(device) for w in widths)
    slope = torch.exp2(3.0 - 11.0 * torch.arange(H) / max(H - 1, 1))
    ld = -slope if decay == "head" else -slope * torch.rand(T, H, generator=g)
    rows = pool or N
    state = torch.randn(rows, H, dk, dv, generator=g).to(state_dtype).to(device) if initial else None
    slots = torch.randperm(rows, generator=g)[:N].to(torch.int32).to(device) if pool else None
    cu = torch.tensor([0] + lengths).cumsum(0).to(torch.int32)
    return {"q": q.unflatten(1, (Hk, dk)), "k": k.unflatten(1, (Hk, dk)), "v": v.unflatten(1, (H, dv)),
            "log_decay": ld.float().to(device), "state": state, "slots": slots, "cu_host": cu,
            "cu": cu.to(device), "lengths": lengths}


def linattn_ref(inp, scale=None):
    """Token by token in 64 bits on the CPU: (o, final states [N], o_abs, s_abs)."""
    q, k, v = (inp[n].cpu().double() for n in ("q", "k", "v"))
    T, Hk, dk = q.shape
    H, dv = v.shape[1:]
    scale = dk ** -0.5 if scale is None else scale
    rep = H // Hk
    q, k = q.repeat_interleave(rep, 1), k.repeat_interleave(rep, 1)
    ld = inp["log_decay"].cpu().double().clamp(max=0.0)
    a = ld.exp().expand(T, H)
    N = len(inp["lengths"])
    rows = inp["slots"].cpu().long() if inp["slots"] is not None else torch.arange(N)
    S = inp["state"].cpu().double()[rows] if inp["state"] is not None else torch.zeros(N, H, dk, dv,
                                                                                      dtype=torch.float64)
    A = S.abs()
    o, oa = torch.zeros(T, H, dv, dtype=torch.float64), torch.zeros(T, H, dv, dtype=torch.float64)
    cu = [0]
    for n in inp["lengths"]:
        cu.append(cu[-1] + n)
    for n in range(N):
        for t in range(cu[n], cu[n + 1]):
            w = a[t][:, None, None]
            S[n] = w * S[n] + k[t][:, :, None] * v[t][:, None, :]
            A[n] = w * A[n] + k[t].abs()[:, :, None] * v[t].abs()[:, None, :]
            o[t] = scale * (q[t][:, None, :] @ S[n])[:, 0]
            oa[t] = scale * (q[t].abs()[:, None, :] @ A[n])[:, 0]
    return o, S, oa, A


def check(x, ref, bound, what):
    """Every element within its bound (NaN never is)."""
    x = x.detach().cpu().double()
    over = (x - ref).abs() - bound
    bad = ~(over <= 0)
    if bad.any():
        i = int(torch.where(bad.flatten(), torch.nan_to_num(over.flatten(), nan=float("inf")), -1.0).argmax())
        raise AssertionError("%s: %d of %d outside, worst at %d: %r against %r, bound %.3g" % (
            what, int(bad.sum()), bad.numel(), i, float(x.flatten()[i]), float(ref.flatten()[i]),
            float(torch.as_tensor(bound).expand(x.shape).flatten()[i])))


def check_linattn(o, state, inp, matrix_cores, what=""):
    """o [T, H, dv] and the final states [N, H, dk, dv] (None: not checked) against the
    recurrence; matrix_cores: whether bf16 products are allowed their operand roundings."""
    ro, rs, oa, sa = linattn_ref(inp)
    n = (320 + max(inp["lengths"] + [0])) * U32
    mc = matrix_cores and inp["v"].dtype == torch.bfloat16
    check(o, ro, half_step(o.dtype) * ro.abs() + (n + (U16 if mc else 0.0)) * oa * 1.01 + TINY, what + " o")
    if state is not None:
        check(state, rs, half_step(state.dtype) * rs.abs() + (n + (U16 * U16 if mc else 0.0)) * sa * 1.01 + TINY,
              what + " state")


def rope_ref(x, weight, norm, eps, positions, inv_freq, interleaved):
    """(y, bound) of one tensor of kda_qk_norm_rope in 64 bits.  Roundings of a normalised
    element: half of the sum of squares' 128, the reciprocal root, scale and weight (80
    with slack); a rotation adds the reduced turn (2 pi 2^-25), sine and cosine and two
    products (16), on the moduli of both of its terms."""
    D = x.shape[-1]
    y = x.cpu().double()
    ss = y.square().sum(-1, keepdim=True)
    n = 0.0
    if norm == "rms":
        y = y / (ss / D + eps).sqrt()
        n = 80 * U32
        if weight is not None:
            y = y * weight.cpu().double()
    elif norm == "l2":
        y = y / (ss + eps).sqrt()
        n = 80 * U32
    mod = y.abs()
    if positions is not None:
        R = 2 * inv_freq.numel()
        th = (positions.cpu().double()[:, None] * inv_freq.cpu().double())[:, None]
        i = torch.arange(R // 2)
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + R // 2)
        ya, yb = y[..., a].clone(), y[..., b].clone()
        y[..., a], y[..., b] = ya * th.cos() - yb * th.sin(), yb * th.cos() + ya * th.sin()
        mod[..., a] = mod[..., b] = ya.abs() + yb.abs()
        n += 16 * U32
    return y, half_step(x.dtype) * y.abs() + n * mod + 4 * U32 * y.abs() + TINY


def gated_ref(x, gate, weight, act, eps):
    """(y, bound) of kda_gated_norm in 64 bits: 80 roundings as above, and for the gate the
    exponential of a rounded argument (2 |z| u32) with a few units for its parts (16)."""
    x, D = x.cpu(), x.shape[-1]
    y = x.double()
    y = y / (y.square().mean(-1, keepdim=True) + eps).sqrt()
    n = torch.full_like(y, 96.0)
    if weight is not None:
        y = y * weight.cpu().double()
    if gate is not None:
        z = gate.cpu().double()
        y = y / (1.0 + (-z).exp()) * (z if act == "silu" else 1.0)
        n = n + 2 * z.abs()
    return y, (half_step(x.dtype) + n * U32) * y.abs() + TINY
