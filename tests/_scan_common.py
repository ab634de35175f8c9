"""Inputs, the plain 64-bit forms and the error bounds of the gated-scan and residual-norm
tests.

Bounds are element by element and follow from the arithmetic.  u32 = 2^-24 is half a step
of fp32 and u16 = 2^-8 half a step of bf16.  For the recurrence, A is the state over
absolute values (the sum of |terms| of h) and E an error that obeys
    E_t = a (E_{t-1} + k_t A_{t-1}) + e_t |b x| + 4 u32 A_t
  * k_t, the relative error of a decay: logarithms are summed over up to 128 tokens, each
    addition rounding a partial sum, so that a token's own log2 a, l, is charged 128 |l| u32,
    the few steps of a logarithm's own formation 12 |l| u32, a rounded argument |z| of the
    exponential in it 4 |z| |l| u32, and the exponentials of a tile's joins 8 u32;
  * e_t, the relative error of b: 17 u32 where 1 - a is a difference (at 1/8 and above),
    a series or an exponential of a rounded argument, 4 |z| u32: 32 + 4 |z| in all;
  * 4 u32 for the roundings of a step.
A bf16 output or state is rounded once: u16 of its value more, and of nothing else."""
import torch

U32 = 2.0 ** -24
U16 = torch.finfo(torch.bfloat16).eps / 2
TINY = 1e-36  # results near the end of fp32's range may be flushed
DEV = torch.device("cuda:0")
BF, F32 = torch.bfloat16, torch.float32
KINDS = [(g, i) for g in ("log", "sigmoid") for i in ("plain", "complement", "norm")]


def half_step(dtype):
    return U16 if dtype == BF else U32


def make_scan(lengths, C, dtype=F32, gate="log", state_dtype=F32, initial=True, pool=0, packed=False, seed=0,
              device="cpu"):
    """Inputs drawn on the host, moved to `device`; channels forget within a token up to
    hundreds of tokens."""
    gen = torch.Generator().manual_seed(seed)
    T, N = sum(lengths), len(lengths)
    spread = torch.rand(C, generator=gen)
    z = torch.randn(T, C, generator=gen)
    z = -torch.exp2(2.0 - 11.0 * spread) * torch.rand(T, C, generator=gen) if gate == "log" else z + 9.0 * spread - 2.0
    x = torch.randn(T, C, generator=gen)
    if packed:
        w = torch.randn(T, 2 * C + 24, generator=gen)
        w[:, 8:8 + C], w[:, 16 + C:16 + 2 * C] = x, z
        w = w.to(dtype).to(device)
        x, z = w[:, 8:8 + C], w[:, 16 + C:16 + 2 * C]
    else:
        x, z = x.to(dtype).to(device), z.to(dtype).to(device)
    rows = pool or N
    state = torch.randn(rows, C, generator=gen).to(state_dtype).to(device) if initial else None
    slots = torch.randperm(rows, generator=gen)[:N].to(torch.int32).to(device) if pool else None
    cu = torch.tensor([0] + list(lengths)).cumsum(0).to(torch.int32)
    return {"x": x, "gate": z, "state": state, "slots": slots, "cu_host": cu, "cu": cu.to(device),
            "lengths": list(lengths)}


def factors(z, gate, inputs):
    """(a, b, |log2 a|, da/dz, -db/da) in 64 bits."""
    if gate == "log":
        g = z.clamp(max=0.0)
        a, c, da = g.exp(), -torch.expm1(g), torch.where(z > 0, 0.0, g.exp())
        l = g.abs() * 1.4426950408889634
    else:
        a, c = torch.sigmoid(z), torch.sigmoid(-z)
        da, l = a * c, torch.nn.functional.softplus(-z) * 1.4426950408889634
    b = {"plain": torch.ones_like(a), "complement": c, "norm": (c * (1.0 + a)).sqrt()}[inputs]
    q = {"plain": torch.zeros_like(a), "complement": torch.ones_like(a),
         "norm": torch.where(b > 0, a / b.clamp(min=1e-300), 0.0)}[inputs]
    return a, b, l, da, q


def _first(inp, C):
    N = len(inp["lengths"])
    if inp["state"] is None:
        return torch.zeros(N, C, dtype=torch.float64)
    rows = inp["slots"].cpu().long() if inp["slots"] is not None else torch.arange(N)
    return inp["state"].cpu().double()[rows]


def scan_ref(inp, gate, inputs):
    """Token by token: (o, final states [N], error bounds of both without their rounding)."""
    x, z = inp["x"].cpu().double(), inp["gate"].cpu().double()
    T, C = x.shape
    a, b, l, _, _ = factors(z, gate, inputs)
    k = ((140 + 4 * z.abs()) * l + 8) * U32
    e = (32 + 4 * z.abs()) * U32 if inputs != "plain" else torch.zeros_like(z)
    h = _first(inp, C)
    A, E = h.abs(), torch.zeros_like(h)
    o, eo = torch.zeros(T, C, dtype=torch.float64), torch.zeros(T, C, dtype=torch.float64)
    t = 0
    for n, L in enumerate(inp["lengths"]):
        for t in range(t, t + L):
            u = b[t] * x[t]
            E[n] = a[t] * (E[n] + k[t] * A[n]) + e[t] * u.abs()
            h[n] = a[t] * h[n] + u
            A[n] = a[t] * A[n] + u.abs()
            E[n] += 4 * U32 * A[n]
            o[t], eo[t] = h[n], E[n]
        t = sum(inp["lengths"][:n + 1])
    return o, h, eo, E


def backward_ref(inp, d_o, o, dstate, gate, inputs):
    """(dx, dgate, dstate_in) in 64 bits and their bounds without the last rounding; o is the
    forward pass's output as it was stored."""
    x, z, d, hs = (t.cpu().double() for t in (inp["x"], inp["gate"], d_o, o))
    T, C = z.shape
    a, b, l, da, q = factors(z, gate, inputs)
    k = ((140 + 4 * z.abs()) * l + 8) * U32
    e = (64 + 8 * z.abs()) * U32
    h0 = _first(inp, C)
    r = dstate.cpu().double().clone() if dstate is not None else torch.zeros_like(h0)
    A, E = r.abs(), torch.zeros_like(r)
    dx, dg, ex, eg = (torch.zeros(T, C, dtype=torch.float64) for _ in range(4))
    end = T
    for n in reversed(range(len(inp["lengths"]))):
        begin = end - inp["lengths"][n]
        for t in range(end - 1, begin - 1, -1):
            dh, dA, dE = d[t] + r[n], d[t].abs() + A[n], E[n] + 2 * U32 * (d[t].abs() + A[n])
            before = hs[t - 1] if t > begin else h0[n]
            part, mod = before - x[t] * q[t], before.abs() + (x[t] * q[t]).abs()
            dx[t], ex[t] = b[t] * dh, b[t] * (dE + e[t] * dA)
            dg[t], eg[t] = dh * da[t] * part, da[t] * (dE * mod + (e[t] + k[t]) * dA * mod)
            r[n], A[n], E[n] = a[t] * dh, a[t] * dA, a[t] * (dE + k[t] * dA)
            E[n] += 2 * U32 * A[n]
        end = begin
    return (dx, dg, r), (ex, eg, E)


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


def check_scan(o, state, inp, gate, inputs, what=""):
    """o [T, C] and the final states [N, C] (None: not checked) against the recurrence."""
    ro, rs, eo, es = scan_ref(inp, gate, inputs)
    check(o, ro, half_step(o.dtype) * ro.abs() + eo + TINY, what + " o")
    if state is not None:
        check(state, rs, half_step(state.dtype) * rs.abs() + es + TINY, what + " state")


def check_backward(got, inp, d_o, o, dstate, gate, inputs, what=""):
    refs, errs = backward_ref(inp, d_o, o, dstate, gate, inputs)
    for x, ref, err, name in zip(got, refs, errs, ("dx", "dgate", "dstate_in")):
        if x is not None:
            check(x, ref, half_step(x.dtype) * ref.abs() + err + TINY, what + " " + name)


def norm_ref(x, residual, weight, eps):
    """(s, y, bound of y without its rounding): a sum of C squares in parts of 64 lanes and
    more (at most C / 64 + 16 roundings of it, halved by the root), the root, and three
    products; the sum x + r itself 1 u32 of s."""
    s = x.cpu().double()
    if residual is not None:
        s = s + residual.cpu().double()
    y = s / (s.square().mean(-1, keepdim=True) + eps).sqrt()
    if weight is not None:
        y = y * weight.cpu().double()
    return s, y, (x.shape[1] / 64 + 24) * U32 * y.abs()


def norm_backward_ref(dy, s, weight, eps, dresidual):
    """(dx, dweight) in 64 bits and their bounds without the last rounding.  The two sums
    over C channels err by C / 64 + 16 roundings of their moduli, the sum over T tokens by
    its length."""
    g, s = dy.cpu().double(), s.cpu().double()
    T, C = s.shape
    w = weight.cpu().double() if weight is not None else torch.ones(C, dtype=torch.float64)
    r = 1.0 / (s.square().mean(-1, keepdim=True) + eps).sqrt()
    n = s * r
    gw = g * w
    dot, mod = (gw * n).mean(-1, keepdim=True), (gw * n).abs().mean(-1, keepdim=True)
    dx = (gw - n * dot) * r
    k = (C / 64 + 40) * U32
    err = k * (gw.abs() + 3 * n.abs() * mod) * r
    if dresidual is not None:
        dx = dx + dresidual.cpu().double()
        err = err + 2 * U32 * dresidual.cpu().double().abs()
    dw = (g * n).sum(0)
    return dx, dw, err, (C / 64 + T + 64) * U32 * (g * n).abs().sum(0)
