"""What is measured of the gated scan and the residual norm: their cases, the inputs, a
plain form of each in elementary torch operations, and the definition in 64 bits.

The operators (per token t of a sequence and channel, decay a, input factor b):
  prefill   h_t = a_t h_{t-1} + b_t x_t over packed prompts
  decode    the same step for one new token of every sequence, state in place
  backward  the gradients of x, the gate and the initial state from those of h and the
            final state
  norm      s = x + residual, y = weight s / rms(s), in 8 bits with scales or not
  norm_grad the gradients of s and of the weight
with a = exp(min(g, 0)) (gate "log") or the logistic function ("sigmoid"), and b = 1
("plain"), 1 - a ("complement") or sqrt(1 - a^2) ("norm").

With `own` false `run` computes the plain form in float32; with `own` true it calls
the package's entry points on the same inputs.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
EPS = 1e-6
TOP = 448.0  # the largest e4m3 value


def _ragged(count, lo, hi, salt):
    """`count` lengths in [lo, hi], spread over their logarithm, as text."""
    out, x = [], salt
    for _ in range(count):
        x = (1103515245 * x + 12345) % 2147483648
        out.append(int(round(math.exp(math.log(lo) + (math.log(hi) - math.log(lo)) * x / 2147483648.0))))
    return ",".join(str(n) for n in out)


def _scan_case(name, op, lengths, C, dtype, gate="log", inputs="plain", state="fp32", initial=False, pool=0,
               packed=False):
    return {"name": name, "op": op, "lengths": lengths, "C": C, "dtype": dtype, "gate": gate, "inputs": inputs,
            "state": state, "initial": initial, "pool": pool, "packed": packed}


def _decode_case(name, N, C, dtype, gate="log", inputs="plain", state="fp32", pool=0, packed=False):
    return {"name": name, "op": "decode", "N": N, "C": C, "dtype": dtype, "gate": gate, "inputs": inputs,
            "state": state, "pool": pool, "packed": packed}


def _norm_case(name, T, C, dtype, quant="none", residual=True, packed=False):
    return {"name": name, "op": "norm", "T": T, "C": C, "dtype": dtype, "quant": quant, "residual": residual,
            "packed": packed}


def _norm_grad_case(name, T, C, dtype, stream=True, packed=False):
    return {"name": name, "op": "norm_grad", "T": T, "C": C, "dtype": dtype, "stream": stream, "packed": packed}


def listed():
    return [
        # one prompt of the benchmark's size, as many channels as its 64 heads of 128
        _scan_case("prefill_1x4096_c8192", "prefill", "4096", 8192, "bf16"),
        # one long prompt, gates as pre-activations
        _scan_case("prefill_1x65536_c4096", "prefill", "65536", 4096, "bf16", "sigmoid", "complement", initial=True),
        # many short continuations, from one token up, 16-bit states in a pool, packed projections
        _scan_case("prefill_40short_c2048_pool", "prefill", "0," + _ragged(39, 1, 90, 3), 2048, "bf16", "log", "norm",
                   "bf16", True, 56, True),
        # float32, odd lengths, channels that fill no whole group
        _scan_case("prefill_4seq_c1000_fp32", "prefill", "1,257,64,1000", 1000, "fp32", "sigmoid", "norm", initial=True),
        # a single request's decode step: latency
        _decode_case("decode_n1_c8192", 1, 8192, "bf16"),
        # the benchmark's batch of decoding sequences, states in a pool
        _decode_case("decode_n256_c8192_pool", 256, 8192, "bf16", "sigmoid", "complement", pool=300, packed=True),
        # a training step's prompt
        _scan_case("backward_1x4096_c8192", "backward", "4096", 8192, "bf16"),
        # a ragged training batch that begins from carried states
        _scan_case("backward_16seq_c4096", "backward", _ragged(16, 512, 16384, 7), 4096, "bf16", "sigmoid",
                   "complement", initial=True),
        # the norm before one token's in-projections: latency
        _norm_case("norm_1_c4096_token", 1, 4096, "bf16", "token"),
        # four prompts, one scale for every 128 channels
        _norm_case("norm_16384_c4096_group", 16384, 4096, "bf16", "group"),
        # a small odd batch in float32
        _norm_grad_case("norm_grad_37_c1000_fp32", 37, 1000, "fp32"),
        # four prompts of a training step
        _norm_grad_case("norm_grad_16384_c4096", 16384, 4096, "bf16"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["prefill", "prefill", "decode", "backward", "backward", "norm", "norm_grad"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "fp32"])
    gate, inputs = rng.choice(["log", "sigmoid"]), rng.choice(["plain", "complement", "norm"])
    state, packed = rng.choice(["fp32", "fp32", "bf16"]), rng.random() < 0.5
    C = 8 * _log_int(rng, 8, 1024)
    if op in ("prefill", "backward"):
        N = _log_int(rng, 1, 48)
        total = _log_int(rng, max(16, N), max(64, min(60000, 60000000 // C)))
        cuts = sorted(rng.randint(0, total) for _ in range(N - 1))
        lengths = [b - a for a, b in zip([0] + cuts, cuts + [total])]
        pool = rng.choice([0, N + rng.randint(0, 9)]) if op == "prefill" else 0
        c = _scan_case("", op, ",".join(str(n) for n in lengths), C, dtype, gate, inputs, state, rng.random() < 0.6,
                       pool, packed)
    elif op == "decode":
        N = _log_int(rng, 1, 400)
        c = _decode_case("", N, C, dtype, gate, inputs, state, rng.choice([0, N + rng.randint(0, 60)]), packed)
    elif op == "norm":
        quant = rng.choice(["none", "token", "group"])
        if quant == "group":
            C = 128 * _log_int(rng, 1, 64)
        c = _norm_case("", _log_int(rng, 1, min(30000, 60000000 // C)), C, dtype, quant, rng.random() < 0.7, packed)
    else:
        c = _norm_grad_case("", _log_int(rng, 1, min(30000, 60000000 // C)), C, dtype, rng.random() < 0.7, packed)
    del c["name"]
    return c


def _lengths(case):
    return [int(n) for n in case["lengths"].split(",")]


def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    C = case["C"]
    if case["op"] == "decode":
        n = case["N"] * C
        return {"bytes": 3 * n * e + 2 * n * (2 if case["state"] == "bf16" else 4), "flops": 8 * n}
    if case["op"] in ("prefill", "backward"):
        n, rows = sum(_lengths(case)) * C, len(_lengths(case)) * C
        states = rows * (2 if case["state"] == "bf16" else 4)
        if case["op"] == "prefill":
            return {"bytes": 3 * n * e + (2 if case["initial"] else 1) * states, "flops": 8 * n}
        tensors = 5 if case["inputs"] == "plain" else 6
        return {"bytes": tensors * n * e + (states + 8 * rows if case["initial"] else 0), "flops": 16 * n}
    n = case["T"] * C
    if case["op"] == "norm":
        scales = {"none": 0, "token": case["T"], "group": n // 128}[case["quant"]]
        ins = 2 * e if case["residual"] else e
        outs = (e if case["quant"] == "none" else 1) + (e if case["residual"] else 0)
        return {"bytes": (ins + outs) * n + 4 * scales + 4 * C, "flops": 8 * n}
    return {"bytes": (4 if case["stream"] else 3) * n * e + 8 * C, "flops": 14 * n}


def _rows(count, T, C, dtype, packed, gen, device):
    """Tensors of T rows of C channels: views of one packed projection, or dense."""
    if packed:
        x = torch.randn(T, count * C + 64, generator=gen, device=device).to(dtype)
        return [x[:, i * C:(i + 1) * C] for i in range(count)]
    return [torch.randn(T, C, generator=gen, device=device).to(dtype) for _ in range(count)]


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(int(seed))
    dt, C = DTYPES[case["dtype"]], case["C"]
    s = {"case": case}
    if case["op"] in ("norm", "norm_grad"):
        T = case["T"]
        s["x"], s["other"] = _rows(2, T, C, dt, case["packed"], gen, dev)
        # channels of very different sizes, as a residual stream has them
        size = torch.exp2(2.0 * torch.randn(C, generator=gen, device=dev)).to(dt)
        s["x"].mul_(size)
        s["weight"] = 1.0 + 0.1 * torch.randn(C, generator=gen, device=dev)
        if case["op"] == "norm_grad":
            s["stream"] = torch.randn(T, C, generator=gen, device=dev).to(dt) if case["stream"] else None
        elif not case["residual"]:
            s["other"] = None
        return s
    lengths = _lengths(case) if case["op"] != "decode" else [1] * case["N"]
    T, N = sum(lengths), len(lengths)
    s["x"], s["gate"] = _rows(2, T, C, dt, case["packed"], gen, dev)
    # channels that forget within a few tokens up to channels that hold hundreds
    spread = torch.rand(C, generator=gen, device=dev)
    if case["gate"] == "log":
        s["gate"].copy_(-torch.exp2(-8.0 * spread) * torch.log1p(torch.exp(s["gate"].float() + 1.0)))
    else:
        s["gate"].copy_(s["gate"].float() + 7.0 * spread - 1.0)
    rows = case.get("pool") or N
    if case["op"] == "decode" or case["initial"] or case["pool"]:
        s["state"] = torch.randn(rows, C, generator=gen, device=dev).to(DTYPES[case["state"]])
    s["slots"] = torch.randperm(rows, generator=gen, device=dev)[:N].to(torch.int32) if case.get("pool") else None
    if case["op"] == "decode":
        return s
    cu = [0]
    for n in lengths:
        cu.append(cu[-1] + n)
    s["cu_host"] = torch.tensor(cu, dtype=torch.int32)
    s["cu"] = s["cu_host"].to(dev)
    if case["op"] == "backward":
        # the forward pass keeps its output; the gradients arrive from the layers above
        first = s["state"].float() if case["initial"] else torch.zeros(N, C, device=dev)
        la, b = _factors(s["gate"].float(), case)
        s["o"] = _states(la, b * s["x"].float(), s, first).to(dt)
        s["do"] = torch.randn(T, C, generator=gen, device=dev).to(dt)
        s["dstate"] = torch.randn(N, C, generator=gen, device=dev) if case["initial"] else None
    return s


# ------------------------------------------------------------------ plain forms
def _factors(z, case):
    """(log a, b) in float32."""
    if case["gate"] == "log":
        la = z.clamp(max=0.0)
    else:  # log sigmoid: exact near 1 and far from it
        la = z.clamp(max=0.0) - torch.log1p(torch.exp(-z.abs()))
    if case["inputs"] == "complement":
        return la, -torch.expm1(la)
    if case["inputs"] == "norm":
        return la, torch.sqrt(-torch.expm1(2.0 * la))
    return la, torch.ones_like(la)


def _scan(la, x):
    """y_i = exp(la_i) y_{i-1} + x_i over the first axis: neighbours joined, half as many
    again, and the ones between from those before them."""
    M = x.shape[0]
    if M <= 1:
        return x.clone()
    le, lo, xe, xo = la[0:M - 1:2], la[1::2], x[0:M - 1:2], x[1::2]
    odd = _scan(le + lo, lo.exp() * xe + xo)
    y = torch.empty_like(x)
    y[1::2] = odd
    y[0] = x[0]
    y[2::2] = la[2::2].exp() * odd[:(M - 1) // 2] + x[2::2]
    return y


def _starts(s):
    """First tokens of the sequences that have any, their numbers, and their last tokens."""
    length = s["cu_host"][1:] - s["cu_host"][:-1]
    some = torch.nonzero(length > 0).flatten()
    dev = s["gate"].device
    return s["cu_host"][some].long().to(dev), some.to(dev), (s["cu_host"][some + 1].long() - 1).to(dev)


def _states(la, u, s, first_state):
    begin, some, _ = _starts(s)
    u[begin] += la[begin].exp() * first_state[some]
    la = la.clone()
    la[begin] = -math.inf
    return _scan(la, u)


def _plain_prefill(s):
    case = s["case"]
    N, C = s["cu_host"].shape[0] - 1, case["C"]
    dev, sdt = s["x"].device, DTYPES[case["state"]]
    rows = torch.arange(N, device=dev) if s["slots"] is None else s["slots"].long()
    first = s["state"][rows].float() if case["initial"] else torch.zeros(N, C, device=dev)
    la, b = _factors(s["gate"].float(), case)
    h = _states(la, b * s["x"].float(), s, first)
    _, some, last = _starts(s)
    first[some] = h[last]
    final = first.to(sdt)
    if s["slots"] is not None:
        s["state"][rows] = final
        final = s["state"]
    return {"o": h.to(s["x"].dtype), "state": final}


def _plain_decode(s):
    la, b = _factors(s["gate"].float(), s["case"])
    rows = slice(None) if s["slots"] is None else s["slots"].long()
    h = la.exp() * s["state"][rows].float() + b * s["x"].float()
    s["state"][rows] = h.to(s["state"].dtype)
    return {"o": h.to(s["x"].dtype), "state": s["state"]}


def _plain_backward(s):
    case = s["case"]
    N, C = s["cu_host"].shape[0] - 1, case["C"]
    dev = s["x"].device
    z, x, do = s["gate"].float(), s["x"].float(), s["do"].float()
    la, b = _factors(z, case)
    a = la.exp()
    begin, some, last = _starts(s)
    dlast = s["dstate"] if case["initial"] else torch.zeros(N, C, device=dev)
    # dh_t = do_t + a_{t+1} dh_{t+1}, the last token's from the final state's gradient
    follow = torch.cat([la[1:], la[:1]])
    follow[last] = -math.inf
    dh = _scan(follow.flip(0), do.index_add(0, last, dlast[some]).flip(0)).flip(0)
    before = torch.cat([s["o"][:1], s["o"][:-1]]).float()
    before[begin] = s["state"][some].float() if case["initial"] else torch.zeros(len(begin), C, device=dev)
    slope = a if case["gate"] == "log" else -a * torch.expm1(la)
    grad = before * slope
    if case["inputs"] == "complement":
        grad = grad - x * slope
    elif case["inputs"] == "norm":
        grad = grad - torch.where(b > 0, x * a * slope / b, 0.0)
    dgate = dh * grad
    if case["gate"] == "log":
        dgate = torch.where(z > 0, 0.0, dgate)
    out = {"dx": (dh * b).to(s["x"].dtype), "dgate": dgate.to(s["x"].dtype)}
    if case["initial"]:
        dfirst = dlast.clone()
        dfirst[some] = a[begin] * dh[begin]
        out["dstate"] = dfirst
    return out


def _plain_norm(s):
    case = s["case"]
    T, C = s["x"].shape
    t = s["x"].float()
    if s["other"] is not None:
        t = t + s["other"].float()
    y = t * torch.rsqrt(t.square().mean(-1, keepdim=True) + EPS) * s["weight"]
    out = {"s": t.to(s["x"].dtype)} if s["other"] is not None else {}
    if case["quant"] == "none":
        return dict(out, y=y.to(s["x"].dtype))
    g = y.unflatten(1, (-1, 128 if case["quant"] == "group" else C))
    top = g.abs().amax(-1, keepdim=True)
    scale = torch.where(top > 0, top / TOP, 1.0)
    q = (g / scale).clamp(-TOP, TOP).to(torch.float8_e4m3fn).reshape(T, C)
    return dict(out, y=q, scale=scale.reshape(T) if case["quant"] == "token" else scale.reshape(T, C // 128))


def _plain_norm_grad(s):
    t, dy = s["x"].float(), s["other"].float()
    r = torch.rsqrt(t.square().mean(-1, keepdim=True) + EPS)
    n = t * r
    g = dy * s["weight"]
    dx = (g - n * (g * n).mean(-1, keepdim=True)) * r
    if s["stream"] is not None:
        dx = dx + s["stream"].float()
    return {"dx": dx.to(s["x"].dtype), "dweight": (dy * n).sum(0)}


# ------------------------------------------------------------------ the package's calls
def _own(s):
    import gated_delta_rule_short_amd as kda
    case = s["case"]
    if case["op"] == "norm":
        y, scale, t = kda.kda_add_norm(s["x"], s["other"], s["weight"], eps=EPS, quant=case["quant"])
        out = {"s": t} if t is not None else {}
        return dict(out, y=y) if scale is None else dict(out, y=y, scale=scale)
    if case["op"] == "norm_grad":
        dx, dw = kda.kda_add_norm_backward(s["other"], s["x"], s["weight"], eps=EPS, dresidual=s["stream"])
        return {"dx": dx, "dweight": dw}
    kinds = {"gate_kind": case["gate"], "input_kind": case["inputs"]}
    if case["op"] == "decode":
        o = kda.kda_gated_scan_decode(s["x"], s["gate"], s["state"], state_slots=s["slots"], **kinds)
        return {"o": o, "state": s["state"]}
    given = s["state"] if case["initial"] else None
    if case["op"] == "prefill":
        out = s["state"] if case["pool"] else True
        if out is True and given is None and case["state"] == "bf16":
            out = torch.empty(s["cu_host"].shape[0] - 1, case["C"], dtype=torch.bfloat16, device=s["x"].device)
        o, state = kda.kda_gated_scan_prefill(s["x"], s["gate"], cu_seqlens=s["cu"], cu_seqlens_host=s["cu_host"],
                                              state_in=given, state_out=out, state_slots=s["slots"], **kinds)
        return {"o": o, "state": state}
    dx, dgate, dstate = kda.kda_gated_scan_backward(
        s["do"], s["gate"], s["o"], None if case["inputs"] == "plain" else s["x"], cu_seqlens=s["cu"],
        cu_seqlens_host=s["cu_host"], state_in=given, dstate_out=s["dstate"], dstate_in=True if case["initial"] else None,
        **kinds)
    out = {"dx": dx, "dgate": dgate}
    return dict(out, dstate=dstate) if case["initial"] else out


def run(state):
    if own:
        return _own(state)
    return {"prefill": _plain_prefill, "decode": _plain_decode, "backward": _plain_backward, "norm": _plain_norm,
            "norm_grad": _plain_norm_grad}[state["case"]["op"]](state)


# ------------------------------------------------------------------ 64 bits
def _exact_factors(z, case):
    a = torch.exp(torch.minimum(z, torch.zeros_like(z))) if case["gate"] == "log" else torch.sigmoid(z)
    b = {"plain": torch.ones_like(a), "complement": 1.0 - a, "norm": torch.sqrt(1.0 - a * a)}[case["inputs"]]
    return a, b


def _order(case):
    """Sequences by falling length, their first tokens, and how many are as long as t."""
    lengths = _lengths(case) if case["op"] != "decode" else [1] * case["N"]
    order = sorted(range(len(lengths)), key=lambda n: -lengths[n])
    start = [sum(lengths[:n]) for n in range(len(lengths))]
    return lengths, order, start


def _exact_scan(s):
    """One token after another, all sequences side by side."""
    case = s["case"]
    dev = s["x"].device
    lengths, order, start = _order(case)
    N = len(lengths)
    rows = torch.arange(N, device=dev) if s["slots"] is None else s["slots"].long()
    held = case["op"] == "decode" or case["initial"]
    S = s["state"][rows].double() if held else torch.zeros(N, case["C"], dtype=torch.float64, device=dev)
    S = S[torch.tensor(order, device=dev)]
    first = torch.tensor([start[n] for n in order], device=dev)
    a, b = _exact_factors(s["gate"].double(), case)
    u = b * s["x"].double()
    for t in range(max(lengths)):
        live = sum(1 for n in lengths if n > t)
        at = first[:live] + t
        S[:live] = u[at] = torch.addcmul(u[at], a[at], S[:live])
    back = torch.empty_like(S)
    back[torch.tensor(order, device=dev)] = S
    if s["slots"] is not None or case["op"] == "decode":
        full = s["state"].double()
        full[rows] = back
        back = full
    return {"o": u, "state": back}


def _exact_backward(s):
    case = s["case"]
    dev = s["x"].device
    lengths, order, start = _order(case)
    N, C = len(lengths), case["C"]
    a, b = _exact_factors(s["gate"].double(), case)
    R = torch.zeros(N, C, dtype=torch.float64, device=dev)
    if case["initial"]:
        R = s["dstate"].double()[torch.tensor(order, device=dev)]
    first = torch.tensor([start[n] for n in order], device=dev)
    dh = s["do"].double()
    for t in range(max(lengths) - 1, -1, -1):
        live = sum(1 for n in lengths if n > t)
        at = first[:live] + t
        dh[at] += R[:live]
        R[:live] = a[at] * dh[at]
    h = torch.empty_like(dh)
    h[1:] = s["o"][:-1].double()
    some = torch.tensor([n for n in range(N) if lengths[n]], device=dev)
    at = torch.tensor([start[n] for n in range(N) if lengths[n]], device=dev)
    h[at] = s["state"].double()[some] if case["initial"] else 0.0
    x, z = s["x"].double(), s["gate"].double()
    da = a if case["gate"] == "log" else a * (1.0 - a)
    if case["gate"] == "log":
        da = da * (z <= 0)
    # the input factor's slope along a: 0, -1, -a / sqrt(1 - a^2), which ends at b = 0
    db = {"plain": torch.zeros_like(a), "complement": -torch.ones_like(a),
          "norm": torch.where(b > 0, -a / torch.where(b > 0, b, 1.0), 0.0)}[case["inputs"]]
    out = {"dx": dh * b, "dgate": dh * da * (h + x * db)}
    if case["initial"]:
        back = torch.empty_like(R)
        back[torch.tensor(order, device=dev)] = R
        out["dstate"] = back
    return out


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] in ("prefill", "decode"):
        return _exact_scan(s)
    if case["op"] == "backward":
        return _exact_backward(s)
    t, w, C = s["x"].double(), s["weight"].double(), case["C"]
    if case["op"] == "norm":
        if s["other"] is not None:
            t = t + s["other"].double()
        y = w * t / torch.sqrt(t.pow(2).sum(-1, keepdim=True) / C + EPS)
        out = {"s": t} if s["other"] is not None else {}
        if case["quant"] == "none":
            return dict(out, y=y)
        width = C if case["quant"] == "token" else 128
        blocks = y.reshape(-1, width)
        scale = blocks.abs().max(dim=1).values / TOP
        scale[scale == 0] = 1.0
        shape = (case["T"],) if case["quant"] == "token" else (case["T"], C // 128)
        return dict(out, y=(blocks / scale[:, None]).reshape(y.shape), scale=scale.reshape(shape))
    dy = s["other"].double()
    rms = torch.sqrt(t.pow(2).sum(-1, keepdim=True) / C + EPS)
    g = dy * w
    dx = g / rms - t * (g * t).sum(-1, keepdim=True) / (C * rms.pow(3))
    if s["stream"] is not None:
        dx = dx + s["stream"].double()
    return {"dx": dx, "dweight": (dy * t / rms).sum(0)}
