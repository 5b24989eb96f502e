"""The operators around the recurrence of a token-mixer layer, as cases to be timed and compared.

Three operators, each for prompts and training (forward, backward) and, where a layer decodes
with it, for single tokens (step):

  conv   the short causal depthwise convolution before the recurrence
  scan   the selective state space scan, a recurrence with a decay per (channel, state)
  norm   the norms after and before a block, fused with the gate, the residual and its scale

``run`` computes them with elementary torch operations in 32 bits (``own`` false) or with the
library's calls (``own`` true); ``exact`` computes them in 64 bits, one sequence and one token
after the other, with gradients by automatic differentiation of that definition.
"""
import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def listed():
    return [
        # q, k and v of 16 heads of 128 before the delta rule, one prompt of 4,096 tokens
        {"name": "conv_prompt_bf16", "op": "conv", "dir": "fwd", "dtype": "bf16", "seqs": 1,
         "packed": False, "tokens": 4096, "channels": 6144, "width": 4, "silu": True,
         "bias": False, "state": True},
        # short ragged requests packed together, an odd channel count, earlier inputs given
        {"name": "conv_packed_f32_odd", "op": "conv", "dir": "fwd", "dtype": "f32", "seqs": 23,
         "packed": True, "tokens": 2311, "channels": 1537, "width": 3, "silu": True,
         "bias": True, "state": True},
        # a training step's gradients of the first case's layer, four sequences packed
        {"name": "conv_train_bf16", "op": "conv", "dir": "bwd", "dtype": "bf16", "seqs": 4,
         "packed": True, "tokens": 4096, "channels": 6144, "width": 4, "silu": True,
         "bias": True, "state": False, "grad": "same"},
        # one decoded token of 64 sequences, 48 value heads over 16 key heads of 128
        {"name": "conv_step_bf16", "op": "conv", "dir": "step", "dtype": "bf16", "seqs": 64,
         "tokens": 64, "channels": 10240, "width": 4, "silu": True, "bias": False},
        # a prompt of 4,096 tokens through a layer of hidden size 2,048 expanded twice
        {"name": "scan_prompt_bf16", "op": "scan", "dir": "fwd", "dtype": "bf16", "seqs": 1,
         "packed": False, "tokens": 4096, "channels": 4096, "states": 16, "groups": 1,
         "gate": True, "state": False},
        # a short prompt of a small layer in fp32: latency
        {"name": "scan_prompt_f32_short", "op": "scan", "dir": "fwd", "dtype": "f32", "seqs": 1,
         "packed": False, "tokens": 197, "channels": 768, "states": 16, "groups": 1,
         "gate": False, "state": False},
        # a serving batch: prompts of different lengths packed, continuing given states
        {"name": "scan_packed_bf16", "op": "scan", "dir": "fwd", "dtype": "bf16", "seqs": 16,
         "packed": True, "tokens": 16384, "channels": 2048, "states": 16, "groups": 1,
         "gate": True, "state": True},
        # a training step's gradients, eight sequences of 512 tokens
        {"name": "scan_train_bf16", "op": "scan", "dir": "bwd", "dtype": "bf16", "seqs": 8,
         "packed": False, "tokens": 4096, "channels": 2048, "states": 16, "groups": 1,
         "gate": True, "state": False, "grad": "same"},
        # gradients in fp32 at odd sizes: two groups of B and C, 24 states, ragged sequences
        {"name": "scan_train_f32_odd", "op": "scan", "dir": "bwd", "dtype": "f32", "seqs": 5,
         "packed": True, "tokens": 1011, "channels": 1002, "states": 24, "groups": 2,
         "gate": True, "state": True, "grad": "f32"},
        # one decoded token of 64 sequences against the pool of fp32 states
        {"name": "scan_step_f32state", "op": "scan", "dir": "step", "dtype": "bf16", "seqs": 64,
         "tokens": 64, "channels": 4096, "states": 16, "groups": 1, "gate": True},
        # the whole block boundary of hidden size 2,048: post-norm, scale, residual, next norm
        {"name": "norm_block_bf16", "op": "norm", "dir": "fwd", "dtype": "bf16", "tokens": 8192,
         "channels": 2048, "weight": True, "gate": False, "residual": "same", "scale": True,
         "next": True},
        # its gradients in a training step, with the residual stream in fp32
        {"name": "norm_train_bf16", "op": "norm", "dir": "bwd", "dtype": "bf16", "tokens": 4096,
         "channels": 2048, "weight": True, "gate": True, "residual": "f32", "scale": True,
         "next": True, "grad": "same"},
    ]


def _spread(rng, lo, hi):
    """A whole number of [lo, hi], even over the logarithm."""
    return max(lo, min(hi, round(lo * (hi / lo) ** rng.random())))


def draw(rng):
    op = rng.choice(("conv", "scan", "norm"))
    case = {"op": op, "dtype": rng.choice(("bf16", "bf16", "f32"))}
    if op == "norm":
        case["dir"] = rng.choice(("fwd", "bwd"))
        case["channels"] = _spread(rng, 16, 8192)
        case["tokens"] = _spread(rng, 1, min(65536, 8192 * 2048 // case["channels"]))
        case["weight"] = rng.random() < 0.7
        case["gate"] = rng.random() < 0.5
        residual = ("", "same", "f32") if case["dtype"] == "bf16" else ("", "same")
        case["residual"] = rng.choice(residual)
        case["scale"] = rng.random() < 0.5
        case["next"] = rng.random() < 0.5
        if not (case["gate"] or case["residual"] or case["scale"] or case["next"]):
            case["weight"] = True
    elif op == "conv":
        case["dir"] = rng.choice(("fwd", "bwd", "step"))
        case["channels"] = _spread(rng, 16, 16384)
        case["width"] = rng.choice((2, 3, 4))
        case["silu"] = rng.random() < 0.7
        case["bias"] = rng.random() < 0.5
        most = 256 if case["dir"] == "step" else 16384
        case["tokens"] = _spread(rng, 1, min(most, 4096 * 6144 // case["channels"]))
        if case["dir"] == "step":
            case["seqs"] = case["tokens"]
        else:
            case["state"] = rng.random() < 0.5
            _layout(rng, case)
    else:
        case["dir"] = rng.choice(("fwd", "bwd", "step"))
        case["states"] = rng.choice((8, 16, 16, 16, rng.randint(1, 64)))
        case["groups"] = rng.choice((1, 1, 2, 4))
        case["channels"] = _spread(rng, 8, 1024) * 4
        per = case["channels"] * case["states"]
        case["gate"] = rng.random() < 0.7
        if case["dir"] == "step":
            case["tokens"] = case["seqs"] = _spread(rng, 1, max(1, min(256, 64 * 65536 // per)))
        else:
            full = (4096 if case["dir"] == "fwd" else 1024) * 65536
            case["tokens"] = _spread(rng, 1, max(1, min(16384, full // per)))
            case["state"] = rng.random() < 0.5
            _layout(rng, case)
    if case["dir"] == "bwd":
        case["grad"] = rng.choice(("same", "f32"))
    return case


def _layout(rng, case):
    """Packed sequences of drawn lengths, or a dense batch of equal ones."""
    case["packed"] = rng.random() < 0.6
    case["seqs"] = _spread(rng, 1, min(64, case["tokens"]))
    if not case["packed"]:
        case["tokens"] -= case["tokens"] % case["seqs"]


# ---- inputs ------------------------------------------------------------------------------


class _Draw:
    def __init__(self, seed):
        self.gen = torch.Generator(device="cuda")
        self.gen.manual_seed(seed)

    def normal(self, *shape, dtype=torch.float32, std=1.0):
        x = torch.randn(*shape, generator=self.gen, device="cuda", dtype=torch.float32)
        return (x * std).to(dtype)

    def uniform(self, lo, hi, *shape):
        x = torch.rand(*shape, generator=self.gen, device="cuda", dtype=torch.float32)
        return lo + (hi - lo) * x

    def cuts(self, seqs, tokens):
        """Offsets of `seqs` sequences of uneven lengths over `tokens` tokens, empty ones among
        them by chance."""
        inner = torch.randint(0, tokens + 1, (seqs - 1,), generator=self.gen, device="cuda")
        ends = torch.tensor([0, tokens], device="cuda")
        return torch.cat((inner, ends)).sort().values.to(torch.int32)

    def slots(self, seqs):
        """Distinct slots of a pool that is a little larger than the batch."""
        order = torch.randperm(seqs + 2, generator=self.gen, device="cuda")
        return order[:seqs].to(torch.int32)


def prepare(case, seed):
    d = _Draw(seed)
    dt = DTYPES[case["dtype"]]
    s = {"case": case, "cu": None}
    T, C = case["tokens"], case["channels"]
    if case["op"] == "norm":
        _prepare_norm(case, d, dt, s, T, C)
        return s
    N = case["seqs"]
    if case["dir"] == "step":
        s["lead"], s["idx"] = (N, 1), d.slots(N)
    elif case["packed"]:
        s["lead"], s["cu"] = (1, T), d.cuts(N, T)
    else:
        s["lead"] = (N, T // N)
    if case["op"] == "conv":
        _prepare_conv(case, d, dt, s, N, C)
    else:
        _prepare_scan(case, d, dt, s, N, C)
    return s


def _grad_type(case, dt):
    return torch.float32 if case.get("grad") == "f32" else dt


def _prepare_conv(case, d, dt, s, N, C):
    W = case["width"]
    # the convolved channels are a column slice of the input projection's output
    s["x"] = d.normal(*s["lead"], C + C // 2, dtype=dt)[..., :C]
    s["weight"] = d.normal(C, W, std=W ** -0.5)
    s["bias"] = d.normal(C, std=0.1) if case["bias"] else None
    if case["dir"] == "step":
        s["pool"] = d.normal(N + 2, W - 1, C)
        return
    s["state0"] = d.normal(N, W - 1, C) if case["state"] else None
    if case["dir"] == "bwd":
        s["dy"] = d.normal(*s["lead"], C, dtype=_grad_type(case, dt))
        s["dstate_T"] = d.normal(N, W - 1, C) if case["state"] else None


def _prepare_scan(case, d, dt, s, N, C):
    M, G = case["states"], case["groups"]
    lead = s["lead"]
    s["x"] = d.normal(*lead, C, dtype=dt)
    s["gate"] = d.normal(*lead, 2 * C, dtype=dt)[..., C:] if case["gate"] else None
    # B and C are slices of the projection that also gives the low-rank step
    R = max(1, C // 16)
    proj = d.normal(*lead, R + 2 * G * M, dtype=dt)
    s["B"] = proj[..., R:R + G * M].unflatten(-1, (G, M))
    s["C"] = proj[..., R + G * M:].unflatten(-1, (G, M))
    s["dt"] = d.normal(*lead, C, dtype=dt, std=0.5)
    # steps of 0.001 to 0.1 at the bias, decay rates of 1 to the number of states
    step = torch.exp(d.uniform(-6.9, -2.3, C))
    s["dt_bias"] = torch.log(torch.expm1(step))
    s["A"] = -torch.arange(1, M + 1, device="cuda") * torch.exp(d.normal(C, M, std=0.1))
    s["D"] = 1.0 + d.normal(C, std=0.1)
    if case["dir"] == "step":
        s["pool"] = d.normal(N + 2, C, M, std=0.3)
        return
    s["S0"] = d.normal(N, C, M, std=0.3) if case["state"] else None
    if case["dir"] == "bwd":
        s["dO"] = d.normal(*lead, C, dtype=_grad_type(case, dt))
        s["dS_T"] = d.normal(N, C, M, std=0.3) if case["state"] else None


def _prepare_norm(case, d, dt, s, T, C):
    rt = torch.float32 if case["residual"] == "f32" else dt
    s["x"] = d.normal(T, C, dtype=dt)
    s["gate"] = d.normal(T, 2 * C, dtype=dt)[:, C:] if case["gate"] else None
    s["residual"] = d.normal(T, C, dtype=rt, std=2.0) if case["residual"] else None
    s["norm_weight"] = 1.0 + d.normal(C, std=0.1) if case["weight"] else None
    s["scale"] = d.uniform(0.1, 1.0, C) if case["scale"] else None
    s["next_weight"] = 1.0 + d.normal(C, std=0.1) if case["next"] else None
    if case["dir"] == "bwd":
        g = _grad_type(case, dt)
        s["dh"] = d.normal(T, C, dtype=torch.float32 if case["residual"] == "f32" else g)
        s["dy"] = d.normal(T, C, dtype=g) if case["next"] else None


# ---- one pass ----------------------------------------------------------------------------


def run(state):
    case = state["case"]
    if own:
        return _OWN[case["op"], case["dir"]](state, case)
    return _PLAIN[case["op"], case["dir"]](state, case)


def _own_conv_fwd(s, case):
    import gated_delta_rule_gdn_amd as g
    y, state_T = g.short_conv_fwd(s["x"], s["weight"], bias=s["bias"], state0=s["state0"],
                                  cu_seqlens=s["cu"], silu=case["silu"])
    return {"y": y, "state_T": state_T}


def _own_conv_bwd(s, case):
    import gated_delta_rule_gdn_amd as g
    return g.short_conv_bwd(s["x"], s["weight"], s["dy"], bias=s["bias"], state0=s["state0"],
                            cu_seqlens=s["cu"], silu=case["silu"], dstate_T=s["dstate_T"])


def _own_conv_step(s, case):
    import gated_delta_rule_gdn_amd as g
    y = g.short_conv_step(s["x"], s["weight"], s["pool"], bias=s["bias"], state_idx=s["idx"],
                          silu=case["silu"])
    return {"y": y, "pool": s["pool"]}


def _own_scan_fwd(s, case):
    import gated_delta_rule_gdn_amd as g
    o, S_T = g.selective_scan_fwd(s["x"], s["dt"], s["A"], s["B"], s["C"], D=s["D"],
                                  gate=s["gate"], dt_bias=s["dt_bias"], dt_softplus=True,
                                  S0=s["S0"], cu_seqlens=s["cu"])
    return {"o": o, "S_T": S_T}


def _own_scan_bwd(s, case):
    import gated_delta_rule_gdn_amd as g
    return g.selective_scan_bwd(s["x"], s["dt"], s["A"], s["B"], s["C"], s["dO"], D=s["D"],
                                gate=s["gate"], dt_bias=s["dt_bias"], dt_softplus=True,
                                S0=s["S0"], cu_seqlens=s["cu"], dS_T=s["dS_T"])


def _own_scan_step(s, case):
    import gated_delta_rule_gdn_amd as g
    o = g.selective_scan_step(s["x"], s["dt"], s["A"], s["B"], s["C"], s["pool"], D=s["D"],
                              gate=s["gate"], dt_bias=s["dt_bias"], dt_softplus=True,
                              state_idx=s["idx"])
    return {"o": o, "pool": s["pool"]}


def _own_norm_fwd(s, case):
    import gated_delta_rule_gdn_amd as g
    h, y = g.block_norm_fwd(s["x"], norm_weight=s["norm_weight"], gate=s["gate"],
                            residual=s["residual"], scale=s["scale"],
                            next_weight=s["next_weight"])
    return {"h": h} if y is None else {"h": h, "y": y}


def _own_norm_bwd(s, case):
    import gated_delta_rule_gdn_amd as g
    return g.block_norm_bwd(s["x"], dh=s["dh"], dy=s["dy"], norm_weight=s["norm_weight"],
                            gate=s["gate"], residual=s["residual"], scale=s["scale"],
                            next_weight=s["next_weight"])


def _where_tokens(s):
    """Of every token: its sequence, and that sequence's first token and end. Of every
    sequence: its first token and end."""
    B, T = s["lead"]
    t = torch.arange(B * T, device="cuda")
    cu = s["cu"] if s["cu"] is not None else torch.arange(B + 1, device="cuda") * T
    cu = cu.long()
    seq = (t[:, None] >= cu[None, 1:]).sum(1)
    return t, seq, cu[seq], cu[seq + 1], cu[:-1], cu[1:]


def _flat(x):
    return x.flatten(0, 1).float()


def _window(x, state0, at, first, seq, W):
    """Row `at` of each sequence's inputs, rows before its first token from state0 or zero."""
    inside = x[at.clamp(0, x.shape[0] - 1)]
    if state0 is None:
        before = torch.zeros_like(inside)
    else:
        before = state0[seq, (at - first + W - 1).clamp(0, W - 2)]
    return torch.where((at >= first)[:, None], inside, before)


def _plain_conv_sum(s, case):
    W = case["width"]
    x = _flat(s["x"])
    t, seq, first, end, _, _ = _where_tokens(s)
    rows = [_window(x, s["state0"], t - (W - 1) + j, first, seq, W) for j in range(W)]
    a = sum(s["weight"][:, j] * rows[j] for j in range(W))
    return (a if s["bias"] is None else a + s["bias"]), rows


def _silu(a):
    return a / (1.0 + torch.exp(-a))


def _silu_slope(a):
    p = 1.0 / (1.0 + torch.exp(-a))
    return p * (1.0 + a * (1.0 - p))


def _plain_conv_fwd(s, case):
    W = case["width"]
    a, _ = _plain_conv_sum(s, case)
    y = _silu(a) if case["silu"] else a
    x = _flat(s["x"])
    _, _, _, _, begins, ends = _where_tokens(s)
    which = torch.arange(case["seqs"], device="cuda")
    last = [_window(x, s["state0"], ends - (W - 1) + r, begins, which, W) for r in range(W - 1)]
    return {"y": y.to(s["x"].dtype).unflatten(0, s["lead"]), "state_T": torch.stack(last, 1)}


def _plain_conv_bwd(s, case):
    W, N = case["width"], case["seqs"]
    a, rows = _plain_conv_sum(s, case)
    e = _flat(s["dy"])
    if case["silu"]:
        e = e * _silu_slope(a)
    t, seq, first, end, begins, ends = _where_tokens(s)
    T = t.shape[0]

    def reached(at, below):
        return torch.where((at < below)[:, None], e[at.clamp(max=T - 1)], 0.0)

    dx = sum(s["weight"][:, j] * reached(t + W - 1 - j, end) for j in range(W))
    out = {"dweight": torch.stack([(e * rows[j]).sum(0) for j in range(W)], 1)}
    if s["dstate_T"] is not None:
        tail = t - (end - (W - 1))
        dx = dx + torch.where((tail >= 0)[:, None], s["dstate_T"][seq, tail.clamp(min=0)], 0.0)
    if s["bias"] is not None:
        out["dbias"] = e.sum(0)
    if s["state0"] is not None:
        d0 = []
        for r in range(W - 1):
            g = sum(s["weight"][:, r - p] * reached(begins + p, ends) for p in range(r + 1))
            back = r - (ends - begins)
            given = s["dstate_T"][torch.arange(N, device="cuda"), back.clamp(min=0)]
            d0.append(g + torch.where((back >= 0)[:, None], given, 0.0))
        out["dstate0"] = torch.stack(d0, 1)
    out["dx"] = dx.to(s["dy"].dtype).unflatten(0, s["lead"])
    return out


def _plain_conv_step(s, case):
    W = case["width"]
    at = s["idx"].long()
    rows = torch.cat((s["pool"][at], s["x"].float()), 1)
    a = (rows * s["weight"].t()).sum(1)
    if s["bias"] is not None:
        a = a + s["bias"]
    y = _silu(a) if case["silu"] else a
    s["pool"][at] = rows[:, 1:]
    return {"y": y.to(s["x"].dtype)[:, None], "pool": s["pool"]}


def _expand(v, C):
    """[T, G, M] of groups as [T, C, M] of channels."""
    T, G, M = v.shape
    return v[:, :, None].expand(T, G, C // G, M).reshape(T, C, M)


def _softplus(x):
    return torch.clamp(x, min=0.0) + torch.log1p(torch.exp(-x.abs()))


def _scan_terms(s):
    C = s["x"].shape[-1]
    x, B, Cm = _flat(s["x"]), _expand(_flat(s["B"]), C), _expand(_flat(s["C"]), C)
    raw = _flat(s["dt"]) + s["dt_bias"]
    dt = _softplus(raw)
    a = torch.exp(dt[..., None] * s["A"])
    return x, B, Cm, raw, dt, a, (dt * x)[..., None] * B


def _linear(a, b):
    """h_t = a_t h_{t-1} + b_t over the first axis, by doubling the reach of every row."""
    reach = 1
    while reach < a.shape[0]:
        b = torch.cat((b[:reach], b[reach:] + a[reach:] * b[:-reach]))
        a = torch.cat((a[:reach], a[reach:] * a[:-reach]))
        reach *= 2
    return b


def _scan_states(s, a, b):
    """All states h_t, and the states entering the tokens' updates times their decay."""
    t, seq, first, end, begins, ends = _where_tokens(s)
    start = (t == first)[:, None, None]
    keep = torch.where(start, 0.0, a)
    if s["S0"] is not None:
        b0 = torch.where(start, b + a * s["S0"][seq], b)
    else:
        b0 = b
    return _linear(keep, b0), keep


def _plain_scan_fwd(s, case):
    x, B, Cm, raw, dt, a, b = _scan_terms(s)
    h, _ = _scan_states(s, a, b)
    y = (h * Cm).sum(-1) + s["D"] * x
    if s["gate"] is not None:
        y = y * _silu(_flat(s["gate"]))
    _, _, _, _, begins, ends = _where_tokens(s)
    S = h[(ends - 1).clamp(min=0)]
    old = torch.zeros_like(S) if s["S0"] is None else s["S0"]
    S_T = torch.where((ends > begins)[:, None, None], S, old)
    return {"o": y.to(s["x"].dtype).unflatten(0, s["lead"]), "S_T": S_T}


def _by_group(v, G):
    """Sums [T, C, M] over the channels of each group."""
    T, C, M = v.shape
    return v.view(T, G, C // G, M).sum(2)


def _plain_scan_bwd(s, case):
    G = case["groups"]
    x, B, Cm, raw, dt, a, b = _scan_terms(s)
    h, keep = _scan_states(s, a, b)
    t, seq, first, end, begins, ends = _where_tokens(s)
    y = (h * Cm).sum(-1) + s["D"] * x
    dy = _flat(s["dO"])
    out = {}
    lead, gt = s["lead"], s["dO"].dtype
    if s["gate"] is not None:
        gate = _flat(s["gate"])
        out["dgate"] = (dy * y * _silu_slope(gate)).to(gt).unflatten(0, lead)
        dy = dy * _silu(gate)
    c = Cm * dy[..., None]
    if s["dS_T"] is not None:
        c = c + torch.where((t == end - 1)[:, None, None], s["dS_T"][seq], 0.0)
    after = torch.cat((keep[1:], torch.zeros_like(keep[:1])))
    gh = _linear(after.flip(0), c.flip(0)).flip(0)
    entering = h - b
    u = gh * entering
    gB = (gh * B).sum(-1)
    ddt = (x * gB + (u * s["A"]).sum(-1)) / (1.0 + torch.exp(-raw))
    out["dx"] = (s["D"] * dy + dt * gB).to(gt).unflatten(0, lead)
    out["ddt"] = ddt.to(gt).unflatten(0, lead)
    out["dB"] = _by_group(gh * (dt * x)[..., None], G).to(gt).unflatten(0, lead)
    out["dC"] = _by_group(h * dy[..., None], G).to(gt).unflatten(0, lead)
    out["dA"] = (u * dt[..., None]).sum(0)
    out["dD"] = (dy * x).sum(0)
    out["ddt_bias"] = ddt.sum(0)
    if s["S0"] is not None:
        at = begins.clamp(max=t.shape[0] - 1)
        out["dS0"] = torch.where((ends > begins)[:, None, None], (a * gh)[at], s["dS_T"])
    return out


def _plain_scan_step(s, case):
    x, B, Cm, raw, dt, a, b = _scan_terms(s)
    at = s["idx"].long()
    h = a * s["pool"][at] + b
    y = (h * Cm).sum(-1) + s["D"] * x
    if s["gate"] is not None:
        y = y * _silu(_flat(s["gate"]))
    s["pool"][at] = h
    return {"o": y.to(s["x"].dtype)[:, None], "pool": s["pool"]}


EPS = 1e-5


def _norm_terms(s):
    x = s["x"].float()
    r = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
    p = x if s["norm_weight"] is None else x * r * s["norm_weight"]
    u = p if s["gate"] is None else p * _silu(s["gate"].float())
    h = u if s["scale"] is None else s["scale"] * u
    if s["residual"] is not None:
        h = s["residual"].float() + h
    q = torch.rsqrt((h * h).mean(-1, keepdim=True) + EPS)
    return x, r, p, u, h, q


def _plain_norm_fwd(s, case):
    x, r, p, u, h, q = _norm_terms(s)
    ht = s["x"].dtype if s["residual"] is None else s["residual"].dtype
    out = {"h": h.to(ht)}
    if s["next_weight"] is not None:
        out["y"] = (h * q * s["next_weight"]).to(s["x"].dtype)
    return out


def _plain_norm_bwd(s, case):
    x, r, p, u, h, q = _norm_terms(s)
    g = s["dh"].float()
    gt = _grad_type(case, s["x"].dtype)
    out = {}
    if s["next_weight"] is not None:
        dy = s["dy"].float()
        out["dnext_weight"] = (dy * h * q).sum(0)
        w = dy * s["next_weight"]
        g = g + q * w - h * q ** 3 * (w * h).mean(-1, keepdim=True)
    if s["residual"] is not None:
        out["dresidual"] = g.to(s["dh"].dtype)
    if s["scale"] is not None:
        out["dscale"] = (g * u).sum(0)
        g = g * s["scale"]
    if s["gate"] is not None:
        gate = s["gate"].float()
        out["dgate"] = (g * p * _silu_slope(gate)).to(gt)
        g = g * _silu(gate)
    if s["norm_weight"] is not None:
        out["dnorm_weight"] = (g * x * r).sum(0)
        w = g * s["norm_weight"]
        g = r * w - x * r ** 3 * (w * x).mean(-1, keepdim=True)
    out["dx"] = g.to(gt)
    return out


_PLAIN = {("conv", "fwd"): _plain_conv_fwd, ("conv", "bwd"): _plain_conv_bwd,
          ("conv", "step"): _plain_conv_step, ("scan", "fwd"): _plain_scan_fwd,
          ("scan", "bwd"): _plain_scan_bwd, ("scan", "step"): _plain_scan_step,
          ("norm", "fwd"): _plain_norm_fwd, ("norm", "bwd"): _plain_norm_bwd}
_OWN = {("conv", "fwd"): _own_conv_fwd, ("conv", "bwd"): _own_conv_bwd,
        ("conv", "step"): _own_conv_step, ("scan", "fwd"): _own_scan_fwd,
        ("scan", "bwd"): _own_scan_bwd, ("scan", "step"): _own_scan_step,
        ("norm", "fwd"): _own_norm_fwd, ("norm", "bwd"): _own_norm_bwd}


# ---- what a pass cannot do without -------------------------------------------------------


def work(case):
    size = 4 if case["dtype"] == "f32" else 2
    grad = 4 if case.get("grad") == "f32" else size
    T, C = case["tokens"], case["channels"]
    cells = T * C
    if case["op"] == "conv":
        W, N = case["width"], case["seqs"]
        params = 4 * C * (W + case["bias"])
        if case["dir"] == "step":
            return {"bytes": 2 * cells * size + params + 2 * N * (W - 1) * C * 4,
                    "flops": 2 * W * cells}
        states = 4 * N * (W - 1) * C
        if case["dir"] == "fwd":
            return {"bytes": 2 * cells * size + params + states * (1 + case["state"]),
                    "flops": 2 * W * cells}
        return {"bytes": cells * (size + 2 * grad) + 2 * params + 3 * states * case["state"],
                "flops": 6 * W * cells}
    if case["op"] == "scan":
        M, G, N = case["states"], case["groups"], case["seqs"]
        gate = int(case["gate"])
        params = 4 * C * (M + 2)
        if case["dir"] == "step":
            return {"bytes": cells * (3 + gate) * size + 2 * T * G * M * size + params
                    + 8 * N * C * M, "flops": 7 * cells * M}
        states = 4 * N * C * M
        if case["dir"] == "fwd":
            return {"bytes": cells * (3 + gate) * size + 2 * T * G * M * size + params
                    + states * (1 + case["state"]), "flops": 7 * cells * M}
        return {"bytes": cells * ((2 + gate) * size + (3 + gate) * grad)
                + 2 * T * G * M * (size + grad) + 2 * params + 3 * states * case["state"],
                "flops": 20 * cells * M}
    res = {"": 0, "same": size, "f32": 4}[case["residual"]]
    inputs = cells * (size * (1 + case["gate"]) + res)
    params = 4 * C * (case["weight"] + case["scale"] + case["next"])
    if case["dir"] == "fwd":
        return {"bytes": inputs + cells * ((res or size) + size * case["next"]) + params,
                "flops": 16 * cells}
    gres = 4 if case["residual"] == "f32" else grad
    grads = grad * (1 + case["gate"] + case["next"]) + gres * (1 + (res > 0))
    return {"bytes": inputs + cells * grads + 2 * params, "flops": 40 * cells}


# ---- the definitions in 64 bits ----------------------------------------------------------


def _double(s, names):
    """The named inputs in 64 bits, as leaves where gradients are wanted."""
    return {n: None if s[n] is None else s[n].double().clone() for n in names}


def _offsets(s):
    B, T = s["lead"]
    return [n * T for n in range(B + 1)] if s["cu"] is None else s["cu"].tolist()


def _leaf(v):
    for x in v.values():
        if x is not None:
            x.requires_grad_(True)


def _exact_conv(s, case):
    W, C = case["width"], case["channels"]
    v = _double(s, ("x", "weight", "bias", "state0"))
    train = case["dir"] == "bwd"
    if train:
        _leaf(v)
    x = v["x"].flatten(0, 1)
    ys, lasts = [], []
    cu = _offsets(s)
    for n in range(case["seqs"]):
        length = cu[n + 1] - cu[n]
        zero = torch.zeros(W - 1, C, device="cuda", dtype=torch.float64)
        seen = torch.cat((zero if v["state0"] is None else v["state0"][n], x[cu[n]:cu[n + 1]]))
        a = torch.zeros(length, C, device="cuda", dtype=torch.float64)
        for j in range(W):
            a = a + seen[j:j + length] * v["weight"][:, j]
        if v["bias"] is not None:
            a = a + v["bias"]
        ys.append(a * torch.sigmoid(a) if case["silu"] else a)
        lasts.append(seen[length:])
    y, last = torch.cat(ys), torch.stack(lasts)
    if not train:
        return {"y": y.unflatten(0, s["lead"]), "state_T": last}
    loss = (y * s["dy"].double().flatten(0, 1)).sum()
    if s["dstate_T"] is not None:
        loss = loss + (last * s["dstate_T"].double()).sum()
    loss.backward()
    return {"d" + n: t.grad for n, t in v.items() if t is not None}


def _exact_conv_step(s, case):
    v = _double(s, ("x", "weight", "bias", "pool"))
    ys = []
    for n, slot in enumerate(s["idx"].tolist()):
        seen = torch.cat((v["pool"][slot], v["x"][n]))
        a = torch.einsum("jc,cj->c", seen, v["weight"])
        if v["bias"] is not None:
            a = a + v["bias"]
        ys.append(a * torch.sigmoid(a) if case["silu"] else a)
        v["pool"][slot] = seen[1:]
    return {"y": torch.stack(ys)[:, None], "pool": v["pool"]}


_SCAN = ("x", "dt", "A", "B", "C", "D", "gate", "dt_bias")


def _exact_tokens(v, rep, h, lo, hi):
    """The outputs of tokens lo .. hi-1 of the flat arrays, one after the other."""
    out = []
    if hi > lo:
        dt = torch.nn.functional.softplus(v["dt"][lo:hi] + v["dt_bias"])
        decay = torch.exp(dt[..., None] * v["A"]).unbind(0)
        B = v["B"][lo:hi].repeat_interleave(rep, 1)
        put = ((dt * v["x"][lo:hi])[..., None] * B).unbind(0)
        hs = []
        for a, b in zip(decay, put):
            h = a * h + b
            hs.append(h)
        C = v["C"][lo:hi].repeat_interleave(rep, 1)
        y = (torch.stack(hs) * C).sum(-1) + v["D"] * v["x"][lo:hi]
        if v["gate"] is not None:
            y = y * v["gate"][lo:hi] * torch.sigmoid(v["gate"][lo:hi])
        out.append(y)
    return out, h


def _exact_scan(s, case):
    train, N = case["dir"] == "bwd", case["seqs"]
    rep = case["channels"] // case["groups"]
    v = _double(s, _SCAN + ("S0",))
    if train:
        _leaf(v)
    flat = {n: x.flatten(0, 1) if x is not None and n in ("x", "dt", "B", "C", "gate") else x
            for n, x in v.items()}
    cu = _offsets(s)
    ys, ends = [], []
    for n in range(N):
        h = torch.zeros_like(v["A"]) if v["S0"] is None else v["S0"][n]
        y, h = _exact_tokens(flat, rep, h, cu[n], cu[n + 1])
        ys += y
        ends.append(h)
    y, S_T = torch.cat(ys), torch.stack(ends)
    if not train:
        return {"o": y.unflatten(0, s["lead"]), "S_T": S_T}
    loss = (y * s["dO"].double().flatten(0, 1)).sum()
    if s["dS_T"] is not None:
        loss = loss + (S_T * s["dS_T"].double()).sum()
    loss.backward()
    return {"d" + n: t.grad for n, t in v.items() if t is not None}


def _exact_scan_step(s, case):
    v = _double(s, _SCAN + ("pool",))
    rep = case["channels"] // case["groups"]
    flat = {n: x.flatten(0, 1) if x is not None and n in ("x", "dt", "B", "C", "gate") else x
            for n, x in v.items()}
    os_ = []
    for n, slot in enumerate(s["idx"].tolist()):
        o, h = _exact_tokens(flat, rep, v["pool"][slot], n, n + 1)
        v["pool"][slot] = h
        os_ += o
    return {"o": torch.stack(os_), "pool": v["pool"]}


def _exact_norm(s, case):
    v = _double(s, ("x", "gate", "residual", "norm_weight", "scale", "next_weight"))
    train = case["dir"] == "bwd"
    if train:
        _leaf(v)

    def rms(t, w):
        return t / (t.square().mean(-1, keepdim=True) + EPS).sqrt() * w

    h = v["x"] if v["norm_weight"] is None else rms(v["x"], v["norm_weight"])
    if v["gate"] is not None:
        h = h * v["gate"] * torch.sigmoid(v["gate"])
    if v["scale"] is not None:
        h = h * v["scale"]
    if v["residual"] is not None:
        h = h + v["residual"]
    y = None if v["next_weight"] is None else rms(h, v["next_weight"])
    if not train:
        return {"h": h} if y is None else {"h": h, "y": y}
    loss = (h * s["dh"].double()).sum()
    if y is not None:
        loss = loss + (y * s["dy"].double()).sum()
    loss.backward()
    return {"d" + n: t.grad for n, t in v.items() if t is not None}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm":
        out = _exact_norm(s, case)
    elif case["dir"] == "step":
        out = (_exact_conv_step if case["op"] == "conv" else _exact_scan_step)(s, case)
    else:
        out = (_exact_conv if case["op"] == "conv" else _exact_scan)(s, case)
    order = {"conv": ("y", "state_T", "dweight", "dbias", "dstate0", "dx", "pool"),
             "scan": ("o", "S_T", "dgate", "dx", "ddt", "dB", "dC", "dA", "dD", "ddt_bias", "dS0", "pool"),
             "norm": ("h", "y", "dnext_weight", "dresidual", "dscale", "dgate", "dnorm_weight", "dx")}
    return {n: out[n].detach() for n in order[case["op"]] if n in out}
