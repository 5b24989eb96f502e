"""The attention layer of a hybrid stack beside the recurrent ones, as cases to be timed and
compared.

Three operators:

  rotary  norms of queries and keys per head with the rotation by position: prompts (fwd), their
          gradients (bwd), and the serving form that puts keys and values into the pages of a
          cache (append)
  attn    attention of the newest tokens of every sequence over that paged cache
  copy    slots of many pools copied at once: pages of a cache, states of recurrent layers

``run`` computes them with elementary torch operations in 32 bits (``own`` false) or with the
library's calls (``own`` true); ``exact`` computes them in 64 bits from the definitions, the
gradients by automatic differentiation, the attention one sequence and one head after the other.
"""
import math
import random

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
EPS = 1e-5


def listed():
    return [
        # queries and keys of one prompt of 4,096 tokens, 16 heads over 4, slices of a projection
        {"name": "rotary_prompt_bf16", "op": "rotary", "dir": "fwd", "dtype": "bf16",
         "tokens": 4096, "hq": 16, "hk": 4, "d": 128, "rot": 128, "interleaved": False,
         "qnorm": True, "knorm": True},
        # a training step's gradients, sequences packed, as many key heads as query heads
        {"name": "rotary_train_bf16", "op": "rotary", "dir": "bwd", "dtype": "bf16",
         "tokens": 8192, "hq": 16, "hk": 16, "d": 128, "rot": 128, "interleaved": False,
         "qnorm": True, "knorm": True, "grad": "same"},
        # gradients in fp32 of a small model with an odd head size, a quarter of it rotated in
        # neighbouring pairs
        {"name": "rotary_train_f32_odd", "op": "rotary", "dir": "bwd", "dtype": "f32",
         "tokens": 1011, "hq": 6, "hk": 2, "d": 80, "rot": 20, "interleaved": True,
         "qnorm": True, "knorm": True, "grad": "same"},
        # one decoded token of 64 sequences into pages of 16 tokens: latency
        {"name": "append_step_bf16", "op": "rotary", "dir": "append", "dtype": "bf16",
         "tokens": 64, "hq": 16, "hk": 2, "d": 256, "rot": 64, "interleaved": False,
         "qnorm": True, "knorm": True, "page": 16},
        # prompts of a serving batch packed, an odd total, into pages of 64 tokens
        {"name": "append_prompt_bf16", "op": "rotary", "dir": "append", "dtype": "bf16",
         "tokens": 6007, "hq": 32, "hk": 8, "d": 128, "rot": 128, "interleaved": False,
         "qnorm": True, "knorm": False, "page": 64},
        # one request with a context of 131,072 tokens
        {"name": "attn_long_bf16", "op": "attn", "dtype": "bf16", "seqs": 1, "new": 1,
         "total": 131072, "hk": 8, "group": 4, "d": 128, "page": 64, "window": 0,
         "pattern": 1, "lse": False},
        # a serving batch of 64 requests of very different lengths
        {"name": "attn_batch_bf16", "op": "attn", "dtype": "bf16", "seqs": 64, "new": 1,
         "total": 262144, "hk": 4, "group": 4, "d": 128, "page": 16, "window": 0,
         "pattern": 2, "lse": False},
        # four requests at their start: latency
        {"name": "attn_short_bf16", "op": "attn", "dtype": "bf16", "seqs": 4, "new": 1,
         "total": 611, "hk": 2, "group": 8, "d": 128, "page": 16, "window": 0,
         "pattern": 3, "lse": False},
        # a small model in fp32, three key heads, with the log-sum-exp for a join by the caller
        {"name": "attn_f32_odd", "op": "attn", "dtype": "f32", "seqs": 7, "new": 1,
         "total": 9001, "hk": 3, "group": 2, "d": 64, "page": 32, "window": 0,
         "pattern": 4, "lse": True},
        # four drafted tokens of 32 requests checked in one call, a window over the last 4,000 keys
        {"name": "attn_verify_bf16", "op": "attn", "dtype": "bf16", "seqs": 32, "new": 4,
         "total": 65536, "hk": 2, "group": 8, "d": 256, "page": 32, "window": 4000,
         "pattern": 5, "lse": False},
        # 64 requests forked: their last pages in the key and value pools of 24 layers
        {"name": "copy_pages_bf16", "op": "copy", "dtype": "bf16", "pools": 48, "slots": 256,
         "pairs": 64, "elems": 8192, "second": 0},
        # 24 states of recurrent layers moved to other slots: 48 heads of 128 x 128 in fp32, and
        # their convolution's last inputs
        {"name": "copy_states_f32", "op": "copy", "dtype": "f32", "pools": 1, "slots": 96,
         "pairs": 24, "elems": 786432, "second": 30720},
    ]


def _spread(rng, lo, hi):
    """A whole number of [lo, hi], even over the logarithm."""
    return max(lo, min(hi, round(lo * (hi / lo) ** rng.random())))


def draw(rng):
    op = rng.choice(("rotary", "rotary", "attn", "attn", "copy"))
    case = {"op": op, "dtype": rng.choice(("bf16", "bf16", "f32"))}
    size = 2 if case["dtype"] == "bf16" else 4
    if op == "rotary":
        case["dir"] = rng.choice(("fwd", "bwd", "append"))
        case["d"] = rng.choice((64, 128, 256, 2 * rng.randint(8, 160)))
        case["rot"] = rng.choice((case["d"], case["d"] // 2 & ~1, case["d"] // 4 & ~1))
        case["interleaved"] = rng.random() < 0.3
        case["hk"] = _spread(rng, 1, 16)
        case["hq"] = case["hk"] * _spread(rng, 1, 8)
        case["qnorm"] = rng.random() < 0.7
        case["knorm"] = rng.random() < 0.7
        per = (case["hq"] + 2 * case["hk"]) * case["d"] * size * 3
        case["tokens"] = _spread(rng, 1, max(1, min(16384, 200_000_000 // per)))
        if case["dir"] == "bwd":
            case["grad"] = rng.choice(("same", "f32"))
        if case["dir"] == "append":
            case["page"] = rng.choice((8, 16, 32, 64, 128))
    elif op == "attn":
        case["d"] = rng.choice((64, 128, 128, 256))
        case["hk"] = _spread(rng, 1, 16)
        case["group"] = _spread(rng, 1, 16)
        case["new"] = rng.choice((1, 1, 1, rng.randint(2, 8)))
        case["page"] = rng.choice((8, 16, 32, 64, 128))
        case["lse"] = rng.random() < 0.3
        per = 2 * case["hk"] * case["d"] * size
        case["seqs"] = _spread(rng, 1, 64)
        least = case["seqs"] * case["new"]
        case["total"] = _spread(rng, least, max(least + 1, min(262144, 500_000_000 // per)))
        case["window"] = 0 if rng.random() < 0.7 else _spread(rng, 1, case["total"])
        case["pattern"] = rng.randint(0, 1 << 20)
    else:
        case["elems"] = _spread(rng, 1, 1 << 20)
        case["second"] = rng.choice((0, _spread(rng, 1, 1 << 15)))
        case["pools"] = _spread(rng, 1, 96)
        per = case["pools"] * (case["elems"] + case["second"]) * size
        case["pairs"] = _spread(rng, 1, max(1, min(512, 100_000_000 // per)))
        case["slots"] = 2 * case["pairs"] + rng.randint(0, case["pairs"])
        case["pools"] = max(1, min(case["pools"], 400_000_000 // (per // case["pools"] * case["slots"])))
    return case


# ---- inputs ------------------------------------------------------------------------------


class _Draw:
    def __init__(self, seed):
        self.gen = torch.Generator(device="cuda")
        self.gen.manual_seed(seed)

    def normal(self, *shape, dtype=torch.float32, std=1.0):
        x = torch.randn(*shape, generator=self.gen, device="cuda", dtype=torch.float32)
        return (x * std).to(dtype)

    def perm(self, n):
        return torch.randperm(n, generator=self.gen, device="cuda")


def _lens(case):
    """Cached lengths of the sequences, the new tokens among them: uneven, `total` together; some
    may be empty unless the log-sum-exp is asked for."""
    n, least = case["seqs"], case["new"] if case["lse"] else 0
    rng = random.Random(case["pattern"])
    free = case["total"] - n * least
    cuts = [0] + sorted(rng.randint(0, free) for _ in range(n - 1)) + [free]
    return [least + b - a for a, b in zip(cuts, cuts[1:])]


def _table(positions, rot):
    """cos and sin of every position's angles, rounded once from 64 bits."""
    i = torch.arange(rot // 2, device="cuda", dtype=torch.float64)
    inv = 10000.0 ** (-2.0 * i / max(rot, 1))
    angle = torch.arange(positions, device="cuda", dtype=torch.float64)[:, None] * inv
    return torch.cat((angle.cos(), angle.sin()), 1).float()


def prepare(case, seed):
    g = _Draw(seed)
    dt = DTYPES[case["dtype"]]
    s = {"case": case}
    {"rotary": _prepare_rotary, "attn": _prepare_attn, "copy": _prepare_copy}[case["op"]](case, g, dt, s)
    return s


def _prepare_rotary(case, g, dt, s):
    T, hq, hk, d = case["tokens"], case["hq"], case["hk"], case["d"]
    lead = (T, 1) if case["dir"] == "append" and T <= 256 else (1, T)
    # queries, keys and values are column slices of one projection's output
    proj = g.normal(*lead, (hq + 2 * hk) * d, dtype=dt)
    s["q"] = proj[..., :hq * d].unflatten(-1, (hq, d))
    s["k"] = proj[..., hq * d:(hq + hk) * d].unflatten(-1, (hk, d))
    s["qw"] = 1.0 + g.normal(d, std=0.1) if case["qnorm"] else None
    s["kw"] = 1.0 + g.normal(d, std=0.1) if case["knorm"] else None
    far = 8192
    s["table"] = _table(far, case["rot"])
    if lead[1] == 1:        # single tokens: every sequence at a place of its own
        pos = torch.randint(0, far, lead, generator=g.gen, device="cuda")
    else:                   # packed sequences: positions start again at every one's first token
        starts = torch.randint(0, T, (min(8, T),), generator=g.gen, device="cuda")
        t = torch.arange(T, device="cuda")
        starts = torch.cat((starts, torch.zeros(1, dtype=torch.long, device="cuda")))
        begin = torch.where(starts[None] <= t[:, None], starts[None], 0).amax(1)
        pos = ((t - begin) % far)[None]
    s["pos"] = pos.to(torch.int32)
    if case["dir"] == "bwd":
        gt = torch.float32 if case["grad"] == "f32" else dt
        s["dq"] = g.normal(*lead, hq, d, dtype=gt)
        s["dk"] = g.normal(*lead, hk, d, dtype=gt)
    if case["dir"] == "append":
        s["v"] = proj[..., (hq + hk) * d:].unflatten(-1, (hk, d))
        page = case["page"]
        pages = -(-T // page) + 3
        s["k_pages"] = g.normal(pages, hk, page, d, dtype=dt)
        s["v_pages"] = g.normal(pages, hk, page, d, dtype=dt)
        s["slots"] = g.perm(pages * page)[:T].to(torch.int32).view(lead)


def _prepare_attn(case, g, dt, s):
    n, t, hk, d, page = case["seqs"], case["new"], case["hk"], case["d"], case["page"]
    lens = _lens(case)
    need = [-(-length // page) for length in lens]
    width = max(1, max(need)) + 1
    pages = sum(need) + 2
    order = g.perm(pages).to(torch.int32)
    # page ids of every sequence, and -1 behind its last page
    table = torch.full((n, width), -1, dtype=torch.int32, device="cuda")
    at = 0
    for i, k in enumerate(need):
        table[i, :k] = order[at:at + k]
        at += k
    s["table"] = table
    s["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    s["k_pages"] = g.normal(pages, hk, page, d, dtype=dt)
    s["v_pages"] = g.normal(pages, hk, page, d, dtype=dt)
    # scores with a spread of about 2.5: a few keys carry most of a row
    s["q"] = g.normal(n, t, hk * case["group"], d, dtype=dt, std=2.5)
    s["scale"] = d ** -0.5


def _prepare_copy(case, g, dt, s):
    slots, pairs = case["slots"], case["pairs"]
    s["pools"] = [g.normal(slots, case["elems"], dtype=dt) for _ in range(case["pools"])]
    if case["second"]:
        s["pools"] += [g.normal(slots, case["second"], dtype=dt) for _ in range(case["pools"])]
    order = g.perm(slots).to(torch.int32)
    s["src"], s["dst"] = order[:pairs].contiguous(), order[pairs:2 * pairs].contiguous()


# ---- one pass ----------------------------------------------------------------------------


def run(state):
    case = state["case"]
    return (_OWN if own else _PLAIN)[case["op"], case.get("dir")](state, case)


def _own_rotary_fwd(s, case):
    import gated_delta_rule_gdn_amd as g
    q, k = g.qk_rotary_fwd(s["q"], s["k"], s["table"], positions=s["pos"], q_weight=s["qw"],
                           k_weight=s["kw"], interleaved=case["interleaved"], eps=EPS)
    return {"q": q, "k": k}


def _own_rotary_bwd(s, case):
    import gated_delta_rule_gdn_amd as g
    return g.qk_rotary_bwd(s["q"], s["k"], s["table"], s["dq"], s["dk"], positions=s["pos"],
                           q_weight=s["qw"], k_weight=s["kw"], interleaved=case["interleaved"],
                           eps=EPS)


def _own_rotary_append(s, case):
    import gated_delta_rule_gdn_amd as g
    q = g.qk_rotary_append(s["q"], s["k"], s["v"], s["table"], s["pos"], s["k_pages"],
                           s["v_pages"], s["slots"], q_weight=s["qw"], k_weight=s["kw"],
                           interleaved=case["interleaved"], eps=EPS)
    return {"q": q, "k_pages": s["k_pages"], "v_pages": s["v_pages"]}


def _own_attn(s, case):
    import gated_delta_rule_gdn_amd as g
    o = g.paged_attention_step(s["q"], s["k_pages"], s["v_pages"], s["table"], s["lens"],
                               scale=s["scale"], window=case["window"], return_lse=case["lse"])
    return {"o": o[0], "lse": o[1]} if case["lse"] else {"o": o}


def _own_copy(s, case):
    import gated_delta_rule_gdn_amd as g
    g.pool_copy(s["pools"], s["src"], s["dst"])
    return s["pools"]


def _halves(x, rot, interleaved):
    """The two members of every rotated pair, and the values that are not rotated."""
    if interleaved:
        return x[..., 0:rot:2], x[..., 1:rot:2], x[..., rot:]
    return x[..., :rot // 2], x[..., rot // 2:rot], x[..., rot:]


def _rejoin(a, b, rest, interleaved):
    ab = torch.stack((a, b), -1).flatten(-2) if interleaved else torch.cat((a, b), -1)
    return torch.cat((ab, rest), -1)


def _angles(s, case):
    rows = s["table"][s["pos"].long()][:, :, None]
    half = case["rot"] // 2
    return rows[..., :half], rows[..., half:]


def _normed(x, w):
    if w is None:
        return x
    return x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * w


def _plain_turn(x, w, s, case):
    cos, sin = _angles(s, case)
    a, b, rest = _halves(_normed(x.float(), w), case["rot"], case["interleaved"])
    y = _rejoin(a * cos - b * sin, b * cos + a * sin, rest, case["interleaved"])
    return y.to(x.dtype)


def _plain_rotary_fwd(s, case):
    return {"q": _plain_turn(s["q"], s["qw"], s, case), "k": _plain_turn(s["k"], s["kw"], s, case)}


def _plain_turn_bwd(x, w, dy, s, case):
    cos, sin = _angles(s, case)
    a, b, rest = _halves(dy.float(), case["rot"], case["interleaved"])
    e = _rejoin(a * cos + b * sin, b * cos - a * sin, rest, case["interleaved"])
    if w is None:
        return e.to(dy.dtype), None
    x = x.float()
    r = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
    dw = (e * x * r).flatten(0, 2).sum(0)
    g = e * w
    dx = r * g - x * r ** 3 * (g * x).mean(-1, keepdim=True)
    return dx.to(dy.dtype), dw


def _plain_rotary_bwd(s, case):
    dq, dqw = _plain_turn_bwd(s["q"], s["qw"], s["dq"], s, case)
    dk, dkw = _plain_turn_bwd(s["k"], s["kw"], s["dk"], s, case)
    out = {"dq": dq, "dk": dk, "dq_weight": dqw, "dk_weight": dkw}
    return {n: t for n, t in out.items() if t is not None}


def _plain_rotary_append(s, case):
    q = _plain_turn(s["q"], s["qw"], s, case)
    k = _plain_turn(s["k"], s["kw"], s, case)
    at = s["slots"].flatten().long()
    page, off = at // case["page"], at % case["page"]
    s["k_pages"][page, :, off] = k.flatten(0, 1)
    s["v_pages"][page, :, off] = s["v"].flatten(0, 1)
    return {"q": q, "k_pages": s["k_pages"], "v_pages": s["v_pages"]}


def _plain_attn(s, case):
    n, t, g, hk, d = case["seqs"], case["new"], case["group"], case["hk"], case["d"]
    ids = s["table"].clamp(min=0).long()

    def rows(pages):        # [n, hk, longest, d]
        return pages[ids].transpose(1, 2).flatten(2, 3).float()

    q = s["q"].float().view(n, t, hk, g, d).permute(0, 2, 1, 3, 4).reshape(n, hk, t * g, d)
    k, v = rows(s["k_pages"]), rows(s["v_pages"])
    score = torch.matmul(q, k.transpose(2, 3).contiguous()) * s["scale"]
    score = score.view(n, hk, t, g, -1)
    j = torch.arange(score.shape[-1], device="cuda")
    at = s["lens"].long()[:, None] - t + torch.arange(t, device="cuda")
    sees = j <= at[..., None]
    if case["window"]:
        sees &= j > at[..., None] - case["window"]
    sees = sees[:, None, :, None]
    score = torch.where(sees, score, -math.inf)
    top = score.amax(-1, keepdim=True).clamp(min=-3e38)
    p = torch.exp(score - top)
    total = p.sum(-1, keepdim=True)
    p = p / total.clamp(min=1e-38)
    o = torch.matmul(p.flatten(2, 3), v).view(n, hk, t, g, d)
    out = {"o": o.permute(0, 2, 1, 3, 4).reshape(n, t, hk * g, d).to(s["q"].dtype)}
    if case["lse"]:
        lse = (top + torch.log(total))[..., 0]
        out["lse"] = lse.permute(0, 2, 1, 3).reshape(n, t, hk * g)
    return out


def _plain_copy(s, case):
    src, dst = s["src"].long(), s["dst"].long()
    for pool in s["pools"]:
        pool[dst] = pool[src]
    return s["pools"]


_PLAIN = {("rotary", "fwd"): _plain_rotary_fwd, ("rotary", "bwd"): _plain_rotary_bwd,
          ("rotary", "append"): _plain_rotary_append, ("attn", None): _plain_attn,
          ("copy", None): _plain_copy}
_OWN = {("rotary", "fwd"): _own_rotary_fwd, ("rotary", "bwd"): _own_rotary_bwd,
        ("rotary", "append"): _own_rotary_append, ("attn", None): _own_attn,
        ("copy", None): _own_copy}


# ---- what a pass cannot do without -------------------------------------------------------


def work(case):
    size = 4 if case["dtype"] == "f32" else 2
    if case["op"] == "rotary":
        T, d = case["tokens"], case["d"]
        cells = T * (case["hq"] + case["hk"]) * d
        extra = 4 * T + 4 * d * (case["qnorm"] + case["knorm"]) + 4 * min(T, 8192) * case["rot"]
        if case["dir"] == "fwd":
            return {"bytes": 2 * cells * size + extra, "flops": 8 * cells}
        if case["dir"] == "append":
            values = T * case["hk"] * d
            return {"bytes": 2 * (cells + values) * size + 4 * T + extra, "flops": 8 * cells}
        grad = 4 if case["grad"] == "f32" else size
        inputs = T * d * (case["hq"] * case["qnorm"] + case["hk"] * case["knorm"])
        return {"bytes": inputs * size + 2 * cells * grad + 2 * extra, "flops": 18 * cells}
    if case["op"] == "attn":
        hk, g, d, t = case["hk"], case["group"], case["d"], case["new"]
        w = case["window"]
        lens = _lens(case)
        # keys that a sequence's new tokens see together, and pairs of a token and a key it sees
        keys = sum(min(n, w + t - 1) if w else n for n in lens)
        pairs = sum(min(n - i, w) if w else n - i for n in lens for i in range(min(t, n)))
        rows = case["seqs"] * t * hk * g
        pages = sum(-(-n // case["page"]) for n in lens)
        return {"bytes": 2 * keys * hk * d * size + 2 * rows * d * size + 4 * pages
                + 4 * case["seqs"] + 4 * rows * case["lse"], "flops": 4 * pairs * hk * g * d}
    moved = case["pools"] * case["pairs"] * (case["elems"] + case["second"]) * size
    return {"bytes": 2 * moved + 8 * case["pairs"], "flops": 0}


# ---- the definitions in 64 bits ----------------------------------------------------------


def _exact_rotate(x, w, s, case):
    """[B, T, H, d] in 64 bits: the norm, then every pair turned as a complex number."""
    rot = case["rot"]
    if w is not None:
        x = x / torch.sqrt(x.square().mean(-1, keepdim=True) + EPS) * w
    if rot == 0:
        return x
    row = s["table"].double()[s["pos"].long()]
    turn = torch.complex(row[..., :rot // 2], row[..., rot // 2:])[:, :, None]
    y = x[..., :rot]
    y = y.unflatten(-1, (rot // 2, 2)) if case["interleaved"] else y.unflatten(-1, (2, rot // 2)).transpose(-1, -2)
    z = torch.view_as_real(torch.view_as_complex(y.contiguous()) * turn)
    z = z.flatten(-2) if case["interleaved"] else z.transpose(-1, -2).flatten(-2)
    return torch.cat((z, x[..., rot:]), -1)


def _exact_rotary(s, case):
    names = {"q": "qw", "k": "kw"}
    leaf = {n: None if s[n] is None else s[n].double().clone() for n in ("q", "k", "qw", "kw")}
    if case["dir"] != "bwd":
        out = {n: _exact_rotate(leaf[n], leaf[w], s, case) for n, w in names.items()}
        if case["dir"] == "fwd":
            return out
        kp, vp = s["k_pages"].double(), s["v_pages"].double()
        k, v = out["k"].flatten(0, 1), s["v"].double().flatten(0, 1)
        for i, slot in enumerate(s["slots"].flatten().tolist()):
            page, off = divmod(slot, case["page"])
            kp[page, :, off], vp[page, :, off] = k[i], v[i]
        return {"q": out["q"], "k_pages": kp, "v_pages": vp}
    for t in leaf.values():
        if t is not None:
            t.requires_grad_(True)
    loss = sum((_exact_rotate(leaf[n], leaf[w], s, case) * s["d" + n].double()).sum()
               for n, w in names.items())
    loss.backward()
    out = {"dq": leaf["q"].grad, "dk": leaf["k"].grad}
    for n, w in names.items():
        if leaf[w] is not None:
            out["d" + n + "_weight"] = leaf[w].grad
    return out


def _exact_attn(s, case):
    n, t, g, hk, d = case["seqs"], case["new"], case["group"], case["hk"], case["d"]
    o = torch.zeros(n, t, hk * g, d, dtype=torch.float64, device="cuda")
    lse = torch.full((n, t, hk * g), -math.inf, dtype=torch.float64, device="cuda")
    for i, length in enumerate(_lens(case)):
        used = s["table"][i, :-(-length // case["page"])].long()
        for h in range(hk):
            k = s["k_pages"][used, h].double().flatten(0, 1)
            v = s["v_pages"][used, h].double().flatten(0, 1)
            for a in range(t):
                end = length - t + a + 1
                begin = max(0, end - case["window"]) if case["window"] else 0
                if end <= begin:
                    continue
                rows = slice(h * g, (h + 1) * g)
                score = s["q"][i, a, rows].double() @ k[begin:end].t() * s["scale"]
                lse[i, a, rows] = torch.logsumexp(score, -1)
                o[i, a, rows] = torch.exp(score - lse[i, a, rows, None]) @ v[begin:end]
    return {"o": o, "lse": lse} if case["lse"] else {"o": o}


def _exact_copy(s, case):
    out = [pool.double() for pool in s["pools"]]
    for a, b in zip(s["src"].tolist(), s["dst"].tolist()):
        for pool in out:
            pool[b] = pool[a]
    return out


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rotary":
        return _exact_rotary(s, case)
    return _exact_attn(s, case) if case["op"] == "attn" else _exact_copy(s, case)
