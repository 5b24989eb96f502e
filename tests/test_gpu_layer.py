"""The operators around the recurrence used together: whole layers with their gradients, a prompt
continued token by token, captured graphs and other streams.

Gate: relative L2 error at most 1e-4 in fp32, the bar of the parity tests (layers of a few
products of at most 64 terms between calls that are each within about 100 * 2^-24)."""
import pytest
import torch
import torch.nn.functional as F

import gated_delta_rule_gdn_amd as g
from gpu_common import TOL
from test_gpu_graphs import capture

pytestmark = pytest.mark.gpu


def setup_module(module):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    g.lib()


def rel(a, b):
    return float((a.double().cpu() - b.double().cpu()).norm() / b.double().norm().clamp(min=1e-30))


def draw(gen, *shape, std=1.0):
    return torch.randn(*shape, generator=gen) * std


def rms(x, w, eps=1e-5):
    return x / (x.square().mean(-1, keepdim=True) + eps).sqrt() * w


# ---- a layer of the selective scan -------------------------------------------------------

HID, CH, M, RANK = 48, 64, 8, 4


def scan_layer_weights(seed):
    gen = torch.Generator().manual_seed(seed)
    return {"norm": 1 + 0.1 * draw(gen, HID), "w_in": draw(gen, HID, 2 * CH, std=HID ** -0.5),
            "conv_w": draw(gen, CH, 4, std=0.5), "conv_b": draw(gen, CH, std=0.1),
            "w_x": draw(gen, CH, RANK + 2 * M, std=CH ** -0.5), "w_dt": draw(gen, RANK, CH, std=0.5),
            "dt_bias": draw(gen, CH, std=0.3) - 3, "A": -torch.arange(1, M + 1) * torch.exp(draw(gen, CH, M, std=0.1)),
            "D": 1 + 0.1 * draw(gen, CH), "out_norm": 1 + 0.1 * draw(gen, CH),
            "w_out": draw(gen, CH, HID, std=CH ** -0.5), "scale": 0.5 + 0.1 * draw(gen, HID),
            "next": 1 + 0.1 * draw(gen, HID)}


def scan_layer_ref(x, p, lens):
    """The layer in 64 bits from the definitions: pre-norm, projection, convolution, scan, gated
    norm, projection, scaled residual, next norm."""
    res = x
    xz = rms(x, p["norm"]) @ p["w_in"]
    u, z = xz.split(CH, -1)
    outs, at = [], 0
    for n in lens:
        uu = F.pad(u[at:at + n], (0, 0, 3, 0))
        c = sum(uu[j:j + n] * p["conv_w"][:, j] for j in range(4)) + p["conv_b"]
        c = c * torch.sigmoid(c)
        dbl = c @ p["w_x"]
        dt = F.softplus(dbl[:, :RANK] @ p["w_dt"] + p["dt_bias"])
        B, C = dbl[:, RANK:RANK + M], dbl[:, RANK + M:]
        h, ys = torch.zeros(CH, M, dtype=x.dtype), []
        for t in range(n):
            h = torch.exp(dt[t][:, None] * p["A"]) * h + (dt[t] * c[t])[:, None] * B[t]
            ys.append((h * C[t]).sum(-1) + p["D"] * c[t])
        outs.append(torch.stack(ys) if ys else c)
        at += n
    y = torch.cat(outs)
    y = rms(y, p["out_norm"]) * z * torch.sigmoid(z)
    hid = res + p["scale"] * (y @ p["w_out"])
    return hid, rms(hid, p["next"])


def scan_layer(x, p, cu):
    """The layer on the GPU, [1,T,HID]; what the backward needs is returned too."""
    n, _ = g.block_norm_fwd(x, norm_weight=p["norm"])
    xz = n @ p["w_in"]
    c, _ = g.short_conv_fwd(xz[..., :CH], p["conv_w"], bias=p["conv_b"], cu_seqlens=cu, silu=True)
    dbl = c @ p["w_x"]
    dt = dbl[..., :RANK] @ p["w_dt"]
    B, C = (dbl[..., RANK + i * M:RANK + (i + 1) * M].unflatten(-1, (1, M)) for i in (0, 1))
    y, _ = g.selective_scan_fwd(c, dt, p["A"], B, C, D=p["D"], dt_bias=p["dt_bias"], dt_softplus=True,
                                cu_seqlens=cu)
    o, _ = g.block_norm_fwd(y, norm_weight=p["out_norm"], gate=xz[..., CH:])
    w = o @ p["w_out"]
    hid, nxt = g.block_norm_fwd(w, residual=x, scale=p["scale"], next_weight=p["next"])
    return hid, nxt, (n, xz, c, dbl, dt, B, C, y, o, w)


def scan_layer_bwd(x, p, cu, kept, dhid, dnxt):
    n, xz, c, dbl, dt, B, C, y, o, w = kept
    gr = {}
    e = g.block_norm_bwd(w, dh=dhid, dy=dnxt, residual=x, scale=p["scale"], next_weight=p["next"])
    gr["scale"], gr["next"], dx = e["dscale"], e["dnext_weight"], e["dresidual"]
    flat = lambda t: t.flatten(0, 1)  # noqa: E731
    gr["w_out"] = flat(o).t() @ flat(e["dx"])
    do = e["dx"] @ p["w_out"].t()
    e = g.block_norm_bwd(y, dh=do, norm_weight=p["out_norm"], gate=xz[..., CH:])
    gr["out_norm"], dz = e["dnorm_weight"], e["dgate"]
    s = g.selective_scan_bwd(c, dt, p["A"], B, C, e["dx"], D=p["D"], dt_bias=p["dt_bias"], dt_softplus=True,
                             cu_seqlens=cu)
    gr["A"], gr["D"], gr["dt_bias"] = s["dA"], s["dD"], s["ddt_bias"]
    gr["w_dt"] = flat(dbl[..., :RANK]).t() @ flat(s["ddt"])
    ddbl = torch.cat((s["ddt"] @ p["w_dt"].t(), s["dB"].flatten(2), s["dC"].flatten(2)), -1)
    gr["w_x"] = flat(c).t() @ flat(ddbl)
    dc = s["dx"] + ddbl @ p["w_x"].t()
    e = g.short_conv_bwd(xz[..., :CH], p["conv_w"], dc, bias=p["conv_b"], cu_seqlens=cu, silu=True)
    gr["conv_w"], gr["conv_b"] = e["dweight"], e["dbias"]
    dxz = torch.cat((e["dx"], dz), -1)
    gr["w_in"] = flat(n).t() @ flat(dxz)
    e = g.block_norm_bwd(x, dh=dxz @ p["w_in"].t(), norm_weight=p["norm"])
    gr["norm"] = e["dnorm_weight"]
    return dx + e["dx"], gr


def test_scan_layer_and_its_gradients():
    lens = [23, 0, 1, 40]
    T = sum(lens)
    p = scan_layer_weights(1)
    gen = torch.Generator().manual_seed(2)
    x, dh, dn = (draw(gen, T, HID) for _ in range(3))
    q = {n: t.double().requires_grad_(True) for n, t in p.items()}
    xd = x.double().requires_grad_(True)
    hid_r, nxt_r = scan_layer_ref(xd, q, lens)
    ((hid_r * dh).sum() + (nxt_r * dn).sum()).backward()
    cu = torch.tensor([0] + list(torch.tensor(lens).cumsum(0)), dtype=torch.int32, device="cuda")
    pg = {n: t.cuda() for n, t in p.items()}
    hid, nxt, kept = scan_layer(x.cuda()[None], pg, cu)
    dx, gr = scan_layer_bwd(x.cuda()[None], pg, cu, kept, dh.cuda()[None], dn.cuda()[None])
    torch.cuda.synchronize()
    tol = TOL[torch.float32]
    assert rel(hid[0], hid_r) <= tol and rel(nxt[0], nxt_r) <= tol
    assert rel(dx[0], xd.grad) <= tol
    assert set(gr) == set(p)
    for n in sorted(p):
        print(f"[layer] d{n}: {rel(gr[n], q[n].grad):.2e}", flush=True)
        assert rel(gr[n], q[n].grad) <= tol, n


def test_scan_layer_prompt_then_tokens():
    """Three requests prefilled together, packed, then decoded from a pool of slots one token at a
    time: the outputs and states of the whole prompts."""
    lens, more, slots = [5, 1, 12], 6, [3, 0, 2]
    p = {n: t.cuda() for n, t in scan_layer_weights(3).items()}
    gen = torch.Generator().manual_seed(4)
    c = [draw(gen, n + more, CH).cuda() for n in lens]       # the projection's output
    dt = [draw(gen, n + more, CH).cuda() for n in lens]
    B, C = ([draw(gen, n + more, 1, M).cuda() for n in lens] for _ in range(2))
    z = [draw(gen, n + more, CH).cuda() for n in lens]

    def prompt(cut):
        part = lambda v: torch.cat([t[:n] for t, n in zip(v, cut)])[None]  # noqa: E731
        cu = torch.tensor([0] + list(torch.tensor(cut).cumsum(0)), dtype=torch.int32, device="cuda")
        x, cs = g.short_conv_fwd(part(c), p["conv_w"], bias=p["conv_b"], cu_seqlens=cu, silu=True)
        o, S = g.selective_scan_fwd(x, part(dt), p["A"], part(B), part(C), D=p["D"], gate=part(z),
                                    dt_bias=p["dt_bias"], dt_softplus=True, cu_seqlens=cu)
        return o[0].split(cut), cs, S

    whole, cs_r, S_r = prompt([n + more for n in lens])
    first, cs, S = prompt(lens)
    idx = torch.tensor(slots, dtype=torch.int32, device="cuda")
    conv_pool = torch.full((5, 3, CH), 7.0, device="cuda")
    pool = torch.full((5, CH, M), 7.0, device="cuda")
    conv_pool[idx.long()], pool[idx.long()] = cs, S
    steps = []
    for t in range(more):
        at = lambda v: torch.stack([a[n + t:n + t + 1] for a, n in zip(v, lens)])  # noqa: E731
        x = g.short_conv_step(at(c), p["conv_w"], conv_pool, bias=p["conv_b"], state_idx=idx, silu=True)
        steps.append(g.selective_scan_step(x, at(dt), p["A"], at(B), at(C), pool, D=p["D"], gate=at(z),
                                           dt_bias=p["dt_bias"], dt_softplus=True, state_idx=idx))
    torch.cuda.synchronize()
    got = torch.cat(steps, 1)
    tol = TOL[torch.float32]
    for i, n in enumerate(lens):
        assert rel(first[i], whole[i][:n]) <= tol and rel(got[i], whole[i][n:]) <= tol
    assert torch.equal(conv_pool[idx.long()], cs_r) and rel(pool[idx.long()], S_r) <= tol
    assert torch.all(pool[[1, 4]] == 7.0) and torch.all(conv_pool[[1, 4]] == 7.0)


# ---- a layer of the delta rule -----------------------------------------------------------


def test_delta_rule_layer_trains_through_its_convolution_and_norm():
    """Short convolution of q, k, v -> chunked forward -> gated norm, and back through
    block_norm_bwd, chunk_bwd and short_conv_bwd (its fp32 gradients go straight in)."""
    B, T, H, d = 2, 70, 2, 64
    gen = torch.Generator().manual_seed(5)
    C = 3 * H * d
    x = draw(gen, B, T, C, std=0.5)
    cw = draw(gen, C, 4, std=0.3)
    la = -F.softplus(draw(gen, B, T, H, d))
    b, w = torch.sigmoid(draw(gen, B, T, H, d)), torch.sigmoid(draw(gen, B, T, H, d))
    gate, nw, dy = draw(gen, B, T, H, d), 1 + 0.1 * draw(gen, d), draw(gen, B, T, H, d)

    v = {n: t.double().requires_grad_(True) for n, t in (("x", x), ("cw", cw), ("gate", gate), ("nw", nw))}
    pad = F.pad(v["x"], (0, 0, 3, 0))
    a = sum(pad[:, j:j + T] * v["cw"][:, j] for j in range(4))
    a = 0.3 * a * torch.sigmoid(a)
    q, k, vv = (t.unflatten(-1, (H, d)) for t in a.split(H * d, -1))
    S, os_ = torch.zeros(B, H, d, d, dtype=torch.float64), []
    lad, bd, wd = la.double(), b.double(), w.double()
    for t in range(T):
        S = torch.exp(lad[:, t])[..., None] * S
        S = S - k[:, t][..., None] * ((bd[:, t] * k[:, t])[..., None] * S).sum(-2, keepdim=True) \
            + k[:, t][..., None] * (wd[:, t] * vv[:, t])[..., None, :]
        os_.append((q[:, t][..., None] * S).sum(-2))
    o_r = rms(torch.stack(os_, 1), v["nw"]) * v["gate"] * torch.sigmoid(v["gate"])
    (o_r * dy.double()).sum().backward()

    dev = lambda t: t.cuda()  # noqa: E731
    y, _ = g.short_conv_fwd(dev(x), dev(cw), silu=True)
    q, k, vv = (0.3 * t.unflatten(-1, (H, d)).contiguous() for t in y.split(H * d, -1))
    o, _ = g.chunk_fwd(q, k, vv, dev(la), dev(b), dev(w))
    out, _ = g.block_norm_fwd(o, norm_weight=dev(nw), gate=dev(gate))
    e = g.block_norm_bwd(o, dh=dev(dy), norm_weight=dev(nw), gate=dev(gate))
    s = g.chunk_bwd(q, k, vv, dev(la), dev(b), dev(w), e["dx"])
    da = 0.3 * torch.cat([s[n].flatten(2) for n in ("dq", "dk", "dv")], -1)
    r = g.short_conv_bwd(dev(x), dev(cw), da, silu=True)
    torch.cuda.synchronize()
    tol = TOL[torch.float32]
    for n, got, want in (("o", out, o_r), ("dx", r["dx"], v["x"].grad), ("dcw", r["dweight"], v["cw"].grad),
                         ("dgate", e["dgate"], v["gate"].grad), ("dnw", e["dnorm_weight"], v["nw"].grad)):
        print(f"[layer] {n}: {rel(got, want):.2e}", flush=True)
        assert rel(got, want) <= tol, n


# ---- graphs and streams ------------------------------------------------------------------


def calls():
    """Every call on its own inputs: name -> (function, state tensors it updates in place)."""
    gen = torch.Generator().manual_seed(6)
    bf = lambda *s: draw(gen, *s).to(torch.bfloat16).cuda()  # noqa: E731
    f32 = lambda *s: draw(gen, *s).cuda()  # noqa: E731
    T, ch, m = 300, 264, 16
    x, dt, z, dO = (bf(1, T, ch) for _ in range(4))
    B, C = bf(1, T, 1, m), bf(1, T, 1, m)
    A, cw, D, bias, w = -f32(ch, m).abs(), f32(ch, 4), f32(ch), f32(ch) - 3, f32(ch)
    cu = torch.tensor([0, 120, 120, 290], dtype=torch.int32, device="cuda")
    S0, s0 = f32(3, ch, m), f32(3, 3, ch)
    cpool, spool = f32(4, 3, ch), f32(4, ch, m)
    idx = torch.tensor([2, -1, 0], dtype=torch.int32, device="cuda")
    xs, Bs = x[:, :6].reshape(3, 2, ch).contiguous(), B[:, :6].reshape(3, 2, 1, m).contiguous()
    scan = dict(D=D, gate=z, dt_bias=bias, dt_softplus=True)
    return {
        "short_conv_fwd": (lambda: g.short_conv_fwd(x, cw, state0=s0, cu_seqlens=cu, silu=True), ()),
        "short_conv_bwd": (lambda: g.short_conv_bwd(x, cw, dO, state0=s0, cu_seqlens=cu, silu=True), ()),
        "short_conv_step": (lambda: g.short_conv_step(xs, cw, cpool, state_idx=idx), (cpool,)),
        "selective_scan_fwd": (lambda: g.selective_scan_fwd(x, dt, A, B, C, S0=S0, cu_seqlens=cu, **scan), ()),
        "selective_scan_bwd": (lambda: g.selective_scan_bwd(x, dt, A, B, C, dO, S0=S0, cu_seqlens=cu, **scan), ()),
        "selective_scan_step": (lambda: g.selective_scan_step(xs, xs, A, Bs, Bs, spool, D=D, state_idx=idx), (spool,)),
        "block_norm_fwd": (lambda: g.block_norm_fwd(x, w, z, dO, D, w), ()),
        "block_norm_bwd": (lambda: g.block_norm_bwd(x, dO, dt, w, z, dO, D, w), ()),
    }


def tensors(out):
    vals = out.values() if isinstance(out, dict) else out if isinstance(out, tuple) else (out,)
    return [t for t in vals if t is not None]


NAMES = ["short_conv_fwd", "short_conv_bwd", "short_conv_step", "selective_scan_fwd", "selective_scan_bwd",
         "selective_scan_step", "block_norm_fwd", "block_norm_bwd"]
LIVE = 290          # tokens of the packed calls that belong to a sequence


def live(name, ts):
    """The rows that a packed call writes."""
    packed = name.startswith(("short_conv", "selective_scan")) and not name.endswith("step")
    return [t[:, :LIVE] if packed and t.dim() >= 3 and t.shape[:2] == (1, 300) else t for t in ts]


@pytest.mark.parametrize("name", NAMES)
def test_replayed_graph_equals_eager(name):
    """Captured once, replayed with eager work and synchronisations between: the eager bits."""
    fn, states = calls()[name]
    keep = [t.clone() for t in states]
    reset = lambda: [t.copy_(k) for t, k in zip(states, keep)]  # noqa: E731
    want = [t.clone() for t in live(name, tensors(fn()))] + [t.clone() for t in states]
    box = {}

    def body():
        box["out"] = fn()

    graph = capture(body)
    for rep in range(3):
        reset()
        for t in tensors(box["out"]):
            t.fill_(float("nan"))
        fn2, _ = calls()[name]      # eager calls on other buffers between the replays
        fn2()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        got = live(name, tensors(box["out"])) + list(states)
        assert all(torch.equal(a, b) for a, b in zip(got, want)), (name, rep)


def test_two_graphs_keep_their_own_workspaces():
    """The backward captured twice: replays in turn, and each gives its own eager bits."""
    made = [calls(), calls()]
    fns = [m["selective_scan_bwd"][0] for m in made]
    want = [[t.clone() for t in live("selective_scan_bwd", tensors(f()))] for f in fns]
    boxes = [{}, {}]
    graphs = [capture(lambda f=f, b=b: b.update(out=f())) for f, b in zip(fns, boxes)]
    for _ in range(3):
        for gr in graphs:
            gr.replay()
        torch.cuda.synchronize()
        for b, w in zip(boxes, want):
            assert all(torch.equal(x, y) for x, y in zip(live("selective_scan_bwd", tensors(b["out"])), w))


@pytest.mark.parametrize("name", NAMES)
def test_runs_on_the_current_stream(name):
    """On a side stream behind a long-running producer of its input: ordered by the stream, and
    the same bits as on the default stream."""
    fn, states = calls()[name]
    keep = [t.clone() for t in states]
    want = [t.clone() for t in live(name, tensors(fn()))] + [t.clone() for t in states]
    for t, k in zip(states, keep):
        t.copy_(k)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        for _ in range(20):
            torch.zeros(1 << 24, device="cuda").add_(1.0)
        got = live(name, tensors(fn())) + list(states)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
