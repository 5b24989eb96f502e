"""The attention layer's operators used together, beside the recurrent ones: a layer's training step, a
batch that is prefilled, decoded, forked and compacted, captured graphs, other streams, two threads.

Gate of whole layers: relative L2 error at most 1e-4 in fp32, the bar of the parity tests."""
import threading

import pytest
import torch

import gated_delta_rule_gdn_amd as g
from gpu_common import TOL
from test_gpu_graphs import capture
from test_gpu_layer_streams import tensors

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16
I32 = dict(dtype=torch.int32, device="cuda")


def setup_module(module):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    g.lib()


def rel(a, b):
    a, b = a.detach().double().cpu(), b.detach().double().cpu()
    return float((a - b).norm() / b.norm().clamp(min=1e-30))


def draw(gen, *shape, std=1.0):
    return torch.randn(*shape, generator=gen) * std


HQ, HK, D, ROT, HID, PAGE = 4, 2, 64, 32, 48, 16


def weights(seed):
    gen = torch.Generator().manual_seed(seed)
    return {"w_in": draw(gen, HID, (HQ + 2 * HK) * D, std=HID ** -0.5), "qw": 1 + 0.1 * draw(gen, D),
            "kw": 1 + 0.1 * draw(gen, D), "w_out": draw(gen, HQ * D, HID, std=(HQ * D) ** -0.5)}


def split(proj):
    return (proj[..., :HQ * D].unflatten(-1, (HQ, D)), proj[..., HQ * D:(HQ + HK) * D].unflatten(-1, (HK, D)),
            proj[..., (HQ + HK) * D:].unflatten(-1, (HK, D)))


def turn_ref(x, w, cs, pos):
    x = x / (x.square().mean(-1, keepdim=True) + 1e-5).sqrt() * w
    c, s = cs[pos][:, None, :ROT // 2].double(), cs[pos][:, None, ROT // 2:].double()
    a, b = x[..., :ROT // 2], x[..., ROT // 2:ROT]
    return torch.cat((a * c - b * s, b * c + a * s, x[..., ROT:]), -1)


def layer_ref(x, p, cs):
    """A sequence [n, HID] through the layer in 64 bits."""
    n = len(x)
    q, k, v = split(x @ p["w_in"])
    pos = torch.arange(n)
    q, k = turn_ref(q, p["qw"], cs, pos), turn_ref(k, p["kw"], cs, pos)
    o = []
    for h in range(HQ):
        s = (q[:, h] @ k[:, h // (HQ // HK)].T) * D ** -0.5
        s = s.masked_fill(torch.ones(n, n).triu(1).bool(), -float("inf"))
        o.append(s.softmax(-1) @ v[:, h // (HQ // HK)])
    return torch.cat(o, -1) @ p["w_out"]


# ---- training ----------------------------------------------------------------------------


def test_layer_training_step():
    """Norms and rotation forward and backward around an attention in 64 bits on the CPU, packed
    sequences with positions of their own: output and every gradient of the layer."""
    lens = [23, 1, 40]
    p, gen = weights(1), torch.Generator().manual_seed(2)
    x, dy = draw(gen, sum(lens), HID), draw(gen, sum(lens), HID)
    cs = g.rotary_table(64, ROT)
    leaf = {n: t.double().requires_grad_(True) for n, t in {**p, "x": x}.items()}
    want = torch.cat([layer_ref(t, leaf, cs) for t in leaf["x"].split(lens)])
    (want * dy).sum().backward()

    pg = {n: t.cuda() for n, t in p.items()}
    xg, dyg, csg = x.cuda(), dy.cuda(), cs.cuda()
    pos = torch.cat([torch.arange(n) for n in lens]).to(torch.int32)[None].cuda()
    proj = (xg @ pg["w_in"])[None]
    q, k, v = split(proj)
    qr, kr = g.qk_rotary_fwd(q, k, csg, pos, pg["qw"], pg["kw"])
    qc, kc, vc = (t[0].double().cpu().requires_grad_(True) for t in (qr, kr, v))
    o = []
    for a, b, c in zip(qc.split(lens), kc.split(lens), vc.split(lens)):
        n = len(a)
        s = torch.einsum("ihd,jhd->hij", a, b.repeat_interleave(HQ // HK, 1)) * D ** -0.5
        s = s.masked_fill(torch.ones(n, n).triu(1).bool(), -float("inf")).softmax(-1)
        o.append(torch.einsum("hij,jhd->ihd", s, c.repeat_interleave(HQ // HK, 1)))
    o = torch.cat(o)
    og = o.detach().float().cuda().flatten(1)
    do = (dyg @ pg["w_out"].T).unflatten(1, (HQ, D))
    o.backward(do.double().cpu())
    gr = g.qk_rotary_bwd(q, k, csg, qc.grad.float().cuda()[None], kc.grad.float().cuda()[None], positions=pos,
                         q_weight=pg["qw"], k_weight=pg["kw"])
    dproj = torch.cat((gr["dq"].flatten(2), gr["dk"].flatten(2), vc.grad.float().cuda()[None].flatten(2)), -1)[0]
    got = {"w_in": xg.T @ dproj, "w_out": og.T @ dyg, "x": dproj @ pg["w_in"].T, "qw": gr["dq_weight"],
           "kw": gr["dk_weight"]}
    assert rel(og @ pg["w_out"], want) <= TOL[F32]
    for n, t in got.items():
        print(f"[attention layer] d{n}: {rel(t, leaf[n].grad):.2e}", flush=True)
        assert rel(t, leaf[n].grad) <= TOL[F32], n


# ---- serving -----------------------------------------------------------------------------


class Server:
    """Pages handed out by a program: a table per request, filled prompt by prompt and token by token."""

    def __init__(self, p, requests, pages, dtype):
        self.p = {n: t.cuda().to(dtype) if n.startswith("w_") else t.cuda() for n, t in p.items()}
        self.cs = g.rotary_table(256, ROT, device="cuda")
        self.kp = torch.full((pages, HK, PAGE, D), float("nan"), dtype=dtype, device="cuda")
        self.vp = torch.full_like(self.kp, float("nan"))
        self.table = torch.full((requests, 8), -1, dtype=torch.int32)
        self.lens = [0] * requests
        order = torch.randperm(pages, generator=torch.Generator().manual_seed(pages)).tolist()
        self.free = order

    def grow(self, i, n):
        self.lens[i] += n
        for j in range(-(-self.lens[i] // PAGE)):
            if self.table[i, j] < 0:
                self.table[i, j] = self.free.pop()

    def place(self, i, t):
        return int(self.table[i, t // PAGE]) * PAGE + t % PAGE

    def append(self, proj, who, where):
        """proj [B,T,...]; the request and the place in it of every token."""
        q, k, v = split(proj)
        slots = torch.tensor([[self.place(i, t) for i, t in zip(a, b)] for a, b in zip(who, where)], **I32)
        return g.qk_rotary_append(q, k, v, self.cs, torch.tensor(where, **I32), self.kp, self.vp, slots, self.p["qw"],
                                  self.p["kw"])

    def attend(self, q, rows):
        o = g.paged_attention_step(q, self.kp, self.vp, self.table[rows].cuda(), torch.tensor([self.lens[i] for i in rows], **I32))
        return o.flatten(2) @ self.p["w_out"]

    def prompts(self, xs):
        """Prompts packed into one append; each request's tokens then attend in one call of their own."""
        for i, x in enumerate(xs):
            self.grow(i, len(x))
        who = [[i for i, x in enumerate(xs) for _ in range(len(x))]]
        where = [[t for x in xs for t in range(len(x))]]
        q = self.append((torch.cat(xs) @ self.p["w_in"])[None], who, where)
        return [self.attend(t[None], [i])[0] for i, t in enumerate(q[0].split([len(x) for x in xs])) if len(t)]

    def tokens(self, x, rows):
        """The next T tokens of each request, x [N,T,HID]."""
        T = x.shape[1]
        for i in rows:
            self.grow(i, T)
        where = [[self.lens[i] - T + t for t in range(T)] for i in rows]
        return self.attend(self.append(x @ self.p["w_in"], [[i] * T for i in rows], where), rows)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_prefill_decode_fork_and_compact(dtype):
    """Three requests: prompts packed, three calls of one token and one of three, a fork that copies the
    last page alone and shares the rest, then all pages moved to the front of the pools. Every output
    is that of the whole sequence. (A recurrent layer's states move in the same call.)"""
    lens, p = [5, 33, 16], weights(3)
    gen = torch.Generator().manual_seed(4)
    total = [n + 12 for n in lens]
    xs = [draw(gen, n, HID).to(dtype).cuda() for n in total]
    s = Server(p, 4, 24, dtype)
    whole = [layer_ref(x.double().cpu(), {n: t.double().cpu() for n, t in s.p.items()}, s.cs.cpu()) for x in xs]
    # the parity bar; in bf16 the layer rounds four times on its way (2^-8 each, projections included)
    tol = TOL[dtype]
    for i, o in enumerate(s.prompts([x[:n] for x, n in zip(xs, lens)])):
        assert rel(o, whole[i][:lens[i]]) <= tol
    at = list(lens)
    for T in (1, 1, 1, 3):
        o = s.tokens(torch.stack([x[a:a + T] for x, a in zip(xs, at)]), [0, 1, 2])
        for i in range(3):
            assert rel(o[i], whole[i][at[i]:at[i] + T]) <= tol, (i, T)
            at[i] += T
    # request 3 is request 1 from here on, with a last page of its own
    states = torch.randn(4, 3, 7, device="cuda")
    last = (s.lens[1] - 1) // PAGE
    s.table[3], s.lens[3] = s.table[1].clone(), s.lens[1]
    s.table[3, last] = s.free.pop()
    pair = [torch.tensor([int(s.table[i, last])], **I32) for i in (1, 3)]
    g.pool_copy([s.kp, s.vp], *pair)
    g.pool_copy(states, torch.tensor([1], **I32), torch.tensor([3], **I32))
    assert torch.equal(states[3], states[1])
    x3 = draw(gen, 2, HID).to(dtype).cuda()
    full3 = layer_ref(torch.cat((xs[1][:at[1]], x3)).double().cpu(), {n: t.double().cpu() for n, t in s.p.items()},
                      s.cs.cpu())
    for t in range(2):
        o = s.tokens(torch.stack((xs[1][at[1] + t:at[1] + t + 1], x3[t:t + 1])), [1, 3])
        assert rel(o[0], whole[1][at[1] + t:at[1] + t + 1]) <= tol and rel(o[1], full3[at[1] + t:at[1] + t + 1]) <= tol
    # pages in use move to the front, those already there stay
    used = sorted(set(int(v) for v in s.table.flatten() if v >= 0))
    n = len(used)
    high, low = [u for u in used if u >= n], [i for i in range(n) if i not in used]
    g.pool_copy([s.kp, s.vp], torch.tensor(high, **I32), torch.tensor(low, **I32))
    moved = dict(zip(high, low))
    s.table = torch.tensor([[moved.get(int(v), int(v)) for v in row] for row in s.table], dtype=torch.int32)
    s.kp, s.vp = s.kp[:n].clone(), s.vp[:n].clone()
    s.free = []
    o = s.tokens(xs[0][at[0]:at[0] + 1][None], [0])
    assert rel(o[0], whole[0][at[0]:at[0] + 1]) <= tol


# ---- graphs ------------------------------------------------------------------------------


def decode_state(seed, N=3, pages=40):
    gen = torch.Generator().manual_seed(seed)
    bf = lambda *s: draw(gen, *s).to(BF16).cuda()  # noqa: E731
    return {"q": bf(N, 1, 4, 128), "k": bf(N, 1, 2, 128), "v": bf(N, 1, 2, 128), "kp": bf(pages, 2, 16, 128),
            "vp": bf(pages, 2, 16, 128), "cs": g.rotary_table(1024, 128, device="cuda"),
            "w": (1 + 0.1 * draw(gen, 128)).cuda(),
            "table": torch.randperm(pages, generator=gen)[:N * 13].view(N, 13).to(torch.int32).cuda(),
            "lens": torch.tensor([1, 100, 200], **I32), "pos": torch.zeros(N, 1, **I32), "slots": torch.zeros(N, 1, **I32)}


def decode_step(s, ws, o, lse):
    """What a captured decoding loop does: lengths, positions and places advance on the device."""
    s["pos"].copy_((s["lens"] - 1)[:, None])
    page = s["table"].gather(1, (s["pos"] // 16).long())
    s["slots"].copy_(page * 16 + s["pos"] % 16)
    q = g.qk_rotary_append(s["q"], s["k"], s["v"], s["cs"], s["pos"], s["kp"], s["vp"], s["slots"], s["w"], s["w"])
    g.paged_attention_step(q, s["kp"], s["vp"], s["table"], s["lens"], out=o, lse=lse, workspace=ws)
    s["lens"].add_(1)


def test_decoding_replays_in_graphs_that_share_a_workspace():
    """Two captured loops take turns on one workspace, with eager work between; every replay equals the
    eager calls, lengths growing from replay to replay (across pages, and across a cut)."""
    a, b = decode_state(1), decode_state(2)
    # long enough a table that sequences may be cut
    for s in (a, b):
        s["table"] = torch.cat((s["table"], torch.zeros(3, 30, **I32)), 1)
    need = g.paged_attention_step_workspace_bytes(3, 1, 4, 2, 128, 16, 43, BF16)
    assert need > 0
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    out = lambda: (torch.empty(3, 1, 4, 128, dtype=BF16, device="cuda"), torch.empty(3, 1, 4, device="cuda"))  # noqa: E731
    eager = [{n: t.clone() for n, t in s.items()} for s in (a, b)]
    keep = [{n: t.clone() for n, t in s.items()} for s in (a, b)]
    outs = [out(), out()]
    graphs = [capture(lambda s=s, o=o: decode_step(s, ws, *o)) for s, o in zip((a, b), outs)]
    for s, k in zip((a, b), keep):                        # as before the captures' own runs
        for n in s:
            s[n].copy_(k[n])
    for rep in range(5):
        for s, e, gr, (o, lse) in zip((a, b), eager, graphs, outs):
            wo, wl = out()
            decode_step(e, torch.empty(need, dtype=torch.uint8, device="cuda"), wo, wl)
            o.fill_(float("nan"))
            gr.replay()
            torch.cuda.synchronize()
            assert torch.equal(o, wo) and torch.equal(lse, wl), rep
            assert torch.equal(s["kp"], e["kp"]) and torch.equal(s["vp"], e["vp"])
        ws.fill_(255)                                     # what another call would leave


def test_gradients_and_copies_replay_in_a_graph():
    gen = torch.Generator().manual_seed(5)
    bf = lambda *s: draw(gen, *s).to(BF16).cuda()  # noqa: E731
    q, k, dq, dk = bf(1, 500, 4, 64), bf(1, 500, 2, 64), bf(1, 500, 4, 64), bf(1, 500, 2, 64)
    w, cs = (1 + 0.1 * draw(gen, 64)).cuda(), g.rotary_table(512, 64, device="cuda")
    pool, src, dst = torch.randn(6, 100, device="cuda"), torch.tensor([0, 1], **I32), torch.tensor([4, 3], **I32)
    ws = torch.empty(g.qk_rotary_bwd_workspace_bytes(1, 500, 64), dtype=torch.uint8, device="cuda")
    got = {}

    def run():
        got.update(g.qk_rotary_bwd(q, k, cs, dq, dk, q_weight=w, k_weight=w, workspace=ws))
        g.pool_copy(pool, src, dst)

    graph = capture(run)
    for rep in range(4):
        for t in (q, k, dq, dk):
            t.copy_(bf(*t.shape))
        pool.copy_(torch.randn(6, 100, device="cuda"))
        want = g.qk_rotary_bwd(q, k, cs, dq, dk, q_weight=w, k_weight=w)
        moved = pool.clone()
        moved[[4, 3]] = pool[[0, 1]]
        for t in got.values():
            t.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(got[n], want[n]) for n in want) and torch.equal(pool, moved)


# ---- streams and threads -----------------------------------------------------------------


def stream_inputs():
    gen = torch.Generator().manual_seed(6)
    bf = lambda *s: draw(gen, *s).to(BF16).cuda()  # noqa: E731
    v = {"q": bf(3, 5, 4, 128), "k": bf(3, 5, 2, 128), "v": bf(3, 5, 2, 128), "dq": bf(3, 5, 4, 128), "dk": bf(3, 5, 2, 128),
         "kp": bf(60, 2, 16, 128), "vp": bf(60, 2, 16, 128)}
    p = {"cs": g.rotary_table(64, 128, device="cuda"), "w": (1 + 0.1 * draw(gen, 128)).cuda(),
         "pos": torch.arange(15, **I32).view(3, 5), "slots": torch.randperm(960, generator=gen)[:15].view(3, 5).to(torch.int32).cuda(),
         "table": torch.randperm(60, generator=gen).view(3, 20).repeat(1, 2).to(torch.int32).cuda(),
         "lens": torch.tensor([300, 7, 600], **I32), "src": torch.tensor([5, 6], **I32), "dst": torch.tensor([9, 8], **I32)}
    return v, p


CALLS = {
    "qk_rotary_fwd": lambda v, p: g.qk_rotary_fwd(v["q"], v["k"], p["cs"], p["pos"], p["w"], p["w"]),
    "qk_rotary_bwd": lambda v, p: g.qk_rotary_bwd(v["q"], v["k"], p["cs"], v["dq"], v["dk"], positions=p["pos"],
                                                  q_weight=p["w"], k_weight=p["w"]),
    "qk_rotary_append": lambda v, p: (g.qk_rotary_append(v["q"], v["k"], v["v"], p["cs"], p["pos"], v["kp"], v["vp"], p["slots"],
                                                         p["w"], p["w"]), v["kp"], v["vp"]),
    "paged_attention_step": lambda v, p: g.paged_attention_step(v["q"], v["kp"], v["vp"], p["table"], p["lens"],
                                                                return_lse=True),
    "pool_copy": lambda v, p: (g.pool_copy([v["kp"], v["vp"]], p["src"], p["dst"]), v["kp"], v["vp"]),
}


@pytest.mark.parametrize("name", list(CALLS))
def test_side_stream_orders_producer_call_and_consumer(name):
    """The inputs hold NaN until a side stream, after milliseconds of other work, fills them; call and
    consumer follow on that stream. A launch anywhere else would read the NaN."""
    v, p = stream_inputs()
    good = {n: t.clone() for n, t in v.items()}
    want = [t.clone() for t in tensors(CALLS[name](v, p))]
    for t in v.values():
        t.fill_(float("nan"))
    busy = torch.zeros(1 << 26, device="cuda")
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        for _ in range(60):
            busy.add_(1.0)                      # 512 MB each
        for n, t in good.items():
            v[n].copy_(t)
        got = [t.clone() for t in tensors(CALLS[name](v, p))]
    side.synchronize()
    assert len(got) == len(want) and all(torch.equal(a, b) for a, b in zip(got, want))


def test_two_threads_at_once():
    """Calls of two threads on streams of their own give what each gives alone."""
    states = [stream_inputs() for _ in range(2)]
    names = ["qk_rotary_fwd", "qk_rotary_bwd", "paged_attention_step"]
    want = [[t.clone() for n in names for t in tensors(CALLS[n](*s))] for s in states]
    torch.cuda.synchronize()
    bad = []

    def work(i):
        stream = torch.cuda.Stream()
        with torch.cuda.stream(stream):
            for _ in range(20):
                got = [t for n in names for t in tensors(CALLS[n](*states[i]))]
                stream.synchronize()
                if not all(torch.equal(a, b) for a, b in zip(got, want[i])):
                    bad.append(i)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad
