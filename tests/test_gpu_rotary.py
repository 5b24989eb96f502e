"""Norms of queries and keys with the rotation by position against the 64-bit form: every head
size class and pairing, with and without weights, padding, slices, alignments, gradients, pages."""
import numpy as np
import pytest
import torch

import gated_delta_rule_gdn_amd as g
from attention_common import rotary_ref
from layer_common import check, f64

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16
EPS = 1e-5


def setup_module(module):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    g.lib()


def make(seed, B, T, hq, hk, d, rot, dtype, weights=(True, True), positions=64, pos=None, pad=0, shift=0):
    """Inputs on the GPU: slices of one projection whose columns begin at `shift`."""
    gen = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    proj = n(B, T, (hq + 2 * hk) * d + pad).to(dtype).cuda()
    at = [shift, shift + hq * d, shift + (hq + hk) * d, shift + (hq + 2 * hk) * d]
    v = {"q": proj[..., at[0]:at[1]].unflatten(-1, (hq, d)), "k": proj[..., at[1]:at[2]].unflatten(-1, (hk, d)),
         "v": proj[..., at[2]:at[3]].unflatten(-1, (hk, d))}
    v["qw"] = (1 + 0.2 * n(d)).cuda() if weights[0] else None
    v["kw"] = (1 + 0.2 * n(d)).cuda() if weights[1] else None
    v["cs"] = g.rotary_table(positions, rot, device="cuda")
    v["pos"] = torch.randint(0, positions, (B, T), generator=gen, dtype=torch.int32).cuda() if pos is None else pos
    v["dq"], v["dk"] = n(B, T, hq, d), n(B, T, hk, d)
    return v


def flat(t):
    return f64(t).reshape(-1, *t.shape[2:])


def check_fwd(v, inter, q, k, pos=None):
    pos = f64(v["pos"] if pos is None else pos).astype(int).ravel()
    for name, got, w in (("q", q, v["qw"]), ("k", k, v["kw"])):
        y, b = rotary_ref(flat(v[name]), f64(w), f64(v["cs"]), pos, inter, EPS)
        check(name, got.flatten(0, 1), y, b, got.dtype)


def run_bwd(v, inter, grad, **kw):
    return g.qk_rotary_bwd(v["q"], v["k"], v["cs"], v["dq"].to(grad).cuda(), v["dk"].to(grad).cuda(),
                           positions=v["pos"], q_weight=v["qw"], k_weight=v["kw"], interleaved=inter, eps=EPS, **kw)


def check_bwd(v, inter, grad, out):
    pos = f64(v["pos"]).astype(int).ravel()
    for n, w in (("q", v["qw"]), ("k", v["kw"])):
        dx, dxb, dw, dwb = rotary_ref(flat(v[n]), f64(w), f64(v["cs"]), pos, inter, EPS,
                                      dy=flat(v["d" + n].to(grad)))
        check("d" + n, out["d" + n].flatten(0, 1), dx, dxb, grad)
        assert (w is None) == (f"d{n}_weight" not in out)
        if w is not None:
            check(f"d{n}_weight", out[f"d{n}_weight"], dw, dwb)


# head sizes of every number of lanes, with whole accesses and without, in both pairings
SIZES = [(2, 2), (10, 4), (16, 16), (32, 16), (64, 64), (80, 20), (96, 48), (128, 128), (128, 64), (130, 130),
         (192, 64), (256, 64), (320, 320), (512, 512), (510, 254), (64, 0)]


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("d,rot", SIZES)
def test_sizes(d, rot, dtype, inter):
    v = make(d * 7 + rot, 2, 9, 5, 2, d, rot, dtype)
    q, k = g.qk_rotary_fwd(v["q"], v["k"], v["cs"], v["pos"], v["qw"], v["kw"], interleaved=inter, eps=EPS)
    check_fwd(v, inter, q, k)
    for grad in {dtype, F32}:
        check_bwd(v, inter, grad, run_bwd(v, inter, grad))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("weights", [(True, False), (False, True), (False, False)])
def test_without_weights(weights, dtype):
    v = make(3, 1, 13, 3, 3, 128, 96, dtype, weights)
    q, k = g.qk_rotary_fwd(v["q"], v["k"], v["cs"], v["pos"], v["qw"], v["kw"], eps=EPS)
    check_fwd(v, False, q, k)
    check_bwd(v, False, dtype, run_bwd(v, False, dtype))


@pytest.mark.parametrize("hq,hk", [(1, 1), (7, 1), (16, 2), (64, 8), (33, 33)])
def test_heads(hq, hk):
    v = make(hq, 1, 6, hq, hk, 128, 128, BF16)
    q, k = g.qk_rotary_fwd(v["q"], v["k"], v["cs"], v["pos"], v["qw"], v["kw"], eps=EPS)
    check_fwd(v, False, q, k)
    check_bwd(v, False, BF16, run_bwd(v, False, BF16))


def test_queries_alone():
    v = make(5, 2, 7, 4, 1, 64, 64, BF16)
    q, k = g.qk_rotary_fwd(v["q"], None, v["cs"], v["pos"], v["qw"], eps=EPS)
    assert k is None
    y, b = rotary_ref(flat(v["q"]), f64(v["qw"]), f64(v["cs"]), f64(v["pos"]).astype(int).ravel(), False, EPS)
    check("q", q.flatten(0, 1), y, b, BF16)
    out = g.qk_rotary_bwd(v["q"], None, v["cs"], v["dq"].to(BF16).cuda(), positions=v["pos"], q_weight=v["qw"],
                          eps=EPS)
    assert set(out) == {"dq", "dq_weight"}
    both = run_bwd(v, False, BF16)
    assert torch.equal(out["dq"], both["dq"]) and torch.equal(out["dq_weight"], both["dq_weight"])


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("pad,shift", [(0, 0), (16, 8), (3, 1), (7, 0)])
def test_slices_at_every_alignment(pad, shift, dtype):
    """Column slices whose stride or first column is odd give what the contiguous tensors give."""
    v = make(11, 2, 5, 4, 2, 64, 32, dtype, pad=pad, shift=shift)
    q, k = g.qk_rotary_fwd(v["q"], v["k"], v["cs"], v["pos"], v["qw"], v["kw"], eps=EPS)
    check_fwd(v, False, q, k)
    check_bwd(v, False, dtype, run_bwd(v, False, dtype))


def test_positions_and_padding():
    """Positions at the table's ends; outside of it a token is padding: zero rows, zero gradients,
    nothing for the weights, whatever its values."""
    pos = torch.tensor([[0, 63, 64, -1, 5, 2 ** 31 - 1, -2 ** 31]], dtype=torch.int32, device="cuda")
    for d, dtype in ((128, BF16), (70, F32)):
        v = make(6, 1, 7, 3, 2, d, 64, dtype, pos=pos)
        for n in ("q", "k"):
            v[n][:, [2, 3, 5, 6]] = float("nan")
        q, k = g.qk_rotary_fwd(v["q"], v["k"], v["cs"], pos, v["qw"], v["kw"], eps=EPS)
        out = run_bwd(v, False, dtype)
        for t in (q, k, out["dq"], out["dk"]):
            assert torch.equal(t[:, [2, 3, 5, 6]], torch.zeros_like(t[:, [2, 3, 5, 6]]))
        for n in ("q", "k"):
            v[n][:, [2, 3, 5, 6]] = 1.0           # for the reference, which multiplies by zero
        check_fwd(v, False, q, k)
        check_bwd(v, False, dtype, out)


def test_positions_default_to_places_in_each_sequence():
    v = make(7, 3, 20, 2, 1, 64, 64, F32)
    q, k = g.qk_rotary_fwd(v["q"], v["k"], v["cs"], None, v["qw"], v["kw"], eps=EPS)
    pos = torch.arange(20, dtype=torch.int32, device="cuda").expand(3, 20).contiguous()
    check_fwd(v, False, q, k, pos=pos)
    q2, k2 = g.qk_rotary_fwd(v["q"], v["k"], v["cs"], pos, v["qw"], v["kw"], eps=EPS)
    assert torch.equal(q, q2) and torch.equal(k, k2)


def test_far_positions_follow_the_table():
    """Angles come from the table, which is made in 64 bits: position 1,048,575 is as exact as 0."""
    P = 1 << 20
    pos = torch.tensor([[P - 1, P // 2 + 1, 77]], dtype=torch.int32, device="cuda")
    v = make(8, 1, 3, 2, 1, 64, 64, F32, positions=P, pos=pos)
    q, k = g.qk_rotary_fwd(v["q"], v["k"], v["cs"], pos, v["qw"], v["kw"], eps=EPS)
    check_fwd(v, False, q, k)
    i = np.arange(32)
    angle = f64(pos).ravel()[:, None] * 10000.0 ** (-2 * i / 64)
    table = f64(v["cs"])[f64(pos).astype(int).ravel()]
    assert np.abs(table - np.concatenate([np.cos(angle), np.sin(angle)], 1)).max() < 2.0 ** -24 + 1e-9


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_in_place(dtype):
    for d in (128, 66):
        v = make(9, 2, 11, 4, 2, d, d, dtype)
        q, k = v["q"].contiguous(), v["k"].contiguous()
        want = g.qk_rotary_fwd(q, k, v["cs"], v["pos"], v["qw"], v["kw"], eps=EPS)
        got = g.qk_rotary_fwd(q, k, v["cs"], v["pos"], v["qw"], v["kw"], eps=EPS, q_out=q, k_out=k)
        assert got[0] is q and all(torch.equal(a, b) for a, b in zip(got, want))


def test_nothing_to_do():
    v = make(10, 1, 4, 2, 1, 64, 64, F32)
    q, k = g.qk_rotary_fwd(v["q"][:, :0], v["k"][:, :0], v["cs"], v["pos"][:, :0].contiguous(), v["qw"], v["kw"])
    assert q.shape == (1, 0, 2, 64)
    out = g.qk_rotary_bwd(v["q"][:, :0], v["k"][:, :0], v["cs"], q, k, positions=v["pos"][:, :0].contiguous(),
                          q_weight=v["qw"], k_weight=v["kw"])
    assert not out["dq_weight"].any() and not out["dk_weight"].any()


@pytest.mark.parametrize("T", [1, 3, 4, 5, 4096, 4097, 9001])
def test_weight_gradients_over_many_tokens(T):
    """Fewer tokens than waves, whole and ragged sets of them, and several per wave."""
    v = make(T, 1, T, 2, 1, 16, 8, F32)
    check_bwd(v, False, F32, run_bwd(v, False, F32))


@pytest.mark.parametrize("inter", [False, True])
def test_gradients_against_differences(inter):
    """The loss moves by the gradient along random directions (central differences in fp32 outputs
    of fp32 inputs: 1e-2 steps, third-order terms of order 1e-4, rounding 1e-7 / 1e-2 per value)."""
    v = make(12, 1, 5, 2, 2, 24, 12, F32)
    q, k = v["q"].contiguous(), v["k"].contiguous()
    out = run_bwd(v, inter, F32)
    gen = torch.Generator().manual_seed(13)
    dq, dk = v["dq"].double(), v["dk"].double()

    def loss(q, k, qw, kw):
        a, b = g.qk_rotary_fwd(q, k, v["cs"], v["pos"], qw, kw, interleaved=inter, eps=EPS)
        return float((a.double().cpu() * dq).sum() + (b.double().cpu() * dk).sum())

    args = [q, k, v["qw"], v["kw"]]
    for i, name in enumerate(("dq", "dk", "dq_weight", "dk_weight")):
        e = torch.randn(args[i].shape, generator=gen).cuda()
        e = e / e.norm()
        up = [t + 1e-2 * e if j == i else t for j, t in enumerate(args)]
        down = [t - 1e-2 * e if j == i else t for j, t in enumerate(args)]
        slope = (loss(*up) - loss(*down)) / 2e-2
        want = float((out[name].double() * e.double()).sum())
        scale = float(out[name].double().norm())
        print(f"[rotary] {name}: {slope:.6f} against {want:.6f} (norm {scale:.3f})", flush=True)
        assert abs(slope - want) < 2e-3 * scale


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("page,d,hk", [(1, 64, 1), (16, 128, 2), (48, 70, 3), (64, 256, 2)])
def test_append_to_pages(page, d, hk, dtype):
    T = 37
    v = make(page, 1, T, 4 * hk, hk, d, d // 2 & ~1, dtype)
    gen = torch.Generator().manual_seed(page)
    pages = -(-T // page) + 2
    kp = torch.randn(pages, hk, page, d, generator=gen).to(dtype).cuda()
    vp = torch.randn(pages, hk, page, d, generator=gen).to(dtype).cuda()
    slots = torch.randperm(pages * page, generator=gen)[:T].to(torch.int32)
    slots[3], slots[5], slots[9] = -1, pages * page, -2 ** 31
    v["pos"][0, 11] = -1                                        # padding: not put anywhere
    want = [kp.clone(), vp.clone()]
    q, k = g.qk_rotary_fwd(v["q"], v["k"], v["cs"], v["pos"], v["qw"], v["kw"], eps=EPS)
    for t, s in enumerate(slots.tolist()):
        if 0 <= s < pages * page and t != 11:
            want[0][s // page, :, s % page] = k[0, t]
            want[1][s // page, :, s % page] = v["v"][0, t]
    got = g.qk_rotary_append(v["q"], v["k"], v["v"], v["cs"], v["pos"], kp, vp, slots[None].cuda(), v["qw"], v["kw"],
                             eps=EPS)
    assert torch.equal(got, q) and torch.equal(kp, want[0]) and torch.equal(vp, want[1])


def test_append_in_place_of_dense_prompts():
    """Three prompts of 11 tokens, q in place; keys and values of a padded batch's end are left out."""
    v = make(17, 3, 11, 4, 2, 64, 64, BF16)
    q, k = v["q"].contiguous(), v["k"].contiguous()
    kp = torch.zeros(9, 2, 8, 64, dtype=BF16, device="cuda")
    vp = torch.zeros_like(kp)
    slots = torch.arange(33, dtype=torch.int32).view(3, 11)
    slots[1, 8:] = -1
    want_q, want_k = g.qk_rotary_fwd(q, k, v["cs"], v["pos"], v["qw"], v["kw"], eps=EPS)
    got = g.qk_rotary_append(q, k, v["v"], v["cs"], v["pos"], kp, vp, slots.cuda(), v["qw"], v["kw"], eps=EPS, q_out=q)
    assert got is q and torch.equal(q, want_q)
    for pool, src in ((kp, want_k), (vp, v["v"])):
        rows = pool.transpose(1, 2).flatten(0, 1)
        for b in range(3):
            for t in range(11):
                s = int(slots[b, t])
                if s >= 0:
                    assert torch.equal(rows[s], src[b, t])
        assert not rows[33:].any() and not rows[19:22].any()


def test_append_far_into_a_large_pool():
    """Places whose elements lie beyond 2^32."""
    pages, hk, page, d = 1100, 16, 1024, 256          # 4.6e9 values of bf16, 9.2 GB
    kp = torch.zeros(pages, hk, page, d, dtype=BF16, device="cuda")
    vp = torch.zeros(pages, hk, page, d, dtype=BF16, device="cuda")
    v = make(14, 3, 1, 16, hk, d, 64, BF16)
    slots = torch.tensor([[pages * page - 1], [(pages - 1) * page], [5]], dtype=torch.int32, device="cuda")
    q, k = g.qk_rotary_fwd(v["q"], v["k"], v["cs"], v["pos"], v["qw"], v["kw"], eps=EPS)
    g.qk_rotary_append(v["q"], v["k"], v["v"], v["cs"], v["pos"], kp, vp, slots, v["qw"], v["kw"], eps=EPS)
    for i, s in enumerate(slots.flatten().tolist()):
        assert torch.equal(kp[s // page, :, s % page], k[i, 0]) and torch.equal(vp[s // page, :, s % page], v["v"][i, 0])
    for pool, given in ((kp, k), (vp, v["v"])):
        assert int(torch.count_nonzero(pool.view(torch.int16))) == int(torch.count_nonzero(given.contiguous().view(torch.int16)))


def test_same_bits_at_every_call():
    v = make(15, 1, 2000, 8, 2, 128, 128, BF16)
    a, b = run_bwd(v, False, BF16), run_bwd(v, False, BF16)
    assert all(torch.equal(a[n], b[n]) for n in a)


def test_refusals():
    v = make(16, 1, 4, 2, 1, 64, 64, BF16)
    with pytest.raises(TypeError):
        g.qk_rotary_fwd(v["q"], v["k"].float(), v["cs"], v["pos"])
    with pytest.raises(ValueError):
        g.qk_rotary_fwd(v["q"], v["k"], v["cs"], v["pos"][:, :3])
    with pytest.raises(g.GDN2Error):
        g.qk_rotary_fwd(v["q"], v["k"], g.rotary_table(8, 66, device="cuda"), v["pos"])
    with pytest.raises(ValueError):
        g.qk_rotary_fwd(v["q"].transpose(1, 2), None, v["cs"])
    with pytest.raises(g.GDN2Error):
        g.qk_rotary_fwd(v["q"].contiguous()[..., :63].contiguous(), None, v["cs"], v["pos"])
    with pytest.raises(ValueError):
        g.qk_rotary_bwd(v["q"], v["k"], v["cs"], v["dq"].to(BF16).cuda())
    q = v["q"].contiguous()
    with pytest.raises(g.GDN2Error):
        g.qk_rotary_bwd(q, None, v["cs"], q.clone(), q_weight=v["qw"], workspace=torch.empty(16, dtype=torch.uint8,
                                                                                             device="cuda"))
