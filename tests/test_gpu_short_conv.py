"""The short convolution over prompts, its gradients and its single-token form, against a plain
64-bit form token by token."""
import numpy as np
import pytest
import torch

import gated_delta_rule_gdn_amd as g
from layer_common import check, conv_ref, f64, offsets

pytestmark = pytest.mark.gpu


def setup_module(module):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    g.lib()


def draw(seed, *shape, dtype=torch.float32, std=1.0):
    gen = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=gen) * std).to(dtype)


def make(lens, C, W, dtype, bias, state, seed, wide=0):
    """Host inputs of one packed call; x is a column slice of a tensor `wide` columns wider."""
    T = int(sum(lens))
    x = draw(seed, 1, T, C + wide, dtype=dtype)
    return {"x": x, "weight": draw(seed + 1, C, W, std=W ** -0.5),
            "bias": draw(seed + 2, C, std=0.3) if bias else None,
            "state0": draw(seed + 3, len(lens), W - 1, C) if state else None}


def gpu(t):
    return None if t is None else t.cuda()


def cu_of(lens):
    return torch.tensor(offsets(lens), dtype=torch.int32, device="cuda")


LENS = [
    [1], [2], [3], [4], [5], [8], [63], [64], [65],            # one sequence
    [0, 1, 0, 0, 2, 3, 1, 1, 0],                                # shorter than the taps, empty ones
    [7, 130, 1, 64, 0, 29],
    [1] * 70,                                                   # more sequences than lanes
    [0] * 66 + [5] + [0] * 70 + [2],
    [0, 0],                                                     # nothing at all
]


@pytest.mark.parametrize("W", [2, 3, 4])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("lens", LENS, ids=lambda v: f"n{len(v)}t{sum(v)}")
def test_packed_forward_and_backward(lens, dtype, W):
    """Lengths around the taps, the batches of a lane and the tiles; vector and odd widths."""
    for C, wide in ((24, 8), (7, 0), (9, 4)):
        h = make(lens, C, W, dtype, bias=True, state=True, seed=W * 100 + len(lens) + C, wide=wide)
        T = int(sum(lens))
        x = h["x"].cuda()[..., :C]
        dy, dst = draw(5, 1, T, C, dtype=dtype), draw(6, len(lens), W - 1, C)
        r = conv_ref(f64(h["x"][0, :, :C]), f64(h["weight"]), f64(h["bias"]), f64(h["state0"]), lens,
                     True, f64(dy[0]), f64(dst))
        args = dict(bias=gpu(h["bias"]), state0=gpu(h["state0"]), cu_seqlens=cu_of(lens), silu=True)
        y, st = g.short_conv_fwd(x, h["weight"].cuda(), **args)
        d = g.short_conv_bwd(x, h["weight"].cuda(), dy.cuda(), dstate_T=dst.cuda(), **args)
        torch.cuda.synchronize()
        check("y", y[0], r["y"], r["y_b"], dtype)
        assert np.array_equal(f64(st), r["state_T"])
        check("dx", d["dx"][0], r["dx"], r["dx_b"], dtype)
        for n in ("dweight", "dbias", "dstate0"):
            check(n, d[n], r[n], r[n + "_b"])


@pytest.mark.parametrize("silu,bias,state", [(False, False, False), (True, False, True),
                                             (False, True, True), (True, True, False)])
@pytest.mark.parametrize("B,T,C", [(1, 1, 64), (3, 50, 520), (2, 257, 40), (5, 3, 1024)])
def test_dense_options_and_fp32_gradients(B, T, C, silu, bias, state):
    W, dtype = 4, torch.bfloat16
    x = draw(1, B, T, C, dtype=dtype)
    w = draw(2, C, W, std=0.5)
    b = draw(3, C) if bias else None
    s0 = draw(4, B, W - 1, C) if state else None
    dy = draw(5, B, T, C)
    flat = lambda t: f64(t).reshape(B * T, C)  # noqa: E731
    r = conv_ref(flat(x), f64(w), f64(b), f64(s0), [T] * B, silu, flat(dy))
    y, st = g.short_conv_fwd(x.cuda(), w.cuda(), bias=gpu(b), state0=gpu(s0), silu=silu)
    d = g.short_conv_bwd(x.cuda(), w.cuda(), dy.cuda(), bias=gpu(b), state0=gpu(s0), silu=silu)
    torch.cuda.synchronize()
    assert set(d) == {"dx", "dweight"} | ({"dbias"} if bias else set()) | ({"dstate0"} if state else set())
    assert d["dx"].dtype == torch.float32
    check("y", flat(y), r["y"], r["y_b"], dtype)
    assert np.array_equal(f64(st), r["state_T"])
    check("dx", flat(d["dx"]), r["dx"], r["dx_b"])
    for n in set(d) - {"dx"}:
        check(n, d[n], r[n], r[n + "_b"])


def test_gradients_against_differences():
    """dL/dx, dL/dweight and dL/dstate0 of L = sum(y dy) + sum(state_T dstate_T) along random
    directions, against central differences of the fp32 forward."""
    lens, C, W = [5, 0, 1, 17], 12, 4
    h = make(lens, C, W, torch.float32, True, True, 40)
    T = sum(lens)
    cu = cu_of(lens)
    dy, dst = draw(41, 1, T, C).cuda(), draw(42, len(lens), W - 1, C).cuda()
    p = {n: gpu(t) for n, t in h.items()}

    def loss(q):
        y, st = g.short_conv_fwd(q["x"], q["weight"], bias=q["bias"], state0=q["state0"],
                                 cu_seqlens=cu, silu=True)
        return float((y.double() * dy.double()).sum() + (st.double() * dst.double()).sum())

    d = g.short_conv_bwd(p["x"], p["weight"], dy, bias=p["bias"], state0=p["state0"],
                         cu_seqlens=cu, silu=True, dstate_T=dst)
    eps = 2.0 ** -7
    for i, n in enumerate(("x", "weight", "bias", "state0")):
        v = draw(50 + i, *p[n].shape).cuda()
        hi, lo = dict(p), dict(p)
        hi[n], lo[n] = p[n] + eps * v, p[n] - eps * v
        num = (loss(hi) - loss(lo)) / (2 * eps)
        want = float((d["d" + n].double() * v.double()).sum())
        # third derivative of silu at most 1, times the direction's size, eps^2 / 6; and the
        # rounding of about 600 fp32 outputs of size 1, divided by eps
        assert abs(num - want) <= 2e-2 * max(1.0, abs(want)), (n, num, want)


def test_rows_behind_the_last_sequence_are_left_alone():
    lens, C, W, T = [5, 9], 32, 4, 200
    x = draw(1, 1, T, C, dtype=torch.bfloat16).cuda()
    x[:, 14:] = float("nan")
    w = draw(2, C, W).cuda()
    cu = cu_of(lens)
    out = torch.full((1, T, C), 7.0, dtype=torch.bfloat16, device="cuda")
    y, st = g.short_conv_fwd(x, w, cu_seqlens=cu, out=out)
    d = g.short_conv_bwd(x, w, torch.ones_like(x), cu_seqlens=cu)
    torch.cuda.synchronize()
    assert torch.all(out[:, 14:] == 7.0) and torch.isfinite(out[:, :14]).all()
    assert torch.isfinite(st).all() and torch.isfinite(d["dweight"]).all()
    assert torch.isfinite(d["dx"][:, :14]).all()


@pytest.mark.parametrize("W", [2, 3, 4])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("N,T,C", [(1, 1, 8), (5, 1, 1030), (3, 6, 129), (70, 2, 64)])
def test_step_continues_a_prompt(N, T, C, dtype, W):
    """Steps against slots in any order, a padding entry among them; other slots untouched."""
    slots = N + 3
    pool = draw(1, slots, W - 1, C)
    x, w, b = draw(2, N, T, C, dtype=dtype), draw(3, C, W), draw(4, C)
    idx = torch.randperm(slots, generator=torch.Generator().manual_seed(9))[:N].to(torch.int32)
    if N > 1:
        idx[1] = -1 if W % 2 else slots
    P = pool.cuda()
    y = g.short_conv_step(x.cuda(), w.cuda(), P, bias=b.cuda(), state_idx=idx.cuda(), silu=True)
    torch.cuda.synchronize()
    want = f64(pool)
    for n, s in enumerate(idx.tolist()):
        if not 0 <= s < slots:
            assert torch.all(y[n] == 0)
            continue
        r = conv_ref(f64(x[n]), f64(w), f64(b), f64(pool[s])[None], [T], True)
        check("y", y[n], r["y"], r["y_b"], dtype)
        want[s] = r["state_T"][0]
    assert np.array_equal(f64(P), want)


def test_prompt_then_tokens_equals_one_prompt():
    """A prompt cut anywhere, its rest fed as a prompt or token by token: the same bits (the
    same sum in the same order)."""
    C, W, T = 72, 4, 40
    x, w = draw(1, 1, T, C, dtype=torch.bfloat16).cuda(), draw(2, C, W).cuda()
    y, st = g.short_conv_fwd(x, w, silu=True)
    for cut in (1, 2, 3, 17, 39):
        y0, s0 = g.short_conv_fwd(x[:, :cut].contiguous(), w, silu=True)
        y1, s1 = g.short_conv_fwd(x[:, cut:].contiguous(), w, state0=s0, silu=True)
        pool = s0.clone()
        y2 = torch.cat([g.short_conv_step(x[:, t:t + 1].contiguous(), w, pool, silu=True)
                        for t in range(cut, T)], 1)
        torch.cuda.synchronize()
        assert torch.equal(torch.cat((y0, y1), 1), y) and torch.equal(s1, st)
        assert torch.equal(y2, y[:, cut:]) and torch.equal(pool, st)


def test_same_convolution_as_the_fused_decode():
    """recurrent_fwd's fused convolution of q, k and v and the separate calls give the same
    o and the same conv state (bf16 inputs; the separate calls round q, k and v to bf16 once)."""
    N, T, Hk, Hv, d = 3, 2, 2, 4, 64
    C = 2 * Hk * d + Hv * d
    q, k = (draw(i, N, T, Hk, d, dtype=torch.bfloat16).cuda() for i in (1, 2))
    v = draw(3, N, T, Hv, d, dtype=torch.bfloat16).cuda()
    la = -draw(4, N, T, Hv, d).abs().to(torch.bfloat16).cuda()
    b, w = (torch.sigmoid(draw(i, N, T, Hv, d)).to(torch.bfloat16).cuda() for i in (5, 6))
    cw, cs = draw(7, C, 4, std=0.5).cuda(), draw(8, N, 3, C).cuda()
    S = draw(9, N, Hv, d, d, std=0.1).cuda()
    S1, S2, cs1, cs2 = S.clone(), S.clone(), cs.clone(), cs.clone()
    o1 = g.recurrent_fwd(q, k, v, la, b, w, S1, conv_weight=cw, conv_state=cs1, conv_silu=True,
                         qk_l2norm=True)
    x = torch.cat([t.reshape(N, T, -1) for t in (q, k, v)], -1)
    y = g.short_conv_step(x, cw, cs2, silu=True)
    q2, k2, v2 = y.split([Hk * d, Hk * d, Hv * d], -1)
    o2 = g.recurrent_fwd(q2.reshape(N, T, Hk, d).contiguous(), k2.reshape(N, T, Hk, d).contiguous(),
                         v2.reshape(N, T, Hv, d).contiguous(), la, b, w, S2, qk_l2norm=True)
    torch.cuda.synchronize()
    assert torch.equal(cs1, cs2)
    # q, k and v each rounded once more: 2^-8 each, and o's own rounding on both sides
    for a, c in ((o1, o2), (S1, S2)):
        assert float((a.double() - c.double()).norm() / a.double().norm()) <= 5 * 2.0 ** -8


def test_large_offsets():
    """A token stride that puts the last rows past 2^31 elements."""
    C, W, T, step = 8, 4, 1100, 1 << 21
    buf = torch.empty(T * step, dtype=torch.bfloat16, device="cuda")
    x = buf.as_strided((1, T, C), (T * step, step, 1))
    x.copy_(draw(1, 1, T, C, dtype=torch.bfloat16).cuda())
    w = draw(2, C, W).cuda()
    y, st = g.short_conv_fwd(x, w, silu=True)
    y2, st2 = g.short_conv_fwd(x.contiguous(), w, silu=True)
    d = g.short_conv_bwd(x, w, y, silu=True)
    d2 = g.short_conv_bwd(x.contiguous(), w, y, silu=True)
    torch.cuda.synchronize()
    assert torch.equal(y, y2) and torch.equal(st, st2)
    assert torch.equal(d["dx"], d2["dx"]) and torch.equal(d["dweight"], d2["dweight"])


def test_refusals():
    x, w = torch.zeros(1, 4, 8, device="cuda"), torch.zeros(8, 4, device="cuda")
    st = torch.zeros(1, 3, 8, device="cuda")
    with pytest.raises(ValueError):
        g.short_conv_fwd(x.cpu(), w)
    with pytest.raises(TypeError):
        g.short_conv_fwd(x.half(), w)
    with pytest.raises(ValueError):
        g.short_conv_fwd(x.transpose(1, 2), w)
    with pytest.raises(ValueError):
        g.short_conv_fwd(x[:, :1].expand(1, 4, 8), w)         # tokens overlap
    with pytest.raises(ValueError):
        g.short_conv_fwd(x, w[:4])
    with pytest.raises(g.GDN2Error):
        g.short_conv_fwd(x, torch.zeros(8, 5, device="cuda"))  # five taps
    with pytest.raises(g.GDN2Error):
        g.short_conv_fwd(x, w, state0=st, final_state=st)      # in place
    with pytest.raises(ValueError):
        g.short_conv_fwd(x, w, state0=torch.zeros(2, 3, 8, device="cuda"))
    with pytest.raises(TypeError):
        g.short_conv_fwd(x, w, cu_seqlens=torch.tensor([0, 4], device="cuda"))
    with pytest.raises(ValueError):
        g.short_conv_fwd(x.expand(2, 4, 8).contiguous(), w,
                         cu_seqlens=torch.tensor([0, 4], dtype=torch.int32, device="cuda"))
    with pytest.raises(TypeError):
        g.short_conv_bwd(x, w, x.to(torch.bfloat16))           # fp32 inputs, bf16 gradients
    with pytest.raises(g.GDN2Error):
        g.short_conv_bwd(x, w, x, workspace=torch.empty(256, dtype=torch.uint8, device="cuda")[:8])
    with pytest.raises(g.GDN2Error):
        g.short_conv_step(x.expand(2, 4, 8).contiguous(), w, st)   # two sequences, one slot
    with pytest.raises(ValueError):
        g.short_conv_fwd(x, w, out=torch.zeros(1, 4, 9, device="cuda"))


@pytest.mark.parametrize("name", ["x", "dy", "state0", "dstate_T"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_values_that_are_not_finite_stay_in_their_sequence(name, bad):
    """The middle one of three sequences, which meet inside tiles, holds NaN or infinities: the
    bits of the others' outputs and gradients do not change."""
    gen = torch.Generator().manual_seed(31)
    n = lambda *s: torch.randn(*s, generator=gen).cuda()  # noqa: E731
    w, b = n(20, 4), n(20)
    d = {"x": n(1, 90, 20), "dy": n(1, 90, 20), "state0": n(3, 3, 20), "dstate_T": n(3, 3, 20)}
    cu = torch.tensor([0, 41, 50, 90], dtype=torch.int32, device="cuda")

    def run():
        y, s = g.short_conv_fwd(d["x"], w, b, d["state0"], cu, silu=True)
        o = g.short_conv_bwd(d["x"], w, d["dy"], b, d["state0"], cu, silu=True, dstate_T=d["dstate_T"])
        return y, o["dx"], s, o["dstate0"]

    clean = run()
    if name in ("x", "dy"):
        d[name][:, 41:50] = bad
    else:
        d[name][1] = bad
    got = run()
    torch.cuda.synchronize()
    for a, c in zip(got[:2], clean[:2]):
        assert torch.equal(a[:, :41], c[:, :41]) and torch.equal(a[:, 50:], c[:, 50:])
    for a, c in zip(got[2:], clean[2:]):
        assert torch.equal(a[[0, 2]], c[[0, 2]])
    assert not all(torch.equal(a, c) for a, c in zip(got, clean))
