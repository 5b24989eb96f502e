"""The selective scan over prompts and of single tokens, against a plain 64-bit form token by
token."""
import numpy as np
import pytest
import torch

import gated_delta_rule_gdn_amd as g
from layer_common import HALF_STEP, check, f64, offsets, scan_ref

pytestmark = pytest.mark.gpu


def setup_module(module):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    g.lib()


class Draw:
    def __init__(self, seed):
        self.gen = torch.Generator().manual_seed(seed)

    def normal(self, *shape, dtype=torch.float32, std=1.0):
        return (torch.randn(*shape, generator=self.gen) * std).to(dtype)


def make(lead, ch, M, G, N, dtype, seed, gate=True, D=True, bias=True, state=True, wide=0):
    """Host inputs; x, dt, gate, B and C are column slices where wide > 0. Rates reach from zero
    to d_state, steps from 0.001 to about 1, so that some states live over many tiles."""
    d = Draw(seed)
    sl = lambda t, n: t[..., wide:wide + n]  # noqa: E731
    bc = d.normal(*lead, wide + 2 * G * M, dtype=dtype)
    h = {"x": sl(d.normal(*lead, ch + wide, dtype=dtype), ch),
         "dt": sl(d.normal(*lead, ch + wide, dtype=dtype, std=0.7), ch),
         "B": bc[..., wide:wide + G * M].unflatten(-1, (G, M)),
         "C": bc[..., wide + G * M:].unflatten(-1, (G, M)),
         "gate": sl(d.normal(*lead, ch + wide, dtype=dtype), ch) if gate else None,
         "A": -torch.arange(M) * torch.exp(d.normal(ch, M, std=0.2)),
         "D": d.normal(ch) if D else None,
         "dt_bias": torch.log(torch.expm1(torch.exp(torch.rand(ch, generator=d.gen) * 6 - 6.9)))
         if bias else None,
         "S0": d.normal(N, ch, M) if state else None}
    return h


def gpu(h):
    return {n: None if t is None else t.cuda() for n, t in h.items()}


def on_gpu_sliced(h, wide):
    """The inputs on the GPU, slices still slices of a wider tensor."""
    out = {}
    for n, t in h.items():
        if t is None:
            out[n] = None
        elif wide and n in ("x", "dt", "gate", "B", "C"):
            flat = t.reshape(*t.shape[:2], -1)
            buf = torch.zeros(*flat.shape[:2], flat.shape[2] + wide, dtype=t.dtype, device="cuda")
            buf[..., wide:] = flat.cuda()
            v = buf[..., wide:]
            out[n] = v.unflatten(-1, t.shape[2:]) if t.dim() == 4 else v
        else:
            out[n] = t.contiguous().cuda()
    return out


def ref(h, lens, softplus=True):
    T = int(sum(lens))
    v = {n: None if t is None else f64(t) for n, t in h.items()}
    fl = lambda a: None if a is None else a.reshape(T, *a.shape[2:])  # noqa: E731
    return scan_ref(fl(v["x"]), fl(v["dt"]), v["A"], fl(v["B"]), fl(v["C"]), v["D"], fl(v["gate"]),
                    v["dt_bias"], softplus, v["S0"], lens)


def cu_of(lens):
    return torch.tensor(offsets(lens), dtype=torch.int32, device="cuda")


def call(d, softplus=True, **kw):
    return g.selective_scan_fwd(d["x"], d["dt"], d["A"], d["B"], d["C"], D=d["D"], gate=d["gate"],
                                dt_bias=d["dt_bias"], dt_softplus=softplus, S0=d["S0"], **kw)


LENS = [[1], [7], [8], [9], [16], [17], [33], [130], [0], [0, 1, 0, 0, 2, 40, 1, 0],
        [15, 1, 16, 1, 33, 0, 20], [1] * 70, [0] * 66 + [19] + [0] * 3 + [2]]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("lens", LENS, ids=lambda v: f"n{len(v)}t{sum(v)}")
def test_packed_lengths(lens, dtype):
    """Lengths around the batches and tiles; sequences that begin and end anywhere in a tile."""
    h = make((1, int(sum(lens))), 70, 16, 1, len(lens), dtype, seed=len(lens) + sum(lens))
    o, S = call(on_gpu_sliced(h, 0), cu_seqlens=cu_of(lens))
    torch.cuda.synchronize()
    r = ref(h, lens)
    check("o", o[0], r["o"], r["o_b"], dtype)
    check("S_T", S, r["S_T"], r["S_T_b"])


@pytest.mark.parametrize("M", [1, 3, 8, 9, 16, 17, 32, 33, 64, 65, 128])
@pytest.mark.parametrize("ch,G", [(1, 1), (66, 2), (300, 3)])
def test_state_sizes_channels_and_groups(ch, G, M):
    lens = [37, 5]
    h = make((1, 42), ch, M, G, 2, torch.bfloat16, seed=ch + M)
    o, S = call(on_gpu_sliced(h, 3), cu_seqlens=cu_of(lens))
    torch.cuda.synchronize()
    r = ref(h, lens)
    check("o", o[0], r["o"], r["o_b"], torch.bfloat16)
    check("S_T", S, r["S_T"], r["S_T_b"])


@pytest.mark.parametrize("gate,D,bias,state,softplus", [
    (False, False, False, False, True), (True, False, True, False, True),
    (False, True, False, True, False), (True, True, True, True, True)])
@pytest.mark.parametrize("B,T,ch", [(1, 1, 8), (3, 40, 65), (2, 200, 260), (260, 9, 16), (4, 0, 8)])
def test_dense_options(B, T, ch, gate, D, bias, state, softplus):
    """Whole sequences per tile (260 short ones), and cut ones."""
    h = make((B, T), ch, 16, 1, B, torch.float32, seed=B + T, gate=gate, D=D, bias=bias, state=state)
    if not softplus:
        h["dt"] = h["dt"].abs() * 0.1           # a step given as it is
        h["dt_bias"] = None if h["dt_bias"] is None else h["dt_bias"].abs() * 0.01
    o, S = call(gpu(h), softplus)
    torch.cuda.synchronize()
    r = ref(h, [T] * B, softplus)
    check("o", o.reshape(B * T, ch), r["o"], r["o_b"])
    check("S_T", S, r["S_T"], r["S_T_b"])


def test_long_sequence_of_slow_states():
    """2,500 tokens over 157 tiles with rates near zero: every tile's state reaches the end."""
    h = make((1, 2500), 40, 4, 1, 1, torch.float32, seed=3)
    h["A"] = -torch.rand(40, 4) * 0.02
    o, S = call(gpu(h))
    torch.cuda.synchronize()
    r = ref(h, [2500])
    check("o", o[0], r["o"], r["o_b"])
    check("S_T", S, r["S_T"], r["S_T_b"])


@pytest.mark.parametrize("low", [float("-inf"), -3e38, -1e4])
def test_masked_steps_leave_the_state(low):
    """Steps whose dt is -inf or the lowest value have dt = 0: the state passes them unchanged,
    whatever B holds there; a sequence of nothing else returns S0's bits."""
    h = make((1, 60), 20, 16, 1, 2, torch.float32, seed=8)
    h["dt"][:, 10:35] = low
    h["dt"][:, 40:] = low
    o, S = call(gpu(h), cu_seqlens=cu_of([40, 20]))
    torch.cuda.synchronize()
    v = {**h, "dt": h["dt"].clamp(min=-300.0)}       # softplus is below 1e-130 there
    r = ref(v, [40, 20])
    check("o", o[0], r["o"], r["o_b"])
    check("S_T", S, r["S_T"], r["S_T_b"])
    assert torch.equal(S[1].cpu(), h["S0"][1])


def test_nan_stays_in_its_sequence_and_channel():
    h = make((1, 90), 70, 16, 1, 3, torch.bfloat16, seed=9)
    d = gpu(h)
    o0, S0 = call(d, cu_seqlens=cu_of([30, 40, 20]))
    d["x"][0, 45, 5] = float("nan")
    o, S = call(d, cu_seqlens=cu_of([30, 40, 20]))
    torch.cuda.synchronize()
    hit = torch.zeros(90, 70, dtype=torch.bool, device="cuda")
    hit[45:70, 5] = True
    assert torch.isnan(o[0][hit]).all() and torch.equal(o[0][~hit], o0[0][~hit])
    assert torch.isnan(S[1, 5]).any() and torch.equal(S[[0, 2]], S0[[0, 2]])


def test_rows_behind_the_last_sequence_are_left_alone():
    h = make((1, 120), 20, 16, 1, 2, torch.bfloat16, seed=10)
    d = gpu(h)
    for n in ("x", "dt", "B", "C", "gate"):
        d[n][:, 50:] = float("nan")
    out = torch.full((1, 120, 20), 7.0, dtype=torch.bfloat16, device="cuda")
    o, S = call(d, cu_seqlens=cu_of([20, 30]), out=out)
    torch.cuda.synchronize()
    assert torch.all(out[:, 50:] == 7.0) and torch.isfinite(out[:, :50]).all()
    assert torch.isfinite(S).all()


def test_large_offsets():
    """Token strides that put the last rows past 2^31 elements."""
    T, ch, M, step = 1100, 8, 16, 1 << 21
    h = make((1, T), ch, M, 1, 1, torch.bfloat16, seed=11)
    d = gpu(h)
    buf = torch.empty(T * step, dtype=torch.bfloat16, device="cuda")
    e, at = dict(d), 0
    for n in ("x", "dt", "gate", "B", "C"):
        w = d[n][0, 0].numel()
        v = buf[at:].as_strided((1, T, w), (T * step, step, 1))
        v.copy_(d[n].reshape(1, T, w))
        e[n] = v.unflatten(-1, (1, M)) if n in "BC" else v
        at += w
    o, S = call(d)
    o2, S2 = call(e)
    torch.cuda.synchronize()
    assert torch.equal(o, o2) and torch.equal(S, S2)


@pytest.mark.parametrize("sdtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("N,T,ch,M,G", [(1, 1, 1, 1, 1), (5, 1, 70, 16, 1), (3, 4, 66, 24, 2),
                                        (2, 2, 40, 5, 1), (70, 1, 33, 64, 3), (2, 3, 9, 128, 1)])
def test_step(N, T, ch, M, G, sdtype):
    """Tokens against slots in any order, a padding entry among them; other slots untouched."""
    dtype = torch.bfloat16
    h = make((N, T), ch, M, G, N, dtype, seed=N + ch, state=False, wide=2)
    pool = Draw(5).normal(N + 3, ch, M, dtype=sdtype)
    idx = torch.randperm(N + 3, generator=torch.Generator().manual_seed(2))[:N].to(torch.int32)
    if N > 2:
        idx[1] = -7
    d, P = on_gpu_sliced(h, 2), pool.cuda()
    o = g.selective_scan_step(d["x"], d["dt"], d["A"], d["B"], d["C"], P, D=d["D"], gate=d["gate"],
                              dt_bias=d["dt_bias"], dt_softplus=True, state_idx=idx.cuda())
    torch.cuda.synchronize()
    want, lim = f64(pool), np.zeros(pool.shape)
    for n, s in enumerate(idx.tolist()):
        if s < 0:
            assert torch.all(o[n] == 0)
            continue
        one = {k: t[n:n + 1] if k in ("x", "dt", "B", "C", "gate") and t is not None else t
               for k, t in h.items()}
        one["S0"] = pool[s:s + 1].float()
        r = ref(one, [T])
        check("o", o[n], r["o"], r["o_b"], dtype)
        want[s] = r["S_T"][0]
        lim[s] = r["S_T_b"][0] + HALF_STEP[sdtype] * np.abs(want[s])
    check("pool", P, want, lim, sdtype)
    rest = [s for s in range(N + 3) if s not in idx.tolist()]
    assert torch.equal(P[rest].cpu(), pool[rest])


def test_slots_behind_two_gib():
    """A bf16 pool of more than 2^31 elements: the last slots hold what a small pool would."""
    ch, M, N = 512, 64, 2
    slots = (1 << 31) // (ch * M) + 3
    h = make((N, 1), ch, M, 1, N, torch.bfloat16, seed=31, state=False)
    d = gpu(h)
    small = Draw(6).normal(N, ch, M, dtype=torch.bfloat16).cuda()
    pool = torch.empty(slots, ch, M, dtype=torch.bfloat16, device="cuda")
    pool[-N:] = small
    args = dict(D=d["D"], gate=d["gate"], dt_bias=d["dt_bias"], dt_softplus=True)
    x = (d["x"], d["dt"], d["A"], d["B"], d["C"])
    idx = torch.tensor([slots - 2, slots - 1], dtype=torch.int32, device="cuda")
    o = g.selective_scan_step(*x, pool, state_idx=idx, **args)
    o2 = g.selective_scan_step(*x, small, **args)
    torch.cuda.synchronize()
    assert torch.equal(o, o2) and torch.equal(pool[-N:], small)


def test_prompt_then_tokens():
    """A prompt's states go on token by token to the same o and states as one longer prompt."""
    T, cut, ch = 50, 37, 66
    h = make((1, T), ch, 16, 1, 1, torch.float32, seed=12)
    d = gpu(h)
    part = {n: t[:, :cut].contiguous() if t is not None and n in ("x", "dt", "B", "C", "gate") else t
            for n, t in d.items()}
    o0, pool = call(part)
    o1 = [g.selective_scan_step(*(d[n][:, t:t + 1].contiguous() if n != "A" else d["A"]
                                  for n in ("x", "dt", "A", "B", "C")), pool, D=d["D"],
                                gate=d["gate"][:, t:t + 1].contiguous(), dt_bias=d["dt_bias"],
                                dt_softplus=True) for t in range(cut, T)]
    torch.cuda.synchronize()
    r = ref(h, [T])
    check("o", torch.cat([o0] + o1, 1)[0], r["o"], r["o_b"])
    check("S", pool, r["S_T"], r["S_T_b"])


def test_refusals():
    h = make((1, 6), 8, 4, 1, 1, torch.float32, seed=13)
    d = gpu(h)
    for change in ({"dt": d["dt"][:, :, :7]}, {"A": d["A"][:, :3]}, {"C": d["C"].to(torch.bfloat16)},
                   {"x": d["x"].cpu()}, {"D": d["D"][:4]}, {"B": d["B"][:, :5]},
                   {"S0": d["S0"].to(torch.bfloat16)}):
        with pytest.raises((ValueError, TypeError)):
            call({**d, **change})
    big = torch.zeros(1, 6, 1, 200, device="cuda")
    with pytest.raises(g.GDN2Error):
        call({**d, "A": torch.zeros(8, 200, device="cuda"), "B": big, "C": big, "S0": None})
    three = torch.zeros(1, 6, 3, 4, device="cuda")
    with pytest.raises(g.GDN2Error):
        call({**d, "B": three, "C": three})                    # 8 channels, 3 groups
    with pytest.raises(g.GDN2Error):
        call(d, final_state=d["S0"])                           # in place
    with pytest.raises(TypeError):
        g.selective_scan_step(d["x"], d["dt"], d["A"], d["B"], d["C"], d["S0"].half())


@pytest.mark.parametrize("T", [12, 200])
def test_rates_of_minus_infinity_and_nan(T):
    """A rate of -inf forgets at every step but keeps the state over steps of zero, over a tile's
    bounds and in single tokens alike. A NaN rate spoils its channel and no other."""
    h = make((1, T), 10, 16, 1, 1, torch.float32, seed=15)
    h["A"][3, 2] = float("-inf")
    h["dt"][:, T // 4:] = float("-inf")
    d = gpu(h)
    o, S = call(d)
    r = ref({**h, "dt": h["dt"].clamp(min=-300.0), "A": h["A"].clamp(min=-1e30)}, [T])
    check("o", o[0], r["o"], r["o_b"])
    check("S_T", S, r["S_T"], r["S_T_b"])
    pool = d["S0"].clone()
    steps = []
    for t in range(T):
        x, dt, B, C, gate = (d[n][:, t:t + 1] for n in ("x", "dt", "B", "C", "gate"))
        steps.append(g.selective_scan_step(x, dt, d["A"], B, C, pool, D=d["D"], gate=gate,
                                           dt_bias=d["dt_bias"], dt_softplus=True)[0])
    check("o by steps", torch.cat(steps), r["o"], r["o_b"])
    check("S by steps", pool, r["S_T"], r["S_T_b"])
    d["A"][5, 1] = float("nan")
    bad, Sb = call(d)
    torch.cuda.synchronize()
    keep = [c for c in range(10) if c != 5]
    assert torch.isnan(bad[0, :, 5]).all() and torch.isnan(Sb[0, 5]).any()
    assert torch.equal(bad[:, :, keep], o[:, :, keep]) and torch.equal(Sb[0, keep], S[0, keep])


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("ch,M,G", [(70, 5, 1), (66, 16, 2), (70, 20, 1), (20, 50, 1), (12, 100, 2)])
def test_many_tiles(ch, M, G, dtype):
    """More tiles than the last pass chains itself, at every number of lanes per channel, with
    sequences that start and end inside tiles."""
    lens = [333, 0, 1, 290, 7, 60, 0]
    T = sum(lens)
    h = make((1, T), ch, M, G, len(lens), dtype, seed=M)
    o, S = call(gpu(h), cu_seqlens=cu_of(lens))
    torch.cuda.synchronize()
    r = ref(h, lens)
    check("o", o[0], r["o"], r["o_b"], dtype)
    check("S_T", S, r["S_T"], r["S_T_b"])


@pytest.mark.parametrize("B,T,ch,M", [(900, 9, 70, 5), (900, 9, 70, 16), (600, 5, 70, 20),
                                      (300, 17, 300, 50), (300, 17, 130, 100)])
def test_whole_sequences_of_a_large_batch(B, T, ch, M):
    """Batches that are not cut and give every SIMD its waves with 8 or 16 states per lane."""
    h = make((B, T), ch, M, 1, B, torch.float32, seed=M)
    o, S = call(gpu(h))
    torch.cuda.synchronize()
    r = ref(h, [T] * B)
    check("o", o.reshape(B * T, ch), r["o"], r["o_b"])
    check("S_T", S, r["S_T"], r["S_T_b"])


@pytest.mark.parametrize("M", [4, 16, 32, 64, 128])
def test_rows_of_states_at_odd_addresses(M):
    """Rates and states that start four bytes behind a 16-byte boundary give the bits of the
    aligned call, in calls of few tokens and of many tiles."""
    for T in (40, 600):
        h = make((1, T), 24, M, 1, 1, torch.float32, seed=T)
        d = gpu(h)
        o, S = call(d)

        def off(t):
            buf = torch.empty(t.numel() + 1, device="cuda")
            v = buf[1:].view(t.shape)
            return v.copy_(t)

        e = {**d, "A": off(d["A"]), "S0": off(d["S0"])}
        o2, S2 = call(e, final_state=off(torch.zeros_like(S)))
        torch.cuda.synchronize()
        assert torch.equal(o, o2) and torch.equal(S, S2)


@pytest.mark.parametrize("name", ["x", "dt", "B", "C", "gate", "S0"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("lens", [[41, 23, 50], [300, 90, 250]])
def test_values_that_are_not_finite_stay_in_their_sequence(name, bad, lens):
    """The middle one of three sequences, which meet inside tiles, holds NaN or infinities: the
    bits of the others' outputs and states do not change, in calls of few tokens and of many."""
    a, b = lens[0], lens[0] + lens[1]
    h = make((1, sum(lens)), 24, 16, 1, 3, torch.float32, seed=14)
    d = gpu(h)
    o0, S0 = call(d, cu_seqlens=cu_of(lens))
    if name == "S0":
        d[name][1] = bad
    else:
        d[name][:, a:b] = bad
    o, S = call(d, cu_seqlens=cu_of(lens))
    torch.cuda.synchronize()
    assert torch.equal(o[:, :a], o0[:, :a]) and torch.equal(o[:, b:], o0[:, b:])
    assert torch.equal(S[[0, 2]], S0[[0, 2]])
    assert not torch.equal(o, o0)
