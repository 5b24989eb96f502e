"""Gradients of the selective scan against a plain 64-bit form token by token, and against
differences of that form."""
import numpy as np
import pytest
import torch

import gated_delta_rule_gdn_amd as g
from layer_common import check, f64, scan_bwd_ref, scan_ref
from test_gpu_selective_scan import Draw, cu_of, gpu, make, on_gpu_sliced

pytestmark = pytest.mark.gpu


def setup_module(module):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    g.lib()


def flat(h, T):
    v = {n: None if t is None else f64(t) for n, t in h.items()}
    return {n: a if a is None or n in ("A", "D", "dt_bias", "S0") else a.reshape(T, *a.shape[2:])
            for n, a in v.items()}


def ref_args(v, softplus, lens):
    return (v["x"], v["dt"], v["A"], v["B"], v["C"], v["D"], v["gate"], v["dt_bias"], softplus, v["S0"], lens)


def call(d, dO, dS, softplus=True, **kw):
    return g.selective_scan_bwd(d["x"], d["dt"], d["A"], d["B"], d["C"], dO, D=d["D"], gate=d["gate"],
                                dt_bias=d["dt_bias"], dt_softplus=softplus, S0=d["S0"], dS_T=dS, **kw)


def run_and_check(h, lens, dtype, gtype, softplus=True, wide=0, packed=True, last=True):
    T, N = int(sum(lens)), len(lens)
    ch, M = h["A"].shape
    q = Draw(T + ch)
    dO = q.normal(*h["x"].shape, dtype=gtype)
    dS = q.normal(N, ch, M) if last else None
    o = call(on_gpu_sliced(h, wide), dO.cuda(), None if dS is None else dS.cuda(), softplus,
             cu_seqlens=cu_of(lens) if packed else None)
    torch.cuda.synchronize()
    r = scan_bwd_ref(*ref_args(flat(h, T), softplus, lens), f64(dO).reshape(T, ch), None if dS is None else f64(dS))
    want = {"dx", "ddt", "dA", "dB", "dC"} | {"d" + n for n in ("D", "gate", "dt_bias", "S0") if h[n] is not None}
    assert set(o) == want
    for n in sorted(want):
        token = n in ("dx", "ddt", "dB", "dC", "dgate")
        assert o[n].dtype == (gtype if token else torch.float32), n
        got = o[n].reshape(T, *o[n].shape[2:]) if token else o[n]
        check(n, got, r[n], r[n + "_b"], gtype if token else torch.float32)
    return o


LENS = [[1], [7], [8], [9], [31], [32], [33], [130], [0], [0, 1, 0, 0, 2, 40, 1, 0],
        [15, 1, 16, 1, 33, 0, 20], [1] * 70, [0] * 66 + [19] + [0] * 3 + [2]]


@pytest.mark.parametrize("dtype,gtype", [(torch.float32, torch.float32), (torch.bfloat16, torch.bfloat16),
                                         (torch.bfloat16, torch.float32)])
@pytest.mark.parametrize("lens", LENS, ids=lambda v: f"n{len(v)}t{sum(v)}")
def test_packed_lengths(lens, dtype, gtype):
    h = make((1, int(sum(lens))), 70, 16, 1, len(lens), dtype, seed=len(lens) + sum(lens))
    run_and_check(h, lens, dtype, gtype)


@pytest.mark.parametrize("M", [1, 3, 8, 9, 16, 17, 32, 33, 64, 65, 128])
@pytest.mark.parametrize("ch,G", [(1, 1), (66, 2), (300, 3)])
def test_state_sizes_channels_and_groups(ch, G, M):
    lens = [37, 5]
    h = make((1, 42), ch, M, G, 2, torch.bfloat16, seed=ch + M)
    run_and_check(h, lens, torch.bfloat16, torch.float32, wide=3)


@pytest.mark.parametrize("gate,D,bias,state,softplus", [
    (False, False, False, False, True), (True, False, True, False, True),
    (False, True, False, True, False), (True, True, True, True, True)])
@pytest.mark.parametrize("B,T,ch", [(1, 1, 8), (3, 40, 65), (2, 200, 260), (70, 9, 16), (4, 0, 8), (2, 32, 5)])
def test_dense_options(B, T, ch, gate, D, bias, state, softplus):
    h = make((B, T), ch, 16, 1, B, torch.float32, seed=B + T, gate=gate, D=D, bias=bias, state=state)
    if not softplus:
        h["dt"] = h["dt"].abs() * 0.1
        h["dt_bias"] = None if h["dt_bias"] is None else h["dt_bias"].abs() * 0.01
    run_and_check(h, [T] * B, torch.float32, torch.float32, softplus, packed=False, last=state)


def test_long_sequence_of_slow_states():
    """1,200 tokens over 150 tiles with rates near zero: the last token's gradient reaches S0."""
    h = make((1, 1200), 40, 4, 1, 1, torch.float32, seed=3)
    h["A"] = -torch.rand(40, 4) * 0.02
    run_and_check(h, [1200], torch.float32, torch.float32)


def test_masked_steps():
    """Steps of dt = -inf: no gradient through them except D's, and the states' passes on."""
    h = make((1, 60), 20, 16, 1, 2, torch.float32, seed=8)
    h["dt"][:, 10:35] = float("-inf")
    h["dt"][:, 40:] = float("-inf")
    d = gpu(h)
    q = Draw(1)
    dO, dS = q.normal(1, 60, 20).cuda(), q.normal(2, 20, 16).cuda()
    o = call(d, dO, dS, cu_seqlens=cu_of([40, 20]))
    torch.cuda.synchronize()
    assert all(torch.isfinite(t).all() for t in o.values())
    assert torch.all(o["ddt"][:, 10:35] == 0) and torch.all(o["dB"][:, 40:] == 0)
    v = flat({**h, "dt": h["dt"].clamp(min=-300.0)}, 60)
    r = scan_bwd_ref(*ref_args(v, True, [40, 20]), f64(dO)[0], f64(dS))
    for n in ("dx", "dC", "dgate"):
        check(n, o[n][0], r[n], r[n + "_b"])
    for n in ("dA", "dD", "dS0"):
        check(n, o[n], r[n], r[n + "_b"])


def test_gradients_against_differences():
    """The reference's own gradients against central differences of the reference's outputs in
    64 bits, along random directions in every input (CPU arithmetic on both sides)."""
    lens, ch, M, G = [9, 0, 4], 6, 5, 2
    h = make((1, 13), ch, M, G, 3, torch.float32, seed=21)
    v = flat(h, 13)
    rng = np.random.default_rng(1)
    dO, dS = rng.standard_normal((13, ch)), rng.standard_normal((3, ch, M))

    def loss(w):
        r = scan_ref(*ref_args(w, True, lens))
        return float((r["o"] * dO).sum() + (r["S_T"] * dS).sum())

    d = scan_bwd_ref(*ref_args(v, True, lens), dO, dS)
    for n in ("x", "dt", "A", "B", "C", "D", "gate", "dt_bias", "S0"):
        p = rng.standard_normal(v[n].shape)
        eps = 1e-6
        num = (loss({**v, n: v[n] + eps * p}) - loss({**v, n: v[n] - eps * p})) / (2 * eps)
        want = float((d["d" + n] * p).sum())
        assert abs(num - want) <= 1e-6 * max(1.0, abs(want)), (n, num, want)


def test_rows_behind_the_last_sequence():
    """Tokens behind the last sequence hold NaN: no gradient of the others sees them."""
    h = make((1, 120), 20, 16, 1, 2, torch.bfloat16, seed=10)
    d = gpu(h)
    dO = Draw(2).normal(1, 120, 20, dtype=torch.bfloat16).cuda()
    for n in ("x", "dt", "B", "C", "gate"):
        d[n][:, 50:] = float("nan")
    dO[:, 50:] = float("nan")
    o = call(d, dO, None, cu_seqlens=cu_of([20, 30]))
    torch.cuda.synchronize()
    for n in ("dx", "ddt", "dB", "dC", "dgate"):
        assert torch.isfinite(o[n][:, :50]).all(), n
    for n in ("dA", "dD", "ddt_bias", "dS0"):
        assert torch.isfinite(o[n]).all(), n


def test_same_bits_at_every_call():
    h = make((1, 700), 300, 16, 1, 1, torch.bfloat16, seed=12)
    d = gpu(h)
    dO = Draw(3).normal(1, 700, 300, dtype=torch.bfloat16).cuda()
    a, b = call(d, dO, None), call(d, dO, None)
    torch.cuda.synchronize()
    assert all(torch.equal(a[n], b[n]) for n in a)


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
    dO = Draw(4).normal(1, T, ch).cuda()
    a, b = call(d, dO, None), call(e, dO, None)
    torch.cuda.synchronize()
    assert all(torch.equal(a[n], b[n]) for n in a)


def test_refusals():
    h = make((1, 6), 8, 4, 1, 1, torch.float32, seed=13)
    d = gpu(h)
    dO = torch.zeros(1, 6, 8, device="cuda")
    with pytest.raises(TypeError):
        call(d, dO.to(torch.bfloat16), None)                   # fp32 inputs, bf16 gradients
    with pytest.raises(ValueError):
        call(d, dO[:, :5], None)
    with pytest.raises(ValueError):
        call(d, dO, torch.zeros(2, 8, 4, device="cuda"))
    with pytest.raises(g.GDN2Error):
        call(d, dO, None, workspace=torch.zeros(16, dtype=torch.uint8, device="cuda"))


@pytest.mark.parametrize("name", ["x", "dt", "B", "C", "gate", "dO", "S0", "dS_T"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_values_that_are_not_finite_stay_in_their_sequence(name, bad):
    """The middle one of three sequences, which meet inside tiles, holds NaN or infinities from
    its start to its end: the bits of the others' gradients do not change."""
    lens = [300, 90, 200]
    h = make((1, 590), 24, 16, 1, 3, torch.float32, seed=14)
    d = gpu(h)
    q = Draw(5)
    d["dO"], d["dS_T"] = q.normal(1, 590, 24).cuda(), q.normal(3, 24, 16).cuda()
    clean = call(d, d["dO"], d["dS_T"], cu_seqlens=cu_of(lens))
    if name in ("S0", "dS_T"):
        d[name][1] = bad
    else:
        d[name][:, 300:390] = bad
    o = call(d, d["dO"], d["dS_T"], cu_seqlens=cu_of(lens))
    torch.cuda.synchronize()
    for n in ("dx", "ddt", "dB", "dC", "dgate"):
        for s in (slice(0, 300), slice(390, 590)):
            assert torch.equal(o[n][:, s], clean[n][:, s]), n
    assert torch.equal(o["dS0"][[0, 2]], clean["dS0"][[0, 2]])
    assert not all(torch.equal(o[n], clean[n]) for n in o)


def test_rates_of_minus_infinity_and_nan():
    """A rate of -inf forgets at every step but keeps the state over steps of zero; the gradients
    of inputs, B, C and gate stay finite. A NaN rate spoils its channel and no other."""
    h = make((1, 200), 10, 16, 1, 2, torch.float32, seed=15)
    h["A"][3, 2] = float("-inf")
    h["dt"][:, 40:180] = float("-inf")
    d = gpu(h)
    q = Draw(6)
    dO, dS = q.normal(1, 200, 10).cuda(), q.normal(2, 10, 16).cuda()
    cu = cu_of([190, 10])
    o = call(d, dO, dS, cu_seqlens=cu)
    v = flat({**h, "dt": h["dt"].clamp(min=-300.0), "A": h["A"].clamp(min=-1e30)}, 200)
    r = scan_bwd_ref(*ref_args(v, True, [190, 10]), f64(dO)[0], f64(dS))
    for n in ("dx", "dB", "dC", "dgate"):
        check(n, o[n][0], r[n], r[n + "_b"])
    d["A"][5, 1] = float("nan")
    bad = call(d, dO, dS, cu_seqlens=cu)
    torch.cuda.synchronize()
    keep = [c for c in range(10) if c != 5]
    assert torch.isnan(bad["dx"][0, :100, 5]).all()
    assert torch.equal(bad["dx"][:, :, keep], o["dx"][:, :, keep])


@pytest.mark.parametrize("ch,M", [(4096, 16), (2048, 17), (1024, 40), (512, 100)])
def test_many_waves(ch, M):
    """Sizes at which the tile pass takes sixteen states per lane, and tiles of 64 tokens."""
    lens = [900, 3, 0, 1197]
    h = make((1, 2100), ch, M, 1, 4, torch.float32, seed=M)
    run_and_check(h, lens, torch.float32, torch.float32)


@pytest.mark.parametrize("M", [4, 16, 32, 64, 128])
def test_rows_of_states_at_odd_addresses(M):
    """Rates and states that start four bytes behind a 16-byte boundary: the aligned call's bits."""
    h = make((1, 100), 24, M, 1, 2, torch.float32, seed=M)
    d = gpu(h)
    q = Draw(7)
    dO, dS = q.normal(1, 100, 24).cuda(), q.normal(2, 24, M).cuda()
    a = call(d, dO, dS, cu_seqlens=cu_of([70, 30]))

    def off(t):
        buf = torch.empty(t.numel() + 1, device="cuda")
        v = buf[1:].view(t.shape)
        return v.copy_(t)

    b = call({**d, "A": off(d["A"]), "S0": off(d["S0"])}, dO, off(dS), cu_seqlens=cu_of([70, 30]))
    torch.cuda.synchronize()
    assert all(torch.equal(a[n], b[n]) for n in a)
