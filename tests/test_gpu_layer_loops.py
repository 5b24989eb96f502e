"""Loops of the operators around the recurrence that small calls do not enter: workgroups that take
several rows or sequences, grids beyond one dimension, searches over thousands of sequences; and two
calls at once from two threads."""
import threading

import numpy as np
import pytest
import torch

import gated_delta_rule_gdn_amd as g
from layer_common import HALF_STEP, act_err, check, f64, scan_bwd_ref, sigmoid, U
from test_gpu_block_norm import make as norm_make
from test_gpu_block_norm import run_and_check as norm_check
from test_gpu_selective_scan import Draw, call as scan_call, gpu, make, on_gpu_sliced, ref
from test_gpu_selective_scan_bwd import call as bwd_call, flat, ref_args

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


def setup_module(module):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    g.lib()


# 768 workgroups of a backward pass hold 16 rows of at most 128 columns, four of at most 512, one of more
@pytest.mark.parametrize("rows,d,dtype,rdtype,gtype,off", [
    (30000, 40, BF16, BF16, BF16, ()), (25000, 33, F32, F32, F32, ("next_weight",)),
    (8000, 130, BF16, F32, F32, ()), (7000, 512, F32, F32, F32, ("norm_weight",)),
    (1700, 520, BF16, BF16, F32, ()), (1700, 1023, BF16, F32, BF16, ("norm_weight",)),
    (1700, 2048, BF16, F32, BF16, ()), (1700, 2048, BF16, BF16, BF16, ("next_weight",)),
    (1600, 2049, F32, F32, F32, ()), (1600, 4096, BF16, F32, F32, ("norm_weight",)),
    (1600, 4100, BF16, BF16, BF16, ()), (1600, 4101, F32, F32, F32, ("next_weight",)),
    (1600, 8200, BF16, F32, BF16, ("norm_weight",)), (1600, 8192, F32, F32, F32, ())],
    ids=lambda v: str(v).replace("torch.", "") if not isinstance(v, tuple) else "-".join(("no",) + v) if v else "all")
def test_norm_gradients_of_many_rows(rows, d, dtype, rdtype, gtype, off):
    """Two and more sets of rows per workgroup at every number of lanes per row, with four, two and
    (one statistic left out) odd numbers of sums over a row."""
    h = norm_make(rows, d, dtype, rdtype, seed=d)
    for n in off:
        h[n] = None
    norm_check(h, dtype, rdtype, gtype)


@pytest.mark.parametrize("sdtype", [F32, BF16])
@pytest.mark.parametrize("N,T,ch,M", [(70, 1, 2050, 16), (45, 2, 4097, 15), (40, 2, 2050, 64)])
def test_scan_step_of_several_sequences_per_workgroup(N, T, ch, M, sdtype):
    """The next sequence's state and token are loaded while one is worked on: padding first, last
    and in between, slots in any order."""
    h = make((N, T), ch, M, 1, N, BF16, seed=N, state=False, wide=4)
    pool = Draw(7).normal(N + 2, ch, M, dtype=sdtype)
    idx = torch.randperm(N + 2, generator=torch.Generator().manual_seed(3))[:N].to(torch.int32)
    idx[0], idx[13], idx[14], idx[N - 1] = -1, N + 2, -(1 << 31), (1 << 31) - 1
    d, P = on_gpu_sliced(h, 4), pool.cuda()
    o = g.selective_scan_step(d["x"], d["dt"], d["A"], d["B"], d["C"], P, D=d["D"], gate=d["gate"],
                              dt_bias=d["dt_bias"], dt_softplus=True, state_idx=idx.cuda())
    torch.cuda.synchronize()
    used = [n for n in range(N) if 0 <= idx[n] < N + 2]
    one = {k: t[used] if k in ("x", "dt", "B", "C", "gate") else t for k, t in h.items()}
    one["S0"] = pool[idx[used].long()].float()
    r = ref(one, [T] * len(used))
    check("o", o[used].reshape(-1, ch), r["o"], r["o_b"], BF16)
    rest = [n for n in range(N) if n not in used]
    assert torch.all(o[rest] == 0)
    lim = r["S_T_b"] + HALF_STEP[sdtype] * np.abs(r["S_T"])
    check("pool", P[idx[used].long().cuda()], r["S_T"], lim, sdtype)
    left = [s for s in range(N + 2) if s not in idx[used].tolist()]
    assert torch.equal(P[left].cpu(), pool[left])


@pytest.mark.parametrize("C", [4, 5])
def test_conv_step_of_more_sequences_than_a_grid_dimension(C):
    N, W = 70000, 4
    gen = torch.Generator().manual_seed(4)
    n = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    x, w, pool = n(N, 1, C), n(C, W), n(N, W - 1, C)
    idx = torch.randperm(N, generator=gen).to(torch.int32)
    idx[69999] = -1
    P = pool.cuda()
    y = g.short_conv_step(x.cuda(), w.cuda(), P, state_idx=idx.cuda(), silu=True)
    torch.cuda.synchronize()
    at = idx.long().clamp(min=0)
    seen = np.concatenate([f64(pool)[at], f64(x)], 1)            # [N, W, C]
    a = (seen * f64(w).T).sum(1)
    da = (W + 2) * U * (np.abs(seen) * np.abs(f64(w).T)).sum(1)
    assert torch.all(y[69999] == 0)
    check("y", y[:69999, 0], (a * sigmoid(a))[:69999], act_err(a, da)[:69999])
    want = f64(pool)
    want[at[:69999]] = seen[:69999, 1:]
    assert np.array_equal(f64(P), want)


def test_scan_over_more_tiles_than_a_grid_dimension():
    """15,000 packed copies of one sequence of 40 tokens: 37,500 tiles, which begin at any of its
    tokens, and a search over 15,000 offsets. Every copy is held to the one's bounds."""
    N, L, ch, M = 15000, 40, 5, 3
    h = make((1, L), ch, M, 1, 1, F32, seed=16)
    many = {n: t.repeat(1, N, *[1] * (t.dim() - 2)) if n in ("x", "dt", "B", "C", "gate") else t for n, t in h.items()}
    many["S0"] = h["S0"].repeat(N, 1, 1)
    cu = (torch.arange(N + 1, dtype=torch.int32) * L).cuda()
    d = gpu(many)
    q = Draw(17)
    dO, dS = q.normal(1, L, ch), q.normal(1, ch, M)
    o, S = scan_call(d, cu_seqlens=cu)
    b = bwd_call(d, dO.repeat(1, N, 1).cuda(), dS.repeat(N, 1, 1).cuda(), cu_seqlens=cu)
    torch.cuda.synchronize()
    r = ref(h, [L])
    every = lambda t: np.broadcast_to(t, (N, *t.shape))  # noqa: E731
    check("o", o.reshape(N, L, ch), every(r["o"]), every(r["o_b"]))
    check("S_T", S, every(r["S_T"][0]), every(r["S_T_b"][0]))
    r = scan_bwd_ref(*ref_args(flat(h, L), True, [L]), f64(dO)[0], f64(dS))
    for n in ("dx", "ddt", "dB", "dC", "dgate"):
        check(n, b[n].reshape(N, L, *b[n].shape[2:]), every(r[n]), every(r[n + "_b"]))
    check("dS0", b["dS0"], every(r["dS0"][0]), every(r["dS0_b"][0]))
    # 37,500 tiles' sums, four waves of 9,375 each, a tile's own first: at most 9,375 + 24 roundings of
    # partial sums, which are at most the sum of the terms' magnitudes; the copies' own bounds add up
    for n, mag in (("dD", np.abs(f64(dO)[0] * sigmoid(f64(h["gate"])[0]) * f64(h["gate"])[0] * f64(h["x"])[0]).sum(0)),
                   ("ddt_bias", np.abs(r["ddt"]).sum(0))):
        check(n, b[n], N * r[n], N * (r[n + "_b"] + (9375 + 24) * U * mag))


def test_two_threads_at_once():
    """Calls from two threads, on streams of their own, with different sizes of the same kernels:
    each gives the bits it gives alone."""
    todo = []
    for T, seed in ((700, 18), (70, 19)):
        d = gpu(make((1, T), 264, 16, 1, 1, BF16, seed=seed))
        dO = Draw(seed).normal(1, T, 264, dtype=BF16).cuda()
        w, cw = torch.rand(264, device="cuda"), torch.rand(264, 4, device="cuda")

        def run(d=d, dO=dO, w=w, cw=cw):
            b = bwd_call(d, dO, None)
            n = g.block_norm_bwd(d["x"], dh=dO, norm_weight=w, gate=d["gate"])
            c = g.short_conv_bwd(d["x"], cw, dO, silu=True)
            return [scan_call(d)[0], *b.values(), *n.values(), *c.values()]

        todo.append((run, [t.clone() for t in run()]))
    torch.cuda.synchronize()
    bad = []

    def work(run, want):
        try:
            st = torch.cuda.Stream()
            with torch.cuda.stream(st):
                for _ in range(20):
                    got = run()
                    if not all(torch.equal(a, b) for a, b in zip(got, want)):
                        bad.append("other bits")
            st.synchronize()
        except Exception as e:      # noqa: BLE001  (reported below, in the test's own thread)
            bad.append(repr(e))

    threads = [threading.Thread(target=work, args=t) for t in todo]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad, bad
