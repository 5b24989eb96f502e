"""The norms around a block and their gradients against a plain 64-bit form."""
import itertools

import numpy as np
import pytest
import torch

import gated_delta_rule_gdn_amd as g
from layer_common import check, f64, norm_ref

pytestmark = pytest.mark.gpu


def setup_module(module):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    g.lib()


def make(rows, d, dtype, rdtype, seed, nw=True, gate=True, res=True, scale=True, nxt=True):
    gen = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    return {"x": n(rows, d).to(dtype), "norm_weight": 1 + 0.2 * n(d) if nw else None,
            "gate": n(rows, d).to(dtype) if gate else None,
            "residual": (2 * n(rows, d)).to(rdtype) if res else None,
            "scale": 0.5 * n(d) if scale else None, "next_weight": 1 + 0.2 * n(d) if nxt else None}


def run_and_check(h, dtype, rdtype, gtype, dev=None, eps=1e-5):
    """Forward and backward against the reference, every output by its type."""
    rows, d = h["x"].shape
    gen = torch.Generator().manual_seed(rows + d)
    res, nxt = h["residual"] is not None, h["next_weight"] is not None
    ht = rdtype if res else dtype
    dht = torch.float32 if res and rdtype == torch.float32 else gtype
    dh = torch.randn(rows, d, generator=gen).to(dht)
    dy = torch.randn(rows, d, generator=gen).to(gtype) if nxt else None
    v = {n: None if t is None else f64(t) for n, t in h.items()}
    r = norm_ref(v["x"], v["norm_weight"], v["gate"], v["residual"], v["scale"], v["next_weight"], eps,
                 f64(dh), None if dy is None else f64(dy))
    c = dev or {n: None if t is None else t.cuda() for n, t in h.items()}
    kw = {n: c[n] for n in ("norm_weight", "gate", "residual", "scale", "next_weight")}
    hh, y = g.block_norm_fwd(c["x"], eps=eps, **kw)
    o = g.block_norm_bwd(c["x"], dh=dh.cuda(), dy=None if dy is None else dy.cuda(), eps=eps,
                         grad_dtype=gtype, **kw)
    torch.cuda.synchronize()
    assert hh.dtype == ht and (y is None) == (not nxt)
    check("h", hh, r["h"], r["h_b"], ht)
    if nxt:
        check("y", y, r["y"], r["y_b"], dtype)
    want = {"dx"} | {"d" + n for n, t in kw.items() if t is not None}
    assert set(o) == want
    for n in sorted(want):
        t = gtype if n in ("dx", "dgate") else dht if n == "dresidual" else torch.float32
        assert o[n].dtype == t, n
        check(n, o[n], r[n], r[n + "_b"], t)


@pytest.mark.parametrize("dtype,rdtype,gtype", [
    (torch.float32, torch.float32, torch.float32), (torch.bfloat16, torch.bfloat16, torch.bfloat16),
    (torch.bfloat16, torch.bfloat16, torch.float32), (torch.bfloat16, torch.float32, torch.bfloat16),
    (torch.bfloat16, torch.float32, torch.float32)])
@pytest.mark.parametrize("rows,d", [(1, 1), (3, 7), (33, 64), (17, 128), (5, 130), (9, 513), (4, 1000),
                                    (7, 1024), (3, 2048), (2, 2050), (3, 4096), (2, 5000), (2, 8192),
                                    (2, 10001), (3, 16384)])
def test_widths_and_types(rows, d, dtype, rdtype, gtype):
    run_and_check(make(rows, d, dtype, rdtype, seed=d), dtype, rdtype, gtype)


@pytest.mark.parametrize("on", list(itertools.product([False, True], repeat=5)))
def test_every_choice_of_stages(on):
    dtype = torch.bfloat16
    run_and_check(make(21, 72, dtype, dtype, 5, *on), dtype, dtype, dtype)


def test_many_rows_over_few_workgroups():
    """More rows than the backward has workgroups: each sums several."""
    run_and_check(make(2100, 264, torch.float32, torch.float32, 6), *[torch.float32] * 3)


@pytest.mark.parametrize("d", [64, 66])
def test_column_slices_and_token_shapes(d):
    """x and gate as column slices of one projection, rows as [B, T]; the same bits as copies."""
    B, T = 3, 11
    buf = torch.randn(B, T, 3 * d, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).cuda()
    x, gate = buf[..., d:2 * d], buf[..., 2 * d:]
    w = torch.rand(d, generator=torch.Generator().manual_seed(2)).cuda()
    a = g.block_norm_fwd(x, norm_weight=w, gate=gate)[0]
    b = g.block_norm_fwd(x.contiguous(), norm_weight=w, gate=gate.contiguous())[0]
    ga = g.block_norm_bwd(x, dh=a, norm_weight=w, gate=gate)
    gb = g.block_norm_bwd(x.contiguous(), dh=a, norm_weight=w, gate=gate.contiguous())
    torch.cuda.synchronize()
    assert a.shape == (B, T, d) and torch.equal(a, b)
    assert all(torch.equal(ga[n], gb[n]) for n in ga)


def test_residual_in_place():
    h = make(40, 256, torch.bfloat16, torch.bfloat16, 7)
    c = {n: t.cuda() for n, t in h.items()}
    want, wy = g.block_norm_fwd(**c)
    got, y = g.block_norm_fwd(**c, out=c["residual"])
    torch.cuda.synchronize()
    assert got.data_ptr() == c["residual"].data_ptr()
    assert torch.equal(got, want) and torch.equal(y, wy)


def test_rows_of_zeros_and_bad_rows():
    """A row of zeros gives zeros through eps; a row with NaN or inf spoils only itself."""
    h = make(6, 96, torch.float32, torch.float32, 8, res=False, scale=False)
    clean = {n: None if t is None else t.cuda() for n, t in h.items()}
    h["x"][1] = 0.0
    h["x"][3, 5] = float("nan")
    h["x"][4, 7] = float("inf")
    c = {n: None if t is None else t.cuda() for n, t in h.items()}
    hh, y = g.block_norm_fwd(**c)
    h0, y0 = g.block_norm_fwd(**clean)
    torch.cuda.synchronize()
    assert torch.all(hh[1] == 0) and torch.all(y[1] == 0)
    assert torch.isnan(y[3]).all() and torch.isnan(hh[4, 7])
    assert torch.equal(hh[[0, 2, 5]], h0[[0, 2, 5]]) and torch.equal(y[[0, 2, 5]], y0[[0, 2, 5]])


def test_no_rows():
    w = torch.ones(8, device="cuda")
    x = torch.zeros(0, 8, device="cuda")
    h, y = g.block_norm_fwd(x, norm_weight=w, next_weight=w)
    o = g.block_norm_bwd(x, dh=x, dy=x, norm_weight=w, next_weight=w)
    torch.cuda.synchronize()
    assert h.shape == (0, 8) and torch.all(o["dnorm_weight"] == 0) and torch.all(o["dnext_weight"] == 0)


def test_same_as_the_fused_output_norm():
    """chunk_fwd's fused gated norm equals chunk_fwd without it followed by this call (fp32)."""
    from gated_delta_rule_gdn_amd import inputs
    x = {n: t.cuda() if isinstance(t, torch.Tensor) else t
         for n, t in inputs.chunk_inputs(inputs.small_chunk(seqlen=70, d_v=128), seed=1).items()}
    a = [x[n] for n in ("q", "k", "v", "log_alpha", "b", "w")]
    gen = torch.Generator().manual_seed(3)
    gate = torch.randn(x["v"].shape, generator=gen).cuda()
    w = 1 + 0.1 * torch.randn(128, generator=gen).cuda()
    o1, _ = g.chunk_fwd(*a, S0=x["S0"], gate=gate, norm_weight=w)
    o2, _ = g.chunk_fwd(*a, S0=x["S0"])
    o3, _ = g.block_norm_fwd(o2, norm_weight=w, gate=gate)
    torch.cuda.synchronize()
    assert float((o1 - o3).norm() / o1.norm()) <= 40 * 2.0 ** -24


def test_refusals():
    h = make(4, 16, torch.bfloat16, torch.bfloat16, 9)
    c = {n: t.cuda() for n, t in h.items()}
    for change in ({"gate": c["gate"][:, :8]}, {"scale": c["scale"].to(torch.bfloat16)},
                   {"residual": c["residual"].half()}, {"x": c["x"].t()}, {"norm_weight": c["norm_weight"].cpu()}):
        with pytest.raises((ValueError, TypeError)):
            g.block_norm_fwd(**{**c, **change})
    with pytest.raises(g.GDN2Error):
        g.block_norm_fwd(torch.zeros(2, 16385, device="cuda"))
    with pytest.raises(g.GDN2Error):
        g.block_norm_fwd(c["x"], out=c["x"])
    with pytest.raises(g.GDN2Error):
        g.block_norm_fwd(c["x"], eps=-1.0)
    with pytest.raises(ValueError):
        g.block_norm_bwd(**c, dh=c["x"])                        # next_weight without dy
    with pytest.raises(ValueError):
        g.block_norm_bwd(c["x"])
    with pytest.raises(TypeError):
        g.block_norm_bwd(c["x"], dh=c["x"].half())


def test_more_rows_than_one_grid_dimension_holds():
    """2^28 + 5 rows of two columns: 16 lanes a row would be more than 2^32 threads in a row."""
    rows = (1 << 28) + 5
    x = torch.zeros(rows, 2, dtype=torch.bfloat16, device="cuda")
    picked = [0, 1, 12345678, (1 << 28) - 1, 1 << 28, rows - 1]
    x[picked] = torch.tensor([3.0, 4.0], dtype=torch.bfloat16, device="cuda")
    w = torch.ones(2, device="cuda")
    h, _ = g.block_norm_fwd(x, norm_weight=w, eps=1e-5)
    torch.cuda.synchronize()
    want = torch.tensor([3.0, 4.0]) / 12.5 ** 0.5       # 1e-5 of 12.5 is below half a bf16 step
    assert torch.equal(h[picked].cpu(), want.to(torch.bfloat16).expand(len(picked), 2))
    assert int(torch.count_nonzero(h)) == 2 * len(picked)
