"""Offsets that decrease or lie outside the batch: wrong results, but no access outside the tensors.
The walk itself is checked over many tables on the host (test_span_walk_host.py); here the calls
run on a few, with rows of other values around every state."""
import pytest
import torch

import gated_delta_rule_gdn_amd as g

pytestmark = pytest.mark.gpu

T, C, M, GUARD = 200, 40, 16, 300
TABLES = [[0, 150, 120, 20, 200], [200, 0, 200, 0, 200], [0, -50, 900, 64, 63], [199, 3, 3, 198, 1]]


def setup_module(module):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    g.lib()


def guarded(n, *row, fill):
    """n rows between GUARD rows of `fill` on either side: (the whole buffer, the rows)."""
    buf = torch.full((n + 2 * GUARD, *row), fill, device="cuda")
    return buf, buf[GUARD:GUARD + n]


def untouched(buf, n, fill):
    return bool(torch.all(buf[:GUARD] == fill)) and bool(torch.all(buf[GUARD + n:] == fill))


@pytest.mark.parametrize("table", TABLES, ids=str)
def test_accesses_stay_inside(table):
    gen = torch.Generator().manual_seed(1)
    n = lambda *s: torch.randn(*s, generator=gen).cuda()  # noqa: E731
    N = len(table) - 1
    cu = torch.tensor(table, dtype=torch.int32, device="cuda")
    x, dt, gate, dy = (n(1, T, C) for _ in range(4))
    w, A, B, Cm = n(C, 4), -n(C, M).abs(), n(1, T, 1, M), n(1, T, 1, M)
    nan = float("nan")
    s0 = guarded(N, 3, C, fill=nan)[1].copy_(n(N, 3, C))
    ds = guarded(N, 3, C, fill=nan)[1].copy_(n(N, 3, C))
    out, st = guarded(T, C, fill=7.0), guarded(N, 3, C, fill=7.0)
    out[1].zero_()
    st[1].zero_()
    y, _ = g.short_conv_fwd(x, w, state0=s0, cu_seqlens=cu, silu=True, out=out[1][None], final_state=st[1])
    g.short_conv_bwd(x, w, dy, state0=s0, cu_seqlens=cu, silu=True, dstate_T=ds)
    S0, S = n(N, C, M), guarded(N, C, M, fill=7.0)
    o = guarded(T, C, fill=7.0)
    g.selective_scan_fwd(x, dt, A, B, Cm, gate=gate, dt_softplus=True, S0=S0, cu_seqlens=cu,
                         out=o[1][None], final_state=S[1])
    g.selective_scan_bwd(x, dt, A, B, Cm, dy, gate=gate, dt_softplus=True, S0=S0, cu_seqlens=cu, dS_T=S0)
    torch.cuda.synchronize()
    assert torch.isfinite(y).all() and torch.isfinite(st[1]).all()     # nothing of the guards was read
    assert untouched(out[0], T, 7.0) and untouched(st[0], N, 7.0)
    assert untouched(o[0], T, 7.0) and untouched(S[0], N, 7.0)
