"""The operators around the recurrence are ordered by the current stream: a call behind work that
makes its input on a side stream sees that input, and work behind it sees its outputs."""
import pytest
import torch

import gated_delta_rule_gdn_amd as g

pytestmark = pytest.mark.gpu

T, CH, M = 300, 264, 16


def setup_module(module):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    g.lib()


def inputs():
    gen = torch.Generator().manual_seed(7)
    n = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    bf = lambda *s: n(*s).to(torch.bfloat16).cuda()  # noqa: E731
    v = {"x": bf(1, T, CH), "dt": bf(1, T, CH), "z": bf(1, T, CH), "dO": bf(1, T, CH), "B": bf(1, T, 1, M),
         "C": bf(1, T, 1, M), "xs": bf(3, 2, CH), "Bs": bf(3, 2, 1, M)}
    p = {"A": -n(CH, M).abs().cuda(), "cw": n(CH, 4).cuda(), "D": n(CH).cuda(), "bias": n(CH).cuda() - 3,
         "w": n(CH).cuda(), "cpool": n(4, 3, CH).cuda(), "spool": n(4, CH, M).cuda(),
         "idx": torch.tensor([2, -1, 0], dtype=torch.int32, device="cuda")}
    return v, p


def scan(p, **kw):
    return dict(D=p["D"], dt_bias=p["bias"], dt_softplus=True, **kw)


CALLS = {
    "short_conv_fwd": lambda v, p: g.short_conv_fwd(v["x"], p["cw"], silu=True),
    "short_conv_bwd": lambda v, p: g.short_conv_bwd(v["x"], p["cw"], v["dO"], silu=True),
    "short_conv_step": lambda v, p: (g.short_conv_step(v["xs"], p["cw"], p["cpool"], state_idx=p["idx"]), p["cpool"]),
    "selective_scan_fwd": lambda v, p: g.selective_scan_fwd(v["x"], v["dt"], p["A"], v["B"], v["C"],
                                                            **scan(p, gate=v["z"])),
    "selective_scan_bwd": lambda v, p: g.selective_scan_bwd(v["x"], v["dt"], p["A"], v["B"], v["C"], v["dO"],
                                                            **scan(p, gate=v["z"])),
    "selective_scan_step": lambda v, p: (g.selective_scan_step(v["xs"], v["xs"], p["A"], v["Bs"], v["Bs"], p["spool"],
                                                               state_idx=p["idx"], **scan(p)), p["spool"]),
    "block_norm_fwd": lambda v, p: g.block_norm_fwd(v["x"], p["w"], v["z"], v["dO"], p["D"], p["w"]),
    "block_norm_bwd": lambda v, p: g.block_norm_bwd(v["x"], v["dO"], v["dt"], p["w"], v["z"], v["dO"], p["D"], p["w"]),
}


def tensors(out):
    vals = out.values() if isinstance(out, dict) else out
    return [t for t in vals if t is not None]


@pytest.mark.parametrize("name", list(CALLS))
def test_side_stream_orders_producer_call_and_consumer(name):
    """The token inputs hold NaN until a side stream, after milliseconds of other work, fills them;
    call and consumer follow on that stream. A launch anywhere else would read the NaN."""
    v, p = inputs()
    pools = {n: p[n].clone() for n in ("cpool", "spool")}
    want = [t.clone() for t in tensors(CALLS[name](v, p))]
    for n, t in pools.items():
        p[n].copy_(t)
    good = {n: t.clone() for n, t in v.items()}
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
