"""Gradients of steps that a mask takes out (dt of -inf or the lowest value: the step and its slope
are zero) beside rates of -inf."""
import numpy as np
import pytest
import torch

import gated_delta_rule_gdn_amd as g
from layer_common import check, f64, scan_bwd_ref
from test_gpu_selective_scan import Draw, cu_of, gpu, make
from test_gpu_selective_scan_bwd import call, flat, ref_args

pytestmark = pytest.mark.gpu


def setup_module(module):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    g.lib()


@pytest.mark.parametrize("low", [float("-inf"), -3e38, -1e4])
@pytest.mark.parametrize("M", [4, 16, 40])
def test_masked_steps_take_no_gradient_whatever_the_rate(M, low):
    """States of size 100 make the product of a state, its gradient and a rate of -inf pass the
    range of fp32; it is of no step."""
    lens = [190, 10]
    h = make((1, 200), 10, M, 1, 2, torch.float32, seed=22)
    h["A"][3, 2], h["A"][7, 0] = float("-inf"), -3e38
    h["S0"] *= 100
    h["dt"][:, 20:30] = low
    h["dt"][:, 40:180] = low
    q = Draw(23)
    dO, dS = q.normal(1, 200, 10), q.normal(2, 10, M)
    d = gpu(h)
    o = call(d, dO.cuda(), dS.cuda(), cu_seqlens=cu_of(lens))
    torch.cuda.synchronize()
    assert torch.all(o["ddt"][:, 20:30] == 0) and torch.all(o["ddt"][:, 40:180] == 0)
    assert all(torch.isfinite(t).all() for t in o.values())
    v = flat({**h, "dt": h["dt"].clamp(min=-300.0), "A": h["A"].clamp(min=-1e30)}, 200)
    r = scan_bwd_ref(*ref_args(v, True, lens), f64(dO)[0], f64(dS))
    # in 64 bits a step of 1e-130 times a rate of -1e30 is as good as none
    assert np.all(np.abs(r["ddt"][20:30]) < 1e-90)
    keep = [c for c in range(10) if c not in (3, 7)]
    for n in ("dx", "dB", "dC", "dgate", "ddt"):
        check(n, o[n][0], r[n], r[n + "_b"])
    check("ddt_bias", o["ddt_bias"], r["ddt_bias"], r["ddt_bias_b"])
    check("dA", o["dA"][keep], r["dA"][keep], r["dA_b"][keep])
