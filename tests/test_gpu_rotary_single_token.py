"""One token of one request, sliced from a batch's projection: whatever its strides say, it is contiguous, so
its queries and keys may be their own outputs."""
import pytest
import torch

import gated_delta_rule_gdn_amd as g
from test_gpu_rotary import EPS, make

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16


def setup_module(module):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    g.lib()


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("pad,shift", [(0, 0), (16, 8), (3, 1)])
def test_one_token_in_place(pad, shift, dtype):
    v = {n: t[:1] if n in ("q", "k", "v", "pos") else t
         for n, t in make(1, 2, 1, 4, 2, 64, 32, dtype, pad=pad, shift=shift).items()}
    q, k = v["q"], v["k"]
    assert q.is_contiguous() and q.stride(0) > 4 * 64
    kp = torch.zeros(2, 2, 4, 64, dtype=dtype, device="cuda")
    vp, slot = torch.zeros_like(kp), torch.tensor([[5]], dtype=torch.int32, device="cuda")
    before, want = (q.clone(), k.clone()), g.qk_rotary_fwd(q, k, v["cs"], v["pos"], v["qw"], v["kw"], eps=EPS)
    got = g.qk_rotary_fwd(q, k, v["cs"], v["pos"], v["qw"], v["kw"], eps=EPS, q_out=q, k_out=k)
    assert got[0] is q and got[1] is k and torch.equal(q, want[0]) and torch.equal(k, want[1])
    q.copy_(before[0])
    k.copy_(before[1])
    got = g.qk_rotary_append(q, k, v["v"], v["cs"], v["pos"], kp, vp, slot, v["qw"], v["kw"], eps=EPS, q_out=q)
    assert got is q and torch.equal(q, want[0])
    assert torch.equal(kp[1, :, 1], want[1][0, 0]) and torch.equal(vp[1, :, 1], v["v"][0, 0]) and torch.equal(k, before[1])
