"""Queries alone, with keys of no heads or a weight for keys that are not there: the queries' outputs and
gradients are what they are without, and the weight's gradient is zeros."""
import ctypes

import pytest
import torch

import gated_delta_rule_gdn_amd as g
from gated_delta_rule_gdn_amd.attention import RotaryDims
from test_gpu_rotary import EPS, make

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16


def setup_module(module):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    g.lib()


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("qw", [True, False])
@pytest.mark.parametrize("d,rot", [(64, 64), (10, 4), (256, 64)])
@pytest.mark.parametrize("T", [1, 37, 5000])
def test_gradient_of_a_weight_without_keys_is_zero(T, d, rot, qw, dtype):
    v = make(T + d, 1, T, 3, 1, d, rot, dtype, weights=(qw, True))
    dq = v["dq"].to(dtype).cuda()
    want = g.qk_rotary_bwd(v["q"], None, v["cs"], dq, positions=v["pos"], q_weight=v["qw"], eps=EPS)
    nothing = torch.empty(1, T, 0, d, dtype=dtype, device="cuda")
    for k, dk in ((None, None), (nothing, nothing.clone())):
        nan = torch.full((d,), float("nan"), device="cuda")      # what the allocator may hand out next
        del nan
        out = g.qk_rotary_bwd(v["q"], k, v["cs"], dq, dk, positions=v["pos"], q_weight=v["qw"], k_weight=v["kw"], eps=EPS)
        assert set(out) == set(want) | {"dk_weight"} | ({"dk"} if k is not None else set())
        assert torch.equal(out["dk_weight"], torch.zeros(d, device="cuda"))
        assert all(torch.equal(out[n], want[n]) for n in want)
        if k is not None:
            assert out["dk"].shape == k.shape


def test_every_output_is_written_whatever_the_workspace_holds():
    """The C call with outputs and a workspace of NaN; and without a dk_weight, which is not needed then."""
    T, d = 37, 64
    v = make(1, 1, T, 3, 1, d, 32, F32)
    q, dq = v["q"].contiguous(), v["dq"].cuda()
    dims = RotaryDims(1, T, 3, 0, d, 32, 0, v["cs"].shape[0], 0, 0, EPS, 0, 0, 0)
    need = g.lib().gdn2_qk_rotary_bwd_workspace_bytes(ctypes.byref(dims))
    nan = lambda *s: torch.full(s, float("nan"), device="cuda")  # noqa: E731
    for asked in (True, False):
        ws, dqo, dqw, dkw = nan(need // 4), nan(1, T, 3, d), nan(d), nan(d)
        st = g.lib().gdn2_qk_rotary_bwd(
            q.data_ptr(), None, v["cs"].data_ptr(), v["pos"].data_ptr(), v["qw"].data_ptr(), v["kw"].data_ptr(),
            dq.data_ptr(), None, dqo.data_ptr(), None, dqw.data_ptr(), dkw.data_ptr() if asked else None,
            ctypes.byref(dims), ws.data_ptr(), need, torch.cuda.current_stream().cuda_stream)
        assert st == 0, g.lib().gdn2_last_error()
        want = g.qk_rotary_bwd(q, None, v["cs"], dq, positions=v["pos"], q_weight=v["qw"], eps=EPS)
        assert torch.equal(dqo, want["dq"]) and torch.equal(dqw, want["dq_weight"])
        assert torch.equal(dkw, torch.zeros_like(dkw)) if asked else torch.isnan(dkw).all()


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("B,T", [(1, 1), (2, 37)])
def test_forward_with_keys_of_no_heads(B, T, dtype):
    v = make(T, B, T, 3, 1, 64, 32, dtype)
    want, _ = g.qk_rotary_fwd(v["q"], None, v["cs"], v["pos"], v["qw"], eps=EPS)
    nothing = torch.empty(B, T, 0, 64, dtype=dtype, device="cuda")
    for kw in (None, v["kw"]):
        q, k = g.qk_rotary_fwd(v["q"], nothing, v["cs"], v["pos"], v["qw"], kw, eps=EPS)
        assert torch.equal(q, want) and k.shape == nothing.shape
    q = v["q"].contiguous()
    assert g.qk_rotary_fwd(q, nothing, v["cs"], v["pos"], v["qw"], eps=EPS, q_out=q)[0] is q and torch.equal(q, want)
