"""Host-side checks of the attention layer's operators: every call here is refused by the C ABI's
validation (or has nothing to do), so no kernel is launched and no device is needed."""
import ctypes
import os

import pytest
import torch

import gated_delta_rule_gdn_amd as g
from gated_delta_rule_gdn_amd.attention import AttentionDims, RotaryDims


def P(i):
    """A pointer that is never dereferenced: every call below fails validation."""
    return ctypes.c_void_p(0x1000 * i)


NULL, SHAPE, UNSUPPORTED, WORKSPACE = 1, 2, 3, 4


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(g.LIB_PATH):
        from gated_delta_rule_gdn_amd import build
        build.build()
    return g.lib()


def dims(cls, ok, **kw):
    return ctypes.byref(cls(**{**ok, **kw}))


ROTARY = dict(batch=2, seqlen=100, h_q=8, h_k=2, d=128, d_rot=64, interleaved=0, num_positions=512,
              dtype=1, grad_dtype=1, eps=1e-5, q_stride=0, k_stride=0, v_stride=0)


def fwd(L, q=P(1), k=P(2), cs=P(3), pos=P(4), qw=P(5), kw_=P(6), qo=P(2), ko=P(8), null=False, **kw):
    # q_out defaults to k's pointer: a call that passed every other check is still refused
    return L.gdn2_qk_rotary_fwd(q, k, cs, pos, qw, kw_, qo, ko,
                                None if null else dims(RotaryDims, ROTARY, **kw), None)


def test_rotary_forward_refusals(L):
    assert fwd(L, null=True) == NULL
    assert fwd(L, dtype=2) == UNSUPPORTED
    for d in (0, 1, 127, 514, -2):
        assert fwd(L, d=d, d_rot=0) == UNSUPPORTED
    assert fwd(L, d_rot=63) == SHAPE and fwd(L, d_rot=130) == SHAPE and fwd(L, d_rot=-2) == SHAPE
    assert fwd(L, h_q=0) == SHAPE and fwd(L, h_k=-1) == SHAPE and fwd(L, h_q=1 << 14) == SHAPE
    assert fwd(L, batch=-1) == SHAPE and fwd(L, seqlen=-1) == SHAPE
    assert fwd(L, batch=1 << 16, seqlen=1 << 15) == SHAPE
    assert fwd(L, num_positions=0) == SHAPE and fwd(L, num_positions=-1, d_rot=0) == SHAPE
    for eps in (-1.0, float("nan"), float("inf")):
        assert fwd(L, eps=eps) == SHAPE
    assert fwd(L, q_stride=1023) == SHAPE and fwd(L, k_stride=255) == SHAPE
    assert fwd(L, q_stride=1 << 40) == SHAPE and fwd(L, k_stride=-256) == SHAPE
    assert fwd(L, q=None) == NULL and fwd(L, k=None) == NULL and fwd(L, cs=None) == NULL
    assert fwd(L, qo=None) == NULL and fwd(L, qo=P(9), ko=None) == NULL
    assert fwd(L) == SHAPE and b"alias" in L.gdn2_last_error()
    assert fwd(L, qo=P(3)) == SHAPE and fwd(L, qo=P(8)) == SHAPE and fwd(L, qo=P(9), ko=P(1)) == SHAPE
    # in place, but not contiguous
    assert fwd(L, qo=P(1), q_stride=2048) == SHAPE and b"contiguous" in L.gdn2_last_error()
    assert fwd(L, qo=P(9), ko=P(2), k_stride=300) == SHAPE
    assert fwd(L, seqlen=0, q=None) == 0 and fwd(L, batch=0, q=None) == 0     # nothing to do


def test_rotary_strides_at_the_limit_of_a_tensor(L):
    top = (1 << 40) // (1 << 24)
    for name in ("q_stride", "k_stride"):
        for stride, status in ((top, b"alias"), (top + 1, b"stride"), (1 << 63 - 24, b"stride")):
            assert fwd(L, batch=1, seqlen=1 << 24, **{name: stride}) == SHAPE
            assert status in L.gdn2_last_error()


def bwd(L, dq=P(9), dk=P(10), dqw=P(1), dkw=P(12), ws=P(16), nbytes=1 << 30, dko=P(8), **kw):
    # dq_weight defaults to q's pointer
    return L.gdn2_qk_rotary_bwd(P(1), P(2), P(3), P(4), P(5), P(6), P(7), dko, dq, dk, dqw, dkw,
                                dims(RotaryDims, ROTARY, **kw), ws, nbytes, None)


def test_rotary_backward_refusals(L):
    need = L.gdn2_qk_rotary_bwd_workspace_bytes(dims(RotaryDims, ROTARY))
    assert need > 0 and need % (2 * 128 * 4) == 0
    assert L.gdn2_qk_rotary_bwd_workspace_bytes(dims(RotaryDims, ROTARY, d=7)) == 0
    assert L.gdn2_qk_rotary_bwd_workspace_bytes(None) == 0
    assert bwd(L, dtype=0) == UNSUPPORTED                            # fp32 inputs, bf16 gradients
    assert bwd(L, grad_dtype=3) == UNSUPPORTED
    assert bwd(L, dq=None) == NULL and bwd(L, dk=None) == NULL and bwd(L, dko=None) == NULL
    assert bwd(L, dqw=None) == NULL and bwd(L, dqw=P(11), dkw=None) == NULL
    assert bwd(L) == SHAPE
    assert bwd(L, dqw=P(11), dq=P(7)) == SHAPE                       # not in place
    assert bwd(L, dqw=P(11), dq=P(10)) == SHAPE
    assert bwd(L, dqw=P(11), ws=None) == WORKSPACE
    assert bwd(L, dqw=P(11), nbytes=need - 1) == WORKSPACE
    assert bwd(L, dqw=P(11), ws=ctypes.c_void_p(0x10080)) == WORKSPACE


def append(L, v=P(7), pos=P(4), slots=P(8), qo=P(2), kp=P(10), vp=P(11), pages=64, size=16, **kw):
    return L.gdn2_qk_rotary_append(P(1), P(2), v, P(3), pos, None, None, slots, qo, kp, vp, pages, size,
                                   dims(RotaryDims, ROTARY, **kw), None)


def test_rotary_append_refusals(L):
    assert append(L, d=3) == UNSUPPORTED
    assert append(L, h_k=0) == SHAPE
    assert append(L, pages=-1) == SHAPE and append(L, size=0) == SHAPE
    assert append(L, pages=1 << 16, size=1 << 15) == SHAPE           # 2^31 places
    assert append(L, pages=(1 << 31) - 1, size=1, h_k=8) == SHAPE    # 2^41 values
    assert append(L, v_stride=255) == SHAPE
    assert append(L, v=None) == NULL and append(L, pos=None) == NULL and append(L, slots=None) == NULL
    assert append(L, qo=P(9), kp=None) == NULL
    assert append(L) == SHAPE and b"alias" in L.gdn2_last_error()
    assert append(L, qo=P(9), vp=P(10)) == SHAPE and append(L, qo=P(9), kp=P(1)) == SHAPE
    assert append(L, qo=P(1), q_stride=2048) == SHAPE
    assert append(L, seqlen=0, v=None) == 0


ATTN = dict(num_seqs=4, new_tokens=1, h_q=8, h_k=2, d=128, num_pages=1000, page_size=16, max_pages=200,
            window=0, dtype=1, scale=0.1, q_stride=0)


def attn(L, q=P(1), kp=P(2), vp=P(3), table=P(4), lens=P(5), o=P(1), lse=None, ws=P(16), nbytes=1 << 40,
         null=False, **kw):
    return L.gdn2_paged_attention_step(q, kp, vp, table, lens, o, lse,
                                       None if null else dims(AttentionDims, ATTN, **kw), ws, nbytes, None)


def test_attention_refusals(L):
    assert attn(L, null=True) == NULL
    assert attn(L, dtype=2) == UNSUPPORTED
    for d in (0, 32, 96, 192, 512):
        assert attn(L, d=d) == UNSUPPORTED
    assert attn(L, num_seqs=-1) == SHAPE and attn(L, new_tokens=0) == SHAPE
    assert attn(L, h_q=0) == SHAPE and attn(L, h_k=0) == SHAPE and attn(L, h_k=3) == SHAPE
    assert attn(L, h_q=1 << 14) == SHAPE
    assert attn(L, num_seqs=1 << 20, new_tokens=1 << 11) == SHAPE
    assert attn(L, num_seqs=1 << 23) == SHAPE                        # workgroups
    assert attn(L, num_seqs=1, new_tokens=1 << 26, h_q=1, h_k=1) == SHAPE
    assert attn(L, num_seqs=1, new_tokens=1 << 20, h_q=16, h_k=1) == SHAPE
    assert attn(L, num_pages=-1) == SHAPE and attn(L, page_size=0) == SHAPE and attn(L, max_pages=-1) == SHAPE
    assert attn(L, num_pages=1 << 26) == SHAPE                       # 2^31 rows
    assert attn(L, page_size=(1 << 31) - 1) == SHAPE
    assert attn(L, max_pages=1 << 27) == SHAPE
    assert attn(L, window=-1) == SHAPE
    for scale in (float("nan"), float("inf")):
        assert attn(L, scale=scale) == SHAPE
    assert attn(L, q_stride=1023) == SHAPE and attn(L, q_stride=1 << 40) == SHAPE
    for name in ("q", "kp", "vp", "table", "lens", "o"):
        assert attn(L, **{name: None}) == NULL
    assert attn(L) == SHAPE and b"alias" in L.gdn2_last_error()
    assert attn(L, o=P(9), lse=P(9)) == SHAPE and attn(L, o=P(9), lse=P(2)) == SHAPE
    odd = ctypes.c_void_p(0x9008)
    assert attn(L, o=odd) == SHAPE and attn(L, o=P(9), kp=odd) == SHAPE and b"aligned" in L.gdn2_last_error()
    assert attn(L, num_seqs=0, q=None) == 0


def test_attention_workspace(L):
    need = L.gdn2_paged_attention_step_workspace_bytes(dims(AttentionDims, ATTN))
    assert need > 0
    assert attn(L, o=P(9), ws=None) == WORKSPACE and attn(L, o=P(9), nbytes=need - 1) == WORKSPACE
    assert attn(L, o=P(9), ws=ctypes.c_void_p(0x10080)) == WORKSPACE
    size = lambda **kw: L.gdn2_paged_attention_step_workspace_bytes(dims(AttentionDims, ATTN, **kw))  # noqa: E731
    assert size(d=96) == 0 and size(num_seqs=0) == 0
    assert size(max_pages=1) == 0                    # too short to be cut
    assert size(max_pages=20000) == need             # not a matter of the lengths
    assert size(num_pages=5) == need
    assert L.gdn2_paged_attention_step_workspace_bytes(None) == 0
    assert g.paged_attention_step_workspace_bytes(4, 1, 8, 2, 128, 16, 200, torch.bfloat16) == need


def test_attention_workspace_of_any_call(L):
    """The size without a window is enough for any window and for fewer sequences."""
    size = lambda **kw: L.gdn2_paged_attention_step_workspace_bytes(dims(AttentionDims, ATTN, **kw))  # noqa: E731
    for d in (64, 128, 256):
        for dtype in (0, 1):
            for T in (1, 4, 40):
                last = 0
                for n in (1, 2, 7, 31, 32, 33, 64, 100, 128, 129, 300, 1000, 5000):
                    whole = size(num_seqs=n, new_tokens=T, d=d, dtype=dtype)
                    assert whole >= last > -1
                    last = whole
                    for w in (1, 64, 250, 500, 1000, 2000, 100000):
                        assert size(num_seqs=n, new_tokens=T, d=d, dtype=dtype, window=w) <= whole
    assert size(num_seqs=200, h_q=8, h_k=4, window=1000) == 0 < size(num_seqs=2, h_q=8, h_k=4, window=1000)


def copy(L, pools=(0x1000, 0x2000), sizes=(64, 64), slots=10, src=P(8), dst=P(9), count=4, n=None):
    n = len(pools) if n is None else n
    return L.gdn2_pool_copy((ctypes.c_void_p * len(pools))(*pools), (ctypes.c_int64 * len(sizes))(*sizes), n, slots,
                            src, dst, count, None)


def test_pool_copy_refusals(L):
    assert copy(L, n=-1) == SHAPE and copy(L, slots=-1) == SHAPE and copy(L, count=-1) == SHAPE
    assert L.gdn2_pool_copy(None, None, 1, 1, P(8), P(9), 1, None) == NULL
    assert copy(L, sizes=(64, 0)) == SHAPE and copy(L, sizes=((1 << 32) + 1, 64)) == SHAPE
    assert copy(L, sizes=(1 << 32, 64), slots=1 << 11) == SHAPE
    assert copy(L, pools=(0x1000, 0)) == NULL
    assert copy(L, pools=(0x1000, 0x1000)) == SHAPE
    assert copy(L, src=None) == NULL and copy(L, dst=None) == NULL
    assert copy(L, pools=(0x1000, 0x8000)) == SHAPE and copy(L, pools=(0x9000,), sizes=(4,)) == SHAPE
    assert copy(L, count=0, src=None) == 0 and copy(L, n=0) == 0 and copy(L, slots=0) == 0
    assert copy(L, src=P(8), dst=P(8)) == 0          # every slot onto itself


def test_calls_need_gpu_tensors():
    x = torch.zeros(1, 4, 2, 64)
    cs = torch.zeros(8, 64)
    i = torch.zeros(1, 4, dtype=torch.int32)
    for call in (lambda: g.qk_rotary_fwd(x, x, cs), lambda: g.qk_rotary_bwd(x, x, cs, x, x),
                 lambda: g.qk_rotary_append(x, x, x, cs, i, x, x, i),
                 lambda: g.paged_attention_step(x, x, x, i, i[0]),
                 lambda: g.pool_copy(x, i[0], i[0])):
        with pytest.raises(ValueError, match="GPU"):
            call()


def test_rotary_table():
    t = g.rotary_table(5, 6, base=100.0)
    assert t.shape == (5, 6) and t.dtype == torch.float32
    angle = torch.arange(5, dtype=torch.float64)[:, None] * torch.tensor([1.0, 100 ** (-1 / 3), 100 ** (-2 / 3)],
                                                                         dtype=torch.float64)
    # the exponent and the power in 64 bits, rounded once to 32
    assert torch.allclose(t.double(), torch.cat((angle.cos(), angle.sin()), 1), rtol=0, atol=2.0 ** -24 + 1e-14)
    assert g.rotary_table(3, 0).shape == (3, 0)
    with pytest.raises(ValueError):
        g.rotary_table(3, 5)
