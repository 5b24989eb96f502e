"""Host-side checks of the operators around the recurrence: every call here is refused by the
C ABI's validation (or has nothing to do), so no kernel is launched and no device is needed."""
import ctypes
import os

import pytest

import gated_delta_rule_gdn_amd as g
from gated_delta_rule_gdn_amd.layer import ConvDims, NormDims, ScanDims


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


CONV = dict(batch=2, seqlen=100, num_seqs=0, channels=64, width=4, dtype=1, grad_dtype=1, silu=1,
            x_stride=0)


def conv_fwd(L, cu=None, x=P(1), w=P(2), y=P(1), state0=None, state_T=None, null=False, **kw):
    # y defaults to x's pointer: a call that passed every other check is still refused
    return L.gdn2_short_conv_fwd(x, w, None, state0, cu, y, state_T,
                                 None if null else dims(ConvDims, CONV, **kw), None)


def test_short_conv_forward_refusals(L):
    assert conv_fwd(L, null=True) == NULL
    assert conv_fwd(L, dtype=2) == UNSUPPORTED
    assert conv_fwd(L, width=1) == UNSUPPORTED and conv_fwd(L, width=5) == UNSUPPORTED
    assert conv_fwd(L, channels=0) == SHAPE and conv_fwd(L, channels=(1 << 20) + 1) == SHAPE
    assert conv_fwd(L, seqlen=-1) == SHAPE and conv_fwd(L, batch=0) == SHAPE
    assert conv_fwd(L, batch=1 << 16, seqlen=1 << 15) == SHAPE
    assert conv_fwd(L, x_stride=63) == SHAPE and conv_fwd(L, x_stride=-64) == SHAPE
    assert conv_fwd(L, x_stride=1 << 40) == SHAPE
    assert conv_fwd(L, cu=P(9)) == SHAPE                             # packed needs batch = 1
    assert conv_fwd(L, cu=P(9), batch=1, num_seqs=0) == SHAPE
    assert conv_fwd(L, x=None) == NULL and conv_fwd(L, w=None) == NULL
    assert conv_fwd(L, y=None) == NULL
    assert conv_fwd(L) == SHAPE and b"alias" in L.gdn2_last_error()
    assert conv_fwd(L, y=P(3), state0=P(4), state_T=P(4)) == SHAPE   # not in place
    assert conv_fwd(L, seqlen=0, x=None, y=None) == 0                # nothing to do


def conv_bwd(L, ws=P(16), nbytes=1 << 30, dw=P(2), bias=None, dbias=None, **kw):
    # dweight defaults to weight's pointer
    return L.gdn2_short_conv_bwd(P(1), P(2), bias, None, None, P(3), None, P(4), dw, dbias, None,
                                 dims(ConvDims, CONV, **kw), ws, nbytes, None)


def test_short_conv_backward_refusals(L):
    need = L.gdn2_short_conv_bwd_workspace_bytes(dims(ConvDims, CONV))
    assert need > 0 and need % (64 * 5 * 4) == 0
    assert L.gdn2_short_conv_bwd_workspace_bytes(dims(ConvDims, CONV, width=7)) == 0
    assert L.gdn2_short_conv_bwd_workspace_bytes(None) == 0
    assert conv_bwd(L, dtype=0) == UNSUPPORTED                       # fp32 inputs, bf16 gradients
    assert conv_bwd(L, dw=None) == NULL
    assert conv_bwd(L, dw=P(5), bias=P(6)) == NULL                   # a bias without dbias
    assert conv_bwd(L) == SHAPE
    assert conv_bwd(L, dw=P(5), ws=None) == WORKSPACE
    assert conv_bwd(L, dw=P(5), nbytes=need - 1) == WORKSPACE
    assert conv_bwd(L, dw=P(5), ws=ctypes.c_void_p(0x10080)) == WORKSPACE
    assert conv_bwd(L, dw=P(4)) == SHAPE                             # dx and dweight


def conv_step(L, slots=8, st=P(3), idx=None, y=P(1), **kw):
    return L.gdn2_short_conv_step(P(1), P(2), None, st, idx, slots, y, dims(ConvDims, CONV, **kw), None)


def test_short_conv_step_refusals(L):
    assert conv_step(L) == SHAPE                                     # y aliases x
    assert conv_step(L, y=P(3)) == SHAPE                             # y aliases the state
    assert conv_step(L, y=P(4), slots=1) == SHAPE
    assert conv_step(L, y=P(4), slots=-1, idx=P(5)) == SHAPE
    assert conv_step(L, y=P(4), seqlen=0) == SHAPE
    assert conv_step(L, y=P(4), st=None) == NULL
    assert conv_step(L, y=None) == NULL
    assert conv_step(L, width=9, batch=0) == UNSUPPORTED
    assert conv_step(L, batch=0) == 0                                # an empty batch


SCAN = dict(batch=2, seqlen=300, num_seqs=0, channels=64, d_state=16, groups=2, dtype=1, grad_dtype=1,
            dt_softplus=1, x_stride=0, dt_stride=0, b_stride=0, c_stride=0, gate_stride=0)


def scan_fwd(L, cu=None, o=P(1), S0=None, S_T=None, ws=P(16), nbytes=1 << 30, x=P(1), null=False, **kw):
    # o defaults to x's pointer: a call that passed every other check is still refused
    return L.gdn2_selective_scan_fwd(x, P(2), P(3), P(4), P(5), None, None, None, S0, cu, o, S_T,
                                     None if null else dims(ScanDims, SCAN, **kw), ws, nbytes, None)


def test_selective_scan_forward_refusals(L):
    assert scan_fwd(L, null=True) == NULL
    assert scan_fwd(L, dtype=5) == UNSUPPORTED
    assert scan_fwd(L, d_state=0) == SHAPE and scan_fwd(L, d_state=129) == UNSUPPORTED
    assert scan_fwd(L, groups=0) == SHAPE and scan_fwd(L, groups=3) == SHAPE
    assert scan_fwd(L, channels=0) == SHAPE
    assert scan_fwd(L, batch=1 << 20, seqlen=1 << 12) == SHAPE
    assert scan_fwd(L, b_stride=31) == SHAPE and scan_fwd(L, gate_stride=-1) == SHAPE
    assert scan_fwd(L, cu=P(9)) == SHAPE
    assert scan_fwd(L, x=None) == NULL and scan_fwd(L, o=None) == NULL
    assert scan_fwd(L) == SHAPE and b"alias" in L.gdn2_last_error()
    assert scan_fwd(L, o=P(6), S0=P(7), S_T=P(7)) == SHAPE
    need = L.gdn2_selective_scan_fwd_workspace_bytes(dims(ScanDims, SCAN))
    assert need > 0
    assert scan_fwd(L, o=P(6), ws=None) == WORKSPACE
    assert scan_fwd(L, o=P(6), nbytes=need - 1) == WORKSPACE
    assert scan_fwd(L, o=P(6), ws=ctypes.c_void_p(0x10010)) == WORKSPACE
    assert scan_fwd(L, seqlen=0, x=None, o=None) == 0
    assert L.gdn2_selective_scan_fwd_workspace_bytes(dims(ScanDims, SCAN, groups=3)) == 0
    # one sequence per tile, or one tile: no workspace
    assert L.gdn2_selective_scan_fwd_workspace_bytes(dims(ScanDims, SCAN, batch=1024)) == 0
    assert L.gdn2_selective_scan_fwd_workspace_bytes(dims(ScanDims, SCAN, batch=1, seqlen=9)) == 0


def scan_step(L, o=P(1), st=P(6), sdt=0, slots=8, idx=None, **kw):
    return L.gdn2_selective_scan_step(P(1), P(2), P(3), P(4), P(5), None, None, None, st, sdt, idx,
                                      slots, o, dims(ScanDims, {**SCAN, "seqlen": 1}, **kw), None)


def test_selective_scan_step_refusals(L):
    assert scan_step(L) == SHAPE and scan_step(L, o=P(6)) == SHAPE
    assert scan_step(L, o=P(7), sdt=2) == UNSUPPORTED
    assert scan_step(L, o=P(7), seqlen=0) == SHAPE
    assert scan_step(L, o=P(7), slots=1) == SHAPE
    assert scan_step(L, o=P(7), st=None) == NULL
    assert scan_step(L, batch=0, groups=5) == SHAPE
    assert scan_step(L, batch=0) == 0


NORM = dict(rows=10, d=64, dtype=1, residual_dtype=1, grad_dtype=1, eps=1e-5, x_stride=0, gate_stride=0)


def norm_fwd(L, x=P(1), h=P(1), res=None, nxt=None, y=None, **kw):
    # h defaults to x's pointer: a call that passed every other check is still refused
    return L.gdn2_block_norm_fwd(x, None, res, None, None, nxt, h, y, dims(NormDims, NORM, **kw), None)


def test_block_norm_forward_refusals(L):
    assert L.gdn2_block_norm_fwd(*[P(1)] * 8, None, None) == NULL
    assert norm_fwd(L, dtype=3) == UNSUPPORTED
    assert norm_fwd(L, dtype=0) == UNSUPPORTED                       # fp32 x, bf16 residual
    assert norm_fwd(L, residual_dtype=2) == UNSUPPORTED
    assert norm_fwd(L, d=0) == SHAPE and norm_fwd(L, d=16385) == UNSUPPORTED
    assert norm_fwd(L, rows=-1) == SHAPE and norm_fwd(L, rows=1 << 31) == SHAPE
    assert norm_fwd(L, eps=-1.0) == SHAPE and norm_fwd(L, eps=float("nan")) == SHAPE
    assert norm_fwd(L, x_stride=63) == SHAPE and norm_fwd(L, gate_stride=-1) == SHAPE
    assert norm_fwd(L, x=None) == NULL and norm_fwd(L, h=None) == NULL
    assert norm_fwd(L, h=P(2), nxt=P(3)) == NULL                     # y is missing
    assert norm_fwd(L) == SHAPE
    assert norm_fwd(L, h=P(2), res=P(4), nxt=P(3), y=P(4)) == SHAPE  # y over the residual
    assert norm_fwd(L, rows=0) == 0


def norm_bwd(L, dx=P(1), dh=P(9), nw=P(2), dnw=P(3), nxt=None, dy=None, gate=None, ws=P(16), nbytes=1 << 30, **kw):
    return L.gdn2_block_norm_bwd(P(1), gate, None, nw, None, nxt, dh, dy, dx, None, None, dnw, None, None,
                                 dims(NormDims, NORM, **kw), ws, nbytes, None)


def test_block_norm_backward_refusals(L):
    need = L.gdn2_block_norm_bwd_workspace_bytes(dims(NormDims, NORM))
    assert need > 0 and L.gdn2_block_norm_bwd_workspace_bytes(dims(NormDims, NORM, d=0)) == 0
    assert norm_bwd(L, grad_dtype=2) == UNSUPPORTED
    assert norm_bwd(L) == SHAPE                                      # dx aliases x
    assert norm_bwd(L, dx=None) == NULL and norm_bwd(L, dx=P(8), dh=None) == NULL
    assert norm_bwd(L, dx=P(8), nxt=P(5)) == NULL                    # dy is missing
    assert norm_bwd(L, dx=P(8), gate=P(5)) == NULL                   # dgate is missing
    assert norm_bwd(L, dx=P(8), dnw=None) == NULL
    assert norm_bwd(L, dx=P(8), ws=None) == WORKSPACE
    assert norm_bwd(L, dx=P(8), nbytes=need - 1) == WORKSPACE
    assert norm_bwd(L, dx=P(8), ws=ctypes.c_void_p(0x10040)) == WORKSPACE


def scan_bwd(L, dx=P(1), dA=P(11), D=None, dD=None, gate=None, ws=P(16), nbytes=1 << 34, dS0=None, **kw):
    # dx defaults to x's pointer
    return L.gdn2_selective_scan_bwd(P(1), P(2), P(3), P(4), P(5), D, gate, None, None, None, P(9), None,
                                     dx, P(10), dA, P(12), P(13), dD, None, None, dS0,
                                     dims(ScanDims, SCAN, **kw), ws, nbytes, None)


def test_selective_scan_backward_refusals(L):
    need = L.gdn2_selective_scan_bwd_workspace_bytes(dims(ScanDims, SCAN))
    assert need > 0 and L.gdn2_selective_scan_bwd_workspace_bytes(dims(ScanDims, SCAN, d_state=200)) == 0
    assert scan_bwd(L, dtype=0) == UNSUPPORTED
    assert scan_bwd(L) == SHAPE
    assert scan_bwd(L, dx=None) == NULL and scan_bwd(L, dx=P(6), dA=None) == NULL
    assert scan_bwd(L, dx=P(6), D=P(7)) == NULL and scan_bwd(L, dx=P(6), gate=P(7)) == NULL
    assert scan_bwd(L, dx=P(6), dS0=P(6)) == SHAPE
    assert scan_bwd(L, dx=P(6), ws=None) == WORKSPACE
    assert scan_bwd(L, dx=P(6), nbytes=need - 1) == WORKSPACE
    assert scan_bwd(L, dx=P(6), ws=ctypes.c_void_p(0x10008)) == WORKSPACE


def test_sizes_beyond_32_bits_are_refused():
    """Python's sizes are checked before they go into the 32-bit fields of the dims."""
    from gated_delta_rule_gdn_amd import layer
    assert layer._fits("n", (1 << 31) - 1) == (1 << 31) - 1
    with pytest.raises(ValueError, match="the number of tokens"):
        layer._fits("the number of tokens", 1 << 31)
