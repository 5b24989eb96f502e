"""Host-side checks of the operators around the recurrence: every call here is refused by the
C ABI's validation (or has nothing to do), so no kernel is launched and no device is needed."""
import ctypes
import os

import pytest

import gated_delta_rule_gdn_amd as g
from gated_delta_rule_gdn_amd.layer import ConvDims


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
