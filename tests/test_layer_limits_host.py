"""Sizes at the limits of the operators around the recurrence: each call is refused by the C ABI's
validation, or would be but for its size, so no kernel is launched and no device is needed."""
import ctypes
import os

import pytest

import gated_delta_rule_gdn_amd as g
from gated_delta_rule_gdn_amd.layer import ConvDims, NormDims, ScanDims

SHAPE = 2
LARGE, ALIAS = b"too large", b"alias"


def P(i):
    """A pointer that is never dereferenced: every call below fails validation."""
    return ctypes.c_void_p(0x1000 * i)


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(g.LIB_PATH):
        from gated_delta_rule_gdn_amd import build
        build.build()
    return g.lib()


# y, o and h are x's pointer, so that a call whose sizes are accepted is still refused


def conv(L, tokens, stride, batch=1):
    d = ConvDims(batch=batch, seqlen=tokens, channels=8, width=4, dtype=1, grad_dtype=1, x_stride=stride)
    st = L.gdn2_short_conv_fwd(P(1), P(2), None, None, None, P(1), None, ctypes.byref(d), None)
    return st, L.gdn2_last_error()


def scan(L, tokens, **strides):
    d = ScanDims(batch=1, seqlen=tokens, channels=8, d_state=16, groups=1, dtype=1, grad_dtype=1, **strides)
    st = L.gdn2_selective_scan_fwd(P(1), P(2), P(3), P(4), P(5), None, None, None, None, None, P(1), None,
                                   ctypes.byref(d), None, 0, None)
    return st, L.gdn2_last_error()


def norm(L, rows, **strides):
    d = NormDims(rows=rows, d=64, dtype=1, residual_dtype=1, grad_dtype=1, eps=1e-5, **strides)
    st = L.gdn2_block_norm_fwd(P(1), None, None, None, None, None, P(1), None, ctypes.byref(d), None)
    return st, L.gdn2_last_error()


@pytest.mark.parametrize("tokens,stride", [
    (1 << 24, 1 << 40),             # the product is 2^64
    (3 << 23, 1 << 40), (1 << 30, 1 << 35), ((1 << 30) - 1, 1 << 40),
    (1 << 20, (1 << 20) + 1), (1, (1 << 40) + 1), (1, (1 << 63) - 1)])
def test_strides_that_reach_too_far_are_refused(L, tokens, stride):
    for st, why in (conv(L, tokens, stride), scan(L, tokens, x_stride=stride), scan(L, tokens, dt_stride=stride),
                    scan(L, tokens, b_stride=stride), scan(L, tokens, c_stride=stride),
                    scan(L, tokens, gate_stride=stride), norm(L, tokens, x_stride=stride),
                    norm(L, tokens, gate_stride=stride)):
        assert st == SHAPE and LARGE in why, why


@pytest.mark.parametrize("tokens,stride", [(1 << 20, 1 << 20), (1 << 30, 1 << 10), (1, 1 << 40)])
def test_the_largest_strides_are_accepted(L, tokens, stride):
    for st, why in (conv(L, tokens, stride), scan(L, tokens, x_stride=stride), norm(L, tokens, x_stride=stride)):
        assert st == SHAPE and ALIAS in why, why
