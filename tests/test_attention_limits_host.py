"""Every refusal of the attention layer's calls by the reason it gives, and beside each limit the largest
call that is within it. Calls that pass all other checks are refused for an output that is an input, so no
kernel is launched and no device is needed."""
import ctypes
import os

import pytest

import gated_delta_rule_gdn_amd as g
from gated_delta_rule_gdn_amd.attention import AttentionDims, RotaryDims

OK, NULL, SHAPE, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3, 4
NAN, INF = float("nan"), float("inf")


def P(i):
    """A pointer that is never dereferenced: every call below fails validation."""
    return ctypes.c_void_p(0x1000 * i)


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(g.LIB_PATH):
        from gated_delta_rule_gdn_amd import build
        build.build()
    return g.lib()


def refused(L, status, why, code):
    assert status == code and why.encode() in L.gdn2_last_error(), (status, L.gdn2_last_error(), why)


ROTARY = dict(batch=2, seqlen=100, h_q=8, h_k=2, d=128, d_rot=64, interleaved=0, num_positions=512,
              dtype=1, grad_dtype=1, eps=1e-5, q_stride=0, k_stride=0, v_stride=0)


def fwd(L, q=P(1), k=P(2), cs=P(3), pos=P(4), qw=P(5), kw=P(6), qo=P(3), ko=P(8), **sizes):
    return L.gdn2_qk_rotary_fwd(q, k, cs, pos, qw, kw, qo, ko, ctypes.byref(RotaryDims(**{**ROTARY, **sizes})), None)


def bwd(L, q=P(1), k=P(2), cs=P(3), pos=P(4), qw=P(5), kw=P(6), dqo=P(7), dko=P(8), dq=P(9), dk=P(10), dqw=P(3),
        dkw=P(12), ws=P(16), nbytes=1 << 30, **sizes):
    return L.gdn2_qk_rotary_bwd(q, k, cs, pos, qw, kw, dqo, dko, dq, dk, dqw, dkw,
                                ctypes.byref(RotaryDims(**{**ROTARY, **sizes})), ws, nbytes, None)


def append(L, q=P(1), k=P(2), v=P(7), cs=P(3), pos=P(4), qw=P(5), kw=P(6), slots=P(8), qo=P(3), kp=P(10), vp=P(11),
           pages=64, size=16, **sizes):
    return L.gdn2_qk_rotary_append(q, k, v, cs, pos, qw, kw, slots, qo, kp, vp, pages, size,
                                   ctypes.byref(RotaryDims(**{**ROTARY, **sizes})), None)


TOKENS, DHEAD, DROT, HEADS = "2^30 tokens", "d must be even", "d_rot must be even", "h_q must be >= 1"
VALUES, POSITIONS, EPS, STRIDE = "2^20 values", "num_positions must be", "eps must be", "a stride is smaller"
BATCH, ALIAS = "batch and seqlen must be", "aliases an input"

ROTARY_REFUSALS = [
    (dict(dtype=2), "dtype must be", UNSUPPORTED), (dict(dtype=-1), "dtype must be", UNSUPPORTED),
    (dict(batch=-1), BATCH, SHAPE), (dict(seqlen=-1), BATCH, SHAPE),
    (dict(batch=1 << 16, seqlen=1 << 15), TOKENS, SHAPE), (dict(batch=(1 << 30) + 1, seqlen=1), TOKENS, SHAPE),
    *[(dict(d=d, d_rot=0), DHEAD, UNSUPPORTED) for d in (0, 1, 127, 513, 514, -2)],
    *[(dict(d_rot=r), DROT, SHAPE) for r in (63, 130, -2)],
    (dict(h_q=0), HEADS, SHAPE), (dict(h_k=-1), HEADS, SHAPE),
    (dict(h_q=(1 << 13) + 1), VALUES, SHAPE), (dict(h_k=(1 << 13) + 1), VALUES, SHAPE),
    (dict(num_positions=0), POSITIONS, SHAPE), (dict(num_positions=-1, d_rot=0), POSITIONS, SHAPE),
    *[(dict(eps=e), EPS, SHAPE) for e in (-1.0, -1e-30, NAN, INF, 1e31)],
    (dict(q_stride=1023), STRIDE, SHAPE), (dict(k_stride=255), STRIDE, SHAPE), (dict(v_stride=255), STRIDE, SHAPE),
    *[({n: s}, STRIDE, SHAPE) for n in ("q_stride", "k_stride", "v_stride")
      for s in (-1, -4096, (1 << 40) // 200 + 1, 1 << 40, (1 << 63) - 1)],
]
ROTARY_ACCEPTED = [
    dict(dtype=0, grad_dtype=0), dict(batch=1 << 15, seqlen=1 << 15, h_q=1, h_k=1), dict(batch=1 << 30, seqlen=1, h_q=1, h_k=1),
    dict(d=2, d_rot=2), dict(d=512, d_rot=512), dict(d_rot=0), dict(d_rot=128), dict(h_q=1, h_k=1),
    dict(h_q=1 << 13), dict(h_k=1 << 13), dict(num_positions=1), dict(num_positions=0, d_rot=0), dict(eps=0.0), dict(eps=9e29),
    dict(q_stride=1024, k_stride=256, v_stride=256), *[{n: (1 << 40) // 200} for n in ("q_stride", "k_stride", "v_stride")],
]


@pytest.mark.parametrize("call", [fwd, bwd, append])
def test_rotary_sizes(L, call):
    for sizes, why, code in ROTARY_REFUSALS:
        if call is bwd and "dtype" in sizes:
            sizes = {**sizes, "grad_dtype": 0}
        refused(L, call(L, **sizes), why, code)
    for sizes in ROTARY_ACCEPTED:
        refused(L, call(L, **sizes), ALIAS, SHAPE)


def test_rotary_without_keys(L):
    refused(L, fwd(L, h_k=0, k=None, ko=None), ALIAS, SHAPE)
    refused(L, bwd(L, h_k=0, k=None, dko=None, dk=None, dkw=None), ALIAS, SHAPE)
    refused(L, append(L, h_k=0), "h_k must be >= 1", SHAPE)


def test_rotary_gradient_types(L):
    refused(L, bwd(L, dtype=0, grad_dtype=1), "grad_dtype must be", UNSUPPORTED)
    refused(L, bwd(L, grad_dtype=2), "grad_dtype must be", UNSUPPORTED)
    refused(L, bwd(L, grad_dtype=0), ALIAS, SHAPE)
    refused(L, bwd(L, dtype=0, grad_dtype=0), ALIAS, SHAPE)


def test_rotary_forward_tensors(L):
    for name in ("q", "k", "cs", "qo", "ko"):
        refused(L, fwd(L, **{name: None}), "are required", NULL)
    refused(L, fwd(L, cs=None, d_rot=0, qo=P(4)), ALIAS, SHAPE)      # no table without a rotation
    for qo in (2, 3, 4, 5, 6, 8):
        refused(L, fwd(L, qo=P(qo)), ALIAS, SHAPE)
    for ko in (1, 3, 4, 5, 6):
        refused(L, fwd(L, qo=P(9), ko=P(ko)), ALIAS, SHAPE)
    refused(L, fwd(L, qo=P(1), q_stride=2048), "only a contiguous input", SHAPE)
    refused(L, fwd(L, qo=P(9), ko=P(2), k_stride=300), "only a contiguous input", SHAPE)
    assert fwd(L, batch=0, q=None) == OK and fwd(L, seqlen=0, q=None) == OK


def test_rotary_backward_tensors(L):
    for name in ("q", "k", "cs", "dqo", "dko", "dq", "dk"):
        refused(L, bwd(L, **{name: None}), "incoming gradients", NULL)
    for name in ("dqw", "dkw"):
        refused(L, bwd(L, **{name: None}), "every weight needs", NULL)
    for out in ("dq", "dk", "dqw", "dkw"):
        for i in (1, 2, 3, 4, 5, 6, 7, 8, 16):
            refused(L, bwd(L, **{"dqw": P(11), out: P(i)}), ALIAS, SHAPE)
    refused(L, bwd(L, dqw=P(11), dq=P(10)), ALIAS, SHAPE)
    refused(L, bwd(L, dqw=P(12)), ALIAS, SHAPE)
    need = L.gdn2_qk_rotary_bwd_workspace_bytes(ctypes.byref(RotaryDims(**ROTARY)))
    refused(L, bwd(L, dqw=P(11), ws=None), "workspace is NULL", WORKSPACE)
    refused(L, bwd(L, dqw=P(11), nbytes=need - 1), "too small", WORKSPACE)
    refused(L, bwd(L, dqw=P(11), ws=ctypes.c_void_p(0x10080)), "256-byte", WORKSPACE)
    assert bwd(L, batch=0, qw=None, kw=None, ws=None) == OK


def test_rotary_append_pages(L):
    refused(L, append(L, pages=-1), "num_pages must be >= 0", SHAPE)
    refused(L, append(L, size=0), "num_pages must be >= 0", SHAPE)
    places = "num_pages * page_size must be"
    refused(L, append(L, pages=1 << 16, size=1 << 15, h_k=1, d=2, d_rot=2), places, SHAPE)
    refused(L, append(L, pages=(1 << 31) - 1, size=1, h_k=1, d=2, d_rot=2), ALIAS, SHAPE)
    refused(L, append(L, pages=1 << 30, size=1, h_k=8, d=128), ALIAS, SHAPE)              # 2^40 values
    refused(L, append(L, pages=(1 << 30) + 1, size=1, h_k=8, d=128), places, SHAPE)
    refused(L, append(L, pages=0), ALIAS, SHAPE)
    for name in ("q", "k", "v", "cs", "pos", "slots", "qo", "kp", "vp"):
        refused(L, append(L, **{name: None}), "are required", NULL)
    for qo in (2, 7, 3, 4, 5, 6, 8, 10, 11):
        refused(L, append(L, qo=P(qo)), ALIAS, SHAPE)
    for out in ("kp", "vp"):
        for i in (1, 2, 7, 3, 4, 5, 6, 8, 9):
            refused(L, append(L, **{"qo": P(9), out: P(i)}), ALIAS, SHAPE)
    refused(L, append(L, qo=P(9), vp=P(10)), ALIAS, SHAPE)
    refused(L, append(L, qo=P(1), q_stride=2048), "only a contiguous input", SHAPE)
    assert append(L, seqlen=0, v=None) == OK


ATTN = dict(num_seqs=4, new_tokens=1, h_q=8, h_k=2, d=128, num_pages=1000, page_size=16, max_pages=200,
            window=0, dtype=1, scale=0.1, q_stride=0)


def attn(L, q=P(1), kp=P(2), vp=P(3), table=P(4), lens=P(5), o=P(1), lse=None, ws=P(16), nbytes=1 << 60, **sizes):
    return L.gdn2_paged_attention_step(q, kp, vp, table, lens, o, lse, ctypes.byref(AttentionDims(**{**ATTN, **sizes})),
                                       ws, nbytes, None)


NUMBERS, MULTIPLE, ROWS, PAGES = "num_seqs must be >= 0", "a multiple of h_k", "2^31 rows of queries", "page_size must be >= 1"
POOL, LONG, TABLE, GROUPS = "num_pages * h_k * page_size", "max_pages * page_size", "page_table is too large", "2^23 workgroups"
ONE = dict(num_seqs=1, new_tokens=1, h_q=1, h_k=1, d=64)

ATTN_REFUSALS = [
    (dict(dtype=2), "dtype must be", UNSUPPORTED), (dict(dtype=-1), "dtype must be", UNSUPPORTED),
    *[(dict(d=d), "d must be 64, 128 or 256", UNSUPPORTED) for d in (0, -64, 32, 96, 192, 512)],
    (dict(num_seqs=-1), NUMBERS, SHAPE), (dict(new_tokens=0), NUMBERS, SHAPE),
    *[(kw, MULTIPLE, SHAPE) for kw in (dict(h_q=0), dict(h_k=0), dict(h_k=3), dict(h_q=-8), dict(h_k=16))],
    (dict(h_q=(1 << 13) + 2), VALUES, SHAPE),
    (dict(num_seqs=1 << 20, new_tokens=1 << 11), ROWS, SHAPE),
    (dict(ONE, new_tokens=(1 << 30) + 1), ROWS, SHAPE), (dict(ONE, new_tokens=1 << 29, h_q=4), ROWS, SHAPE),
    (dict(num_pages=-1), PAGES, SHAPE), (dict(page_size=0), PAGES, SHAPE), (dict(max_pages=-1), PAGES, SHAPE),
    (dict(num_pages=1 << 26), POOL, SHAPE), (dict(page_size=(1 << 31) - 1), POOL, SHAPE),
    (dict(ONE, num_pages=1 << 30, page_size=2, max_pages=1), POOL, SHAPE),
    (dict(num_pages=1 << 30, page_size=1), POOL, SHAPE),
    (dict(max_pages=(1 << 25) + 1), LONG, SHAPE), (dict(num_pages=1, page_size=(1 << 29) + 1, max_pages=1), LONG, SHAPE),
    (dict(ONE, num_seqs=1 << 20, page_size=1, max_pages=(1 << 20) + 1), TABLE, SHAPE),
    (dict(window=-1), "window must be >= 0", SHAPE),
    *[(dict(scale=s), "scale must be finite", SHAPE) for s in (NAN, INF, -INF)],
    (dict(q_stride=1023), "q_stride is smaller", SHAPE), (dict(q_stride=-1024), "q_stride is smaller", SHAPE),
    (dict(q_stride=(1 << 38) + 1), "q_stride is smaller", SHAPE), (dict(q_stride=(1 << 63) - 1), "q_stride is smaller", SHAPE),
    # a workgroup takes one sequence, and 32 rows of queries
    (dict(ONE, num_seqs=1 << 29, max_pages=1), GROUPS, SHAPE), (dict(ONE, new_tokens=1 << 29, max_pages=1), GROUPS, SHAPE),
    (dict(ONE, new_tokens=1 << 26, h_q=16, max_pages=1), GROUPS, SHAPE),
]
ATTN_ACCEPTED = [
    dict(dtype=0), dict(d=64), dict(d=256), dict(num_seqs=1), dict(h_k=8), dict(h_k=1), dict(h_q=1 << 13),
    dict(ONE, num_seqs=1 << 23, max_pages=1),                        # 2^23 workgroups of whole sequences
    dict(ONE, new_tokens=1 << 24, max_pages=1), dict(ONE, new_tokens=1 << 20, h_q=16), dict(num_pages=0), dict(max_pages=0),
    dict(ONE, num_pages=(1 << 31) - 1, page_size=1), dict(num_pages=(1 << 26) - 1),
    dict(max_pages=1 << 25), dict(ONE, num_pages=1, page_size=1 << 29, max_pages=1),
    dict(ONE, num_seqs=1 << 20, page_size=1, max_pages=1 << 20),
    dict(window=(1 << 31) - 1), dict(scale=0.0), dict(scale=-3e38), dict(scale=3e38), dict(q_stride=1024), dict(q_stride=1 << 38),
]


def test_attention_sizes(L):
    for sizes, why, code in ATTN_REFUSALS:
        refused(L, attn(L, **sizes), why, code)
    for sizes in ATTN_ACCEPTED:
        refused(L, attn(L, **sizes), ALIAS, SHAPE)


def test_attention_tensors(L):
    for name in ("q", "kp", "vp", "table", "lens", "o"):
        refused(L, attn(L, **{name: None}), "are required", NULL)
    for o in (1, 2, 3, 4, 5, 16):
        refused(L, attn(L, o=P(o)), ALIAS, SHAPE)
        refused(L, attn(L, o=P(9), lse=P(o)), ALIAS, SHAPE)
    refused(L, attn(L, o=P(9), lse=P(9)), ALIAS, SHAPE)
    odd = ctypes.c_void_p(0x9008)
    for name in ("kp", "vp", "o"):
        refused(L, attn(L, **{"o": P(9), name: odd}), "16-byte aligned", SHAPE)
    refused(L, attn(L, o=P(9), ws=None), "workspace is NULL", WORKSPACE)
    refused(L, attn(L, o=P(9), ws=ctypes.c_void_p(0x10080)), "256-byte", WORKSPACE)
    need = L.gdn2_paged_attention_step_workspace_bytes(ctypes.byref(AttentionDims(**ATTN)))
    refused(L, attn(L, o=P(9), nbytes=need - 1), "too small", WORKSPACE)
    assert attn(L, num_seqs=0, q=None) == OK


def copy(L, pools=(0x1000, 0x8000), sizes=(64, 64), slots=10, src=P(8), dst=P(9), count=4):
    return L.gdn2_pool_copy((ctypes.c_void_p * len(pools))(*pools), (ctypes.c_int64 * len(sizes))(*sizes), len(pools), slots,
                            src, dst, count, None)


def test_pool_copy(L):
    refused(L, L.gdn2_pool_copy(None, None, -1, 1, P(8), P(9), 1, None), "must be >= 0", SHAPE)
    refused(L, copy(L, slots=-1), "must be >= 0", SHAPE)
    refused(L, copy(L, count=-1), "must be >= 0", SHAPE)
    refused(L, L.gdn2_pool_copy(None, None, 1, 1, P(8), P(9), 1, None), "pools and slot_bytes", NULL)
    for sizes in ((64, 0), (64, -1), ((1 << 32) + 1, 64)):
        refused(L, copy(L, sizes=sizes, slots=1), "slot_bytes must be", SHAPE)
    refused(L, copy(L, sizes=(1 << 32, 64), slots=(1 << 10) + 1), "slot_bytes must be", SHAPE)
    refused(L, copy(L, sizes=(1 << 32, 64), slots=1 << 10), "a pool aliases", SHAPE)
    refused(L, copy(L, sizes=(1 << 11, 64), slots=(1 << 31) - 1), "a pool aliases", SHAPE)
    refused(L, copy(L, pools=(0x1000, 0)), "a pool is NULL", NULL)
    refused(L, copy(L, pools=(0x1000, 0x2000, 0x1000), sizes=(64, 64, 64)), "a pool is given twice", SHAPE)
    refused(L, copy(L, src=None), "src and dst", NULL)
    refused(L, copy(L, dst=None), "src and dst", NULL)
    refused(L, copy(L), "a pool aliases", SHAPE)
    refused(L, copy(L, pools=(0x9000,), sizes=(4,)), "a pool aliases", SHAPE)
    assert copy(L, count=0, src=None) == OK and copy(L, slots=0, src=None) == OK and copy(L, dst=P(8)) == OK
