"""The attention layer that hybrid stacks put beside the recurrent ones, bound to libgdn2.so: norms
of queries and keys with the rotation by position, attention of new tokens over a paged cache,
and copies of slots of pools.

    q, k  = qk_rotary_fwd(q, k, cos_sin, positions=None, q_weight=None, k_weight=None)
    grads = qk_rotary_bwd(q, k, cos_sin, dq_out, dk_out, ...)
    q     = qk_rotary_append(q, k, v, cos_sin, positions, k_pages, v_pages, slots, ...)
                                                        # the pages are updated in place
    o     = paged_attention_step(q, k_pages, v_pages, page_table, seq_lens)
    pool_copy(pools, src, dst)                          # slots copied inside every pool

As in ``layer``, these functions check shapes, allocate outputs and workspaces and call the C ABI
(``include/gdn2.h``) on the current HIP stream of the tensors' device. Token inputs may be column
slices of a wider tensor (one stride from token to token); everything else is contiguous.
Gradients are returned in a dict, ``d`` before each input's name.
"""
from __future__ import annotations

import ctypes
from typing import Optional, Sequence, Tuple, Union

import torch

from . import _dtype_code, _ptr, lib
from .layer import _call, _check, _fits, _gpu_of, _grad_code, _tokens, _whole, _workspace

_i32, _i64, _f32, _vp, _sz = (ctypes.c_int32, ctypes.c_int64, ctypes.c_float, ctypes.c_void_p,
                              ctypes.c_size_t)


class RotaryDims(ctypes.Structure):
    _fields_ = [("batch", _i32), ("seqlen", _i32), ("h_q", _i32), ("h_k", _i32), ("d", _i32),
                ("d_rot", _i32), ("interleaved", _i32), ("num_positions", _i32), ("dtype", _i32),
                ("grad_dtype", _i32), ("eps", _f32), ("q_stride", _i64), ("k_stride", _i64),
                ("v_stride", _i64)]


class AttentionDims(ctypes.Structure):
    _fields_ = [("num_seqs", _i32), ("new_tokens", _i32), ("h_q", _i32), ("h_k", _i32), ("d", _i32),
                ("num_pages", _i32), ("page_size", _i32), ("max_pages", _i32), ("window", _i32),
                ("dtype", _i32), ("scale", _f32), ("q_stride", _i64)]


def declare(L: ctypes.CDLL) -> None:
    """Argument types of this module's calls (lib() runs it once)."""
    rd, ad = ctypes.POINTER(RotaryDims), ctypes.POINTER(AttentionDims)
    for name, restype, argtypes in (
            ("gdn2_qk_rotary_fwd", _i32, [_vp] * 8 + [rd, _vp]),
            ("gdn2_qk_rotary_bwd_workspace_bytes", _sz, [rd]),
            ("gdn2_qk_rotary_bwd", _i32, [_vp] * 12 + [rd, _vp, _sz, _vp]),
            ("gdn2_qk_rotary_append", _i32, [_vp] * 11 + [_i32, _i32, rd, _vp]),
            ("gdn2_paged_attention_step_workspace_bytes", _sz, [ad]),
            ("gdn2_paged_attention_step", _i32, [_vp] * 7 + [ad, _vp, _sz, _vp]),
            ("gdn2_pool_copy", _i32, [_vp, _vp, _i32, _i32, _vp, _vp, _i32, _vp])):
        f = getattr(L, name)
        f.restype, f.argtypes = restype, argtypes


# ---- norms and rotation ------------------------------------------------------------------


def rotary_table(num_positions: int, d_rot: int, base: float = 10000.0, device=None) -> torch.Tensor:
    """The usual table of qk_rotary_fwd: fp32 [num_positions,d_rot], the cosines, then the sines, of
    position * base^(-2 i / d_rot), i < d_rot/2, rounded once from 64 bits. A program makes it once;
    other frequencies (scaled contexts) go into a table of the same layout."""
    if num_positions < 0 or d_rot < 0 or d_rot % 2:
        raise ValueError("num_positions must be >= 0 and d_rot even and >= 0")
    i = torch.arange(d_rot // 2, dtype=torch.float64, device=device)
    angle = torch.arange(num_positions, dtype=torch.float64, device=device)[:, None] \
        * float(base) ** (-2.0 * i / max(d_rot, 1))
    return torch.cat((angle.cos(), angle.sin()), 1).float()


def _rotary_dims(q, k, v, cos_sin, positions, q_weight, k_weight, interleaved, eps, grad_code
                 ) -> RotaryDims:
    """The checked dims of a rotary call."""
    dev, dtype = _gpu_of("q", q), q.dtype
    if q.dim() != 4:
        raise ValueError("q must be [B,T,h_q,d]")
    B, T, hq, d = q.shape
    _fits("the number of tokens", B * T)
    _fits("a token's values", hq * d)
    code = _dtype_code(dtype)
    qs = _tokens("q", q, dev, dtype, q.shape, hq * d)
    hk, ks, vs = 0, 0, 0
    if k is not None:
        if k.dim() != 4:
            raise ValueError("k must be [B,T,h_k,d]")
        hk = k.shape[2]
        _fits("a token's values", hk * d)
        ks = _tokens("k", k, dev, dtype, (B, T, hk, d), hk * d)
    if v is not None:
        vs = _tokens("v", v, dev, dtype, (B, T, hk, d), hk * d)
    f32 = torch.float32
    if cos_sin.dim() != 2:
        raise ValueError("cos_sin must be fp32 [num_positions,d_rot]")
    P, rot = cos_sin.shape
    _whole("cos_sin", cos_sin, dev, f32, (P, rot))
    _whole("positions", positions, dev, torch.int32, (B, T))
    _whole("q_weight", q_weight, dev, f32, (d,))
    _whole("k_weight", k_weight, dev, f32, (d,))
    return RotaryDims(B, T, hq, hk, d, _fits("d_rot", rot), 1 if interleaved else 0,
                      _fits("num_positions", P), code, grad_code, eps, qs, ks, vs)


def qk_rotary_fwd(q, k: Optional[torch.Tensor], cos_sin, positions: Optional[torch.Tensor] = None,
                  q_weight: Optional[torch.Tensor] = None, k_weight: Optional[torch.Tensor] = None,
                  interleaved: bool = False, eps: float = 1e-5,
                  q_out: Optional[torch.Tensor] = None, k_out: Optional[torch.Tensor] = None
                  ) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """Norms of queries and keys per head and their rotation by position:
        y = x / sqrt(mean(x^2) + eps) weight,   (y_a, y_b) -> (y_a cos - y_b sin, y_b cos + y_a sin)
    for the pairs (i, i + d_rot/2) of a head, or (2i, 2i+1) if interleaved; without a weight there is
    no norm, and values from d_rot on are not rotated. q [B,T,h_q,d], k [B,T,h_k,d] or None (each may
    be a column slice); cos_sin fp32 [num_positions,d_rot] (rotary_table makes the usual one);
    positions int32 [B,T] (None: 0 .. T-1 in every sequence), one outside the table marking a padding
    token (zero rows); q_weight, k_weight fp32 [d]. Returns (q_out, k_out), which may be given and
    may be contiguous q and k themselves."""
    d = _rotary_dims(q, k, None, cos_sin, positions, q_weight, k_weight, interleaved, eps, 0)
    dev = q.device
    qo = torch.empty(q.shape, dtype=q.dtype, device=dev) if q_out is None else q_out
    pq = _whole("q_out", qo, dev, q.dtype, q.shape)
    ko = None
    if k is not None:
        ko = torch.empty(k.shape, dtype=k.dtype, device=dev) if k_out is None else k_out
        _whole("k_out", ko, dev, k.dtype, k.shape)
    elif k_out is not None:
        raise ValueError("k_out needs k")
    _call(dev, lib().gdn2_qk_rotary_fwd, q.data_ptr(), _ptr(k), cos_sin.data_ptr(), _ptr(positions),
          _ptr(q_weight), _ptr(k_weight), pq, _ptr(ko), ctypes.byref(d))
    return qo, ko


def qk_rotary_bwd(q, k: Optional[torch.Tensor], cos_sin, dq_out,
                  dk_out: Optional[torch.Tensor] = None, positions: Optional[torch.Tensor] = None,
                  q_weight: Optional[torch.Tensor] = None, k_weight: Optional[torch.Tensor] = None,
                  interleaved: bool = False, eps: float = 1e-5,
                  workspace: Optional[torch.Tensor] = None) -> dict:
    """Gradients of qk_rotary_fwd given dq_out = dL/dq_out and dk_out = dL/dk_out (both in q's dtype
    or both in fp32). Returns dq (and dk) in that dtype, and dq_weight, dk_weight fp32 [d] for the
    weights given."""
    if (dk_out is None) != (k is None):
        raise ValueError("k and dk_out go together")
    gt = dq_out.dtype
    d = _rotary_dims(q, k, None, cos_sin, positions, q_weight, k_weight, interleaved, eps,
                     _grad_code("dq_out", dq_out, q.dtype))
    dev, f32 = q.device, torch.float32
    pdq = _whole("dq_out", dq_out, dev, gt, q.shape)
    pdk = None if k is None else _whole("dk_out", dk_out, dev, gt, k.shape)
    if k is None:
        k_weight = None
    new = lambda like, dtype: None if like is None else torch.empty(  # noqa: E731
        like.shape, dtype=dtype, device=dev)
    out = {"dq": new(q, gt), "dk": new(k, gt), "dq_weight": new(q_weight, f32),
           "dk_weight": new(k_weight, f32)}
    ws = _workspace(workspace, lib().gdn2_qk_rotary_bwd_workspace_bytes(ctypes.byref(d)), dev)
    _call(dev, lib().gdn2_qk_rotary_bwd, q.data_ptr(), _ptr(k), cos_sin.data_ptr(), _ptr(positions),
          _ptr(q_weight), _ptr(k_weight), pdq, pdk, *(_ptr(t) for t in out.values()),
          ctypes.byref(d), ws.data_ptr(), ws.numel())
    return {n: t for n, t in out.items() if t is not None}


def qk_rotary_bwd_workspace_bytes(batch: int, seqlen: int, d: int) -> int:
    n = RotaryDims(batch, seqlen, 1, 0, d, 0, 0, 0, 0, 0, 0.0, 0, 0, 0)
    return int(lib().gdn2_qk_rotary_bwd_workspace_bytes(ctypes.byref(n)))


def _pages(k_pages, v_pages, dev, dtype, hk: int, d: int) -> Tuple[int, int]:
    """Checks the pools of a cache. Returns (num_pages, page_size)."""
    if k_pages.dim() != 4:
        raise ValueError(f"k_pages must be [num_pages,{hk},page_size,{d}]")
    n, size = k_pages.shape[0], k_pages.shape[2]
    _whole("k_pages", k_pages, dev, dtype, (n, hk, size, d))
    _whole("v_pages", v_pages, dev, dtype, (n, hk, size, d))
    return _fits("num_pages", n), _fits("page_size", size)


def qk_rotary_append(q, k, v, cos_sin, positions, k_pages, v_pages, slots,
                     q_weight: Optional[torch.Tensor] = None,
                     k_weight: Optional[torch.Tensor] = None, interleaved: bool = False,
                     eps: float = 1e-5, q_out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """qk_rotary_fwd in front of a cache: the normed and rotated keys and the values (v [B,T,h_k,d],
    as they are) go to k_pages, v_pages [num_pages,h_k,page_size,d], updated in place. slots int32
    [B,T]: the place of each token, page * page_size + row; distinct; outside the pool the token is
    not put anywhere, and neither is a padding token (a position outside the table). For prompts,
    packed or not, and for single tokens alike. Returns q_out [B,T,h_q,d]."""
    d = _rotary_dims(q, k, v, cos_sin, positions, q_weight, k_weight, interleaved, eps, 0)
    dev = q.device
    pages, size = _pages(k_pages, v_pages, dev, q.dtype, d.h_k, d.d)
    ps = _whole("slots", slots, dev, torch.int32, q.shape[:2])
    qo = torch.empty(q.shape, dtype=q.dtype, device=dev) if q_out is None else q_out
    pq = _whole("q_out", qo, dev, q.dtype, q.shape)
    _call(dev, lib().gdn2_qk_rotary_append, q.data_ptr(), k.data_ptr(), v.data_ptr(),
          cos_sin.data_ptr(), positions.data_ptr(), _ptr(q_weight), _ptr(k_weight), ps, pq,
          k_pages.data_ptr(), v_pages.data_ptr(), pages, size, ctypes.byref(d))
    return qo


# ---- attention ---------------------------------------------------------------------------


def paged_attention_step(q, k_pages, v_pages, page_table, seq_lens, scale: Optional[float] = None,
                         window: int = 0, return_lse: bool = False,
                         out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                         workspace: Optional[torch.Tensor] = None
                         ) -> Union[torch.Tensor, Tuple[torch.Tensor, torch.Tensor]]:
    """Attention of the last T tokens of each of N sequences over the sequence's cached tokens, the
    new ones among them. q [N,T,h_q,d], d = 64, 128 or 256 (may be a column slice); k_pages, v_pages
    [num_pages,h_k,page_size,d] in q's dtype; page_table int32 [N,max_pages]; seq_lens int32 [N].
    Token t stands at place seq_lens[n] - T + t and sees the places up to its own, with a window > 0
    the last `window` of them. scale: of the products (None: d^-1/2). Returns o [N,T,h_q,d], or
    (o, lse fp32 [N,T,h_q]) with return_lse: lse = log sum exp of a row's scaled products. A token
    that sees nothing gives zeros, and an lse of -inf."""
    dev, dtype = _gpu_of("q", q), q.dtype
    if q.dim() != 4:
        raise ValueError("q must be [N,T,h_q,d]")
    N, T, hq, d = q.shape
    _fits("the number of tokens", N * T)
    _fits("a token's values", hq * d)
    code = _dtype_code(dtype)
    step = _tokens("q", q, dev, dtype, q.shape, hq * d)
    if k_pages.dim() != 4:
        raise ValueError(f"k_pages must be [num_pages,h_k,page_size,{d}]")
    hk = _fits("h_k", k_pages.shape[1])
    pages, size = _pages(k_pages, v_pages, dev, dtype, hk, d)
    if page_table.dim() != 2:
        raise ValueError(f"page_table must be int32 [{N},max_pages]")
    most = _fits("max_pages", page_table.shape[1])
    pt = _whole("page_table", page_table, dev, torch.int32, (N, most))
    pl = _whole("seq_lens", seq_lens, dev, torch.int32, (N,))
    dims = AttentionDims(N, T, hq, hk, d, pages, size, most, _fits("window", window), code,
                         d ** -0.5 if scale is None else scale, step)
    o = torch.empty(q.shape, dtype=dtype, device=dev) if out is None else out
    po = _whole("out", o, dev, dtype, q.shape)
    if return_lse and lse is None:
        lse = torch.empty((N, T, hq), dtype=torch.float32, device=dev)
    ple = _whole("lse", lse, dev, torch.float32, (N, T, hq))
    need = lib().gdn2_paged_attention_step_workspace_bytes(ctypes.byref(dims))
    if workspace is not None or need:
        ws = _workspace(workspace, need, dev)
        pw, nw = ws.data_ptr(), ws.numel() * ws.element_size()
    else:
        pw, nw = None, 0
    _call(dev, lib().gdn2_paged_attention_step, q.data_ptr(), k_pages.data_ptr(),
          v_pages.data_ptr(), pt, pl, po, ple, ctypes.byref(dims), pw, nw)
    return (o, lse) if return_lse else o


def paged_attention_step_workspace_bytes(num_seqs: int, new_tokens: int, h_q: int, h_k: int, d: int,
                                         page_size: int, max_pages: int, dtype: torch.dtype) -> int:
    n = AttentionDims(num_seqs, new_tokens, h_q, h_k, d, 0, page_size, max_pages, 0,
                      _dtype_code(dtype), 1.0, 0)
    return int(lib().gdn2_paged_attention_step_workspace_bytes(ctypes.byref(n)))


# ---- pools -------------------------------------------------------------------------------


def pool_copy(pools: Union[torch.Tensor, Sequence[torch.Tensor]], src, dst) -> None:
    """Copies slots inside each of several pools, in place: pool[dst[i]] = pool[src[i]]. pools: a
    tensor [num_slots,...] or a sequence of them (any types and shapes, one num_slots), such as the
    key and value pages of every layer, or the states of recurrent layers; src, dst int32 [count]. A
    pair with an entry outside the pool is skipped. One source may have many destinations; the
    destinations must be distinct, and none may be the source of another pair."""
    if isinstance(pools, torch.Tensor):
        pools = [pools]
    dev = _gpu_of("src", src)
    if src.dim() != 1:
        raise ValueError("src must be int32 [count]")
    count = _fits("count", src.numel())
    ps = _whole("src", src, dev, torch.int32, (count,))
    pd = _whole("dst", dst, dev, torch.int32, (count,))
    if not pools:
        return
    if pools[0].dim() < 1:
        raise ValueError("a pool must be [num_slots,...]")
    slots = _fits("the number of slots", pools[0].shape[0])
    ptrs, sizes = [], []
    for t in pools:
        if t.device != dev or t.dim() < 1 or t.shape[0] != slots or not t.is_contiguous():
            if t.dim() >= 1:
                _check("a pool", t, dev, t.dtype, (slots, *t.shape[1:]))
            raise ValueError("a pool must be a contiguous [num_slots,...]")
        if t.numel():
            ptrs.append(t.data_ptr())
            sizes.append(t.numel() // slots * t.element_size())
    n = len(ptrs)
    _call(dev, lib().gdn2_pool_copy, (_vp * n)(*ptrs), (_i64 * n)(*sizes), n, slots, ps, pd, count)
