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
from array import array
from typing import Optional, Sequence, Tuple, Union

import torch

from . import _dtype_code, _ptr, lib
from .layer import _call, _check, _gpu_of, _grad_code, _tokens, _workspace

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


_MOST = (1 << 31) - 1             # what the C structs hold in 32 bits


def _small(**sizes) -> None:
    """Refuses sizes that the C structs cannot hold; the C ABI checks everything smaller."""
    for name, value in sizes.items():
        if value > _MOST:
            raise ValueError(f"{name} is {value}, at most {_MOST}")


def _whole(name: str, t: Optional[torch.Tensor], dev, dtype, shape) -> Optional[int]:
    """Checks a contiguous tensor of one type and shape (None is let through); its pointer. (One
    comparison per property: a call of single tokens takes as long on the host as on the GPU.)"""
    if t is None:
        return None
    if t.dtype is not dtype or t.get_device() != dev.index or t.shape != shape:
        _check(name, t, dev, dtype, shape)
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _heads(name: str, t: torch.Tensor, dev, dtype, shape) -> int:
    """Checks a token input [B,T,H,d] that may be a column slice. Returns the elements from one
    token to the next."""
    if t.dtype is not dtype or t.get_device() != dev.index or t.shape != shape:
        _check(name, t, dev, dtype, shape)
    B, T, H, d = shape
    row = H * d
    sb, st, sh, sd = t.stride()
    if T > 1 and sd == 1 and sh == d and st >= row and sb == T * st:
        return st
    if T == 1 and sd == 1 and sh == d and sb >= row:
        return sb
    return _tokens(name, t, dev, dtype, shape, row)


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


def _rotary_dims(q, k, v, cos_sin, positions, q_weight, k_weight, interleaved, eps, grad_code):
    """The checked dims of a rotary call and the pointers of its inputs, without v."""
    dev, dtype = _gpu_of("q", q), q.dtype
    if q.dim() != 4:
        raise ValueError("q must be [B,T,h_q,d]")
    B, T, hq, d = shape = q.shape
    code = _dtype_code(dtype)
    qs = _heads("q", q, dev, dtype, shape)
    hk = ks = vs = 0
    pk = None
    if k is not None:
        if k.dim() != 4:
            raise ValueError("k must be [B,T,h_k,d]")
        hk = k.shape[2]
        ks = _heads("k", k, dev, dtype, (B, T, hk, d))
        pk = k.data_ptr()
    if v is not None:
        vs = _heads("v", v, dev, dtype, (B, T, hk, d))
    f32 = torch.float32
    if cos_sin.dim() != 2:
        raise ValueError("cos_sin must be fp32 [num_positions,d_rot]")
    P, rot = cos_sin.shape
    if B * T > _MOST or hq * d > _MOST or hk * d > _MOST or P > _MOST or rot > _MOST:
        _small(tokens=B * T, values=max(hq, hk) * d, num_positions=P, d_rot=rot)
    ptrs = (q.data_ptr(), pk, _whole("cos_sin", cos_sin, dev, f32, (P, rot)),
            _whole("positions", positions, dev, torch.int32, (B, T)),
            _whole("q_weight", q_weight, dev, f32, (d,)),
            _whole("k_weight", k_weight, dev, f32, (d,)))
    return RotaryDims(B, T, hq, hk, d, rot, 1 if interleaved else 0, P, code, grad_code, eps, qs,
                      ks, vs), ptrs


def _output(name: str, given: Optional[torch.Tensor], like: torch.Tensor):
    """A contiguous output of the shape and type of an input, new or given, and its pointer."""
    if given is None:
        out = torch.empty_like(like, memory_format=torch.contiguous_format)
        return out, out.data_ptr()
    return given, _whole(name, given, like.device, like.dtype, like.shape)


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
    d, ptrs = _rotary_dims(q, k, None, cos_sin, positions, q_weight, k_weight, interleaved, eps, 0)
    dev = q.device
    qo, pq = _output("q_out", q_out, q)
    ko = pk = None
    if k is not None:
        ko, pk = _output("k_out", k_out, k)
    elif k_out is not None:
        raise ValueError("k_out needs k")
    _call(dev, lib().gdn2_qk_rotary_fwd, *ptrs, pq, pk, ctypes.byref(d))
    return qo, ko


def qk_rotary_bwd(q, k: Optional[torch.Tensor], cos_sin, dq_out,
                  dk_out: Optional[torch.Tensor] = None, positions: Optional[torch.Tensor] = None,
                  q_weight: Optional[torch.Tensor] = None, k_weight: Optional[torch.Tensor] = None,
                  interleaved: bool = False, eps: float = 1e-5,
                  workspace: Optional[torch.Tensor] = None) -> dict:
    """Gradients of qk_rotary_fwd given dq_out = dL/dq_out and dk_out = dL/dk_out (both in q's dtype
    or both in fp32). Returns dq (and dk) in that dtype, and dq_weight, dk_weight fp32 [d] for the
    weights given (zeros for k_weight without keys)."""
    if (dk_out is None) != (k is None):
        raise ValueError("k and dk_out go together")
    gt = dq_out.dtype
    d, ptrs = _rotary_dims(q, k, None, cos_sin, positions, q_weight, k_weight, interleaved, eps,
                           _grad_code("dq_out", dq_out, q.dtype))
    dev = q.device
    pdq = _whole("dq_out", dq_out, dev, gt, q.shape)
    out = {"dq": torch.empty_like(dq_out)}
    pdk = None
    if k is not None:
        pdk = _whole("dk_out", dk_out, dev, gt, k.shape)
        out["dk"] = torch.empty_like(dk_out)
    if q_weight is not None:
        out["dq_weight"] = torch.empty_like(q_weight)
    if k_weight is not None:
        out["dk_weight"] = torch.empty_like(k_weight)
    dims = ctypes.byref(d)
    pw = nw = 0
    if q_weight is not None or k_weight is not None or workspace is not None:
        ws = _workspace(workspace, lib().gdn2_qk_rotary_bwd_workspace_bytes(dims), dev)
        pw, nw = ws.data_ptr(), ws.numel() * ws.element_size()
    _call(dev, lib().gdn2_qk_rotary_bwd, *ptrs, pdq, pdk, out["dq"].data_ptr(), _ptr(out.get("dk")),
          _ptr(out.get("dq_weight")), _ptr(out.get("dk_weight")), dims, pw, nw)
    return out


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
    if n > _MOST or size > _MOST:
        _small(num_pages=n, page_size=size)
    return n, size


def qk_rotary_append(q, k, v, cos_sin, positions, k_pages, v_pages, slots,
                     q_weight: Optional[torch.Tensor] = None,
                     k_weight: Optional[torch.Tensor] = None, interleaved: bool = False,
                     eps: float = 1e-5, q_out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """qk_rotary_fwd in front of a cache: the normed and rotated keys and the values (v [B,T,h_k,d],
    as they are) go to k_pages, v_pages [num_pages,h_k,page_size,d], updated in place. slots int32
    [B,T]: the place of each token, page * page_size + row; distinct; outside the pool the token is
    not put anywhere, and neither is a padding token (a position outside the table). For prompts,
    packed or not, and for single tokens alike. Returns q_out [B,T,h_q,d]."""
    d, ptrs = _rotary_dims(q, k, v, cos_sin, positions, q_weight, k_weight, interleaved, eps, 0)
    dev, dtype, shape = q.device, q.dtype, q.shape
    pages, size = _pages(k_pages, v_pages, dev, dtype, d.h_k, d.d)
    ps = _whole("slots", slots, dev, torch.int32, shape[:2])
    qo, pq = _output("q_out", q_out, q)
    pq_in, pk, pcs, ppos, pqw, pkw = ptrs
    _call(dev, lib().gdn2_qk_rotary_append, pq_in, pk, v.data_ptr(), pcs, ppos, pqw, pkw, ps, pq,
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
    that sees nothing, or nothing but products of -inf, gives zeros, and an lse of -inf."""
    dev, dtype = _gpu_of("q", q), q.dtype
    if q.dim() != 4:
        raise ValueError("q must be [N,T,h_q,d]")
    N, T, hq, d = shape = q.shape
    code = _dtype_code(dtype)
    step = _heads("q", q, dev, dtype, shape)
    if k_pages.dim() != 4:
        raise ValueError(f"k_pages must be [num_pages,h_k,page_size,{d}]")
    hk = k_pages.shape[1]
    pages, size = _pages(k_pages, v_pages, dev, dtype, hk, d)
    if page_table.dim() != 2:
        raise ValueError(f"page_table must be int32 [{N},max_pages]")
    most = page_table.shape[1]
    if N * T > _MOST or hq * d > _MOST or hk > _MOST or most > _MOST or window > _MOST:
        _small(tokens=N * T, values=hq * d, h_k=hk, max_pages=most, window=window)
    pt = _whole("page_table", page_table, dev, torch.int32, (N, most))
    pl = _whole("seq_lens", seq_lens, dev, torch.int32, (N,))
    dims = AttentionDims(N, T, hq, hk, d, pages, size, most, window, code,
                         d ** -0.5 if scale is None else scale, step)
    o, po = _output("out", out, q)
    if return_lse and lse is None:
        lse = torch.empty((N, T, hq), dtype=torch.float32, device=dev)
        ple = lse.data_ptr()
    else:
        ple = _whole("lse", lse, dev, torch.float32, (N, T, hq))
    need = lib().gdn2_paged_attention_step_workspace_bytes(ctypes.byref(dims))
    pw = nw = 0
    if workspace is not None or need:
        ws = _workspace(workspace, need, dev)
        pw, nw = ws.data_ptr(), ws.numel() * ws.element_size()
    _call(dev, lib().gdn2_paged_attention_step, q.data_ptr(), k_pages.data_ptr(),
          v_pages.data_ptr(), pt, pl, po, ple, ctypes.byref(dims), pw, nw)
    return (o, lse) if return_lse else o


def paged_attention_step_workspace_bytes(num_seqs: int, new_tokens: int, h_q: int, h_k: int, d: int,
                                         page_size: int, max_pages: int, dtype: torch.dtype) -> int:
    """Bytes that are enough for these sizes with any window, and with fewer sequences."""
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
    count = src.numel()
    ps = _whole("src", src, dev, torch.int32, (count,))
    pd = _whole("dst", dst, dev, torch.int32, (count,))
    if not pools:
        return
    index = dev.index
    slots = pools[0].shape[0] if pools[0].dim() else -1
    if slots > _MOST or count > _MOST:
        _small(num_slots=slots, count=count)
    for t in pools:
        if t.get_device() != index or not t.dim() or t.shape[0] != slots or not t.is_contiguous():
            if t.dim():
                _check("a pool", t, dev, t.dtype, (slots, *t.shape[1:]))
            raise ValueError("a pool must be a contiguous [num_slots,...]")
    if slots == 0:
        return
    sizes = array("q", [t.nbytes // slots for t in pools])
    if 0 in sizes:
        pools = [t for t in pools if t.nbytes]
        sizes = array("q", [n for n in sizes if n])
    ptrs = array("q", [t.data_ptr() for t in pools])
    _call(dev, lib().gdn2_pool_copy, ptrs.buffer_info()[0], sizes.buffer_info()[0], len(ptrs), slots,
          ps, pd, count)
