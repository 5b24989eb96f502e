"""The operators around the recurrence, bound to libgdn2.so: the short causal convolution and
the selective state space scan, over prompts, their gradients, and for single tokens, and the
norms around a block.

    y, state_T = short_conv_fwd(x, weight, bias=None, state0=None, cu_seqlens=None, silu=False)
    grads      = short_conv_bwd(x, weight, dy, ...)
    y          = short_conv_step(x, weight, conv_state, ...)        # conv_state updated in place
    o, S_T     = selective_scan_fwd(x, dt, A, B, C, D=None, gate=None, ...)
    grads      = selective_scan_bwd(x, dt, A, B, C, dO, ...)
    o          = selective_scan_step(x, dt, A, B, C, state, ...)    # state updated in place
    h, y       = block_norm_fwd(x, norm_weight, gate, residual, scale, next_weight)
    grads      = block_norm_bwd(x, dh, dy, ...)

As in the rest of the package, these functions check shapes, allocate outputs and workspaces
and call the C ABI (``include/gdn2.h``) on the current HIP stream of the tensors' device. Token
inputs may be column slices of a wider tensor (one stride from token to token); everything else
is contiguous. Rows behind the last sequence of a packed batch are not written, in outputs and
gradients alike. Gradients are returned in a dict, ``d`` before each input's name: those of token
tensors in the type of the incoming gradient, those of parameters and states in fp32.
"""
from __future__ import annotations

import ctypes
from typing import Optional, Tuple

import torch

from . import _dtype_code, _need_gpu, _ptr, _raise_on, lib

_i32, _i64, _f32, _vp, _sz = (ctypes.c_int32, ctypes.c_int64, ctypes.c_float, ctypes.c_void_p,
                              ctypes.c_size_t)


class ConvDims(ctypes.Structure):
    _fields_ = [("batch", _i32), ("seqlen", _i32), ("num_seqs", _i32), ("channels", _i32),
                ("width", _i32), ("dtype", _i32), ("grad_dtype", _i32), ("silu", _i32),
                ("x_stride", _i64)]


class ScanDims(ctypes.Structure):
    _fields_ = [("batch", _i32), ("seqlen", _i32), ("num_seqs", _i32), ("channels", _i32),
                ("d_state", _i32), ("groups", _i32), ("dtype", _i32), ("grad_dtype", _i32),
                ("dt_softplus", _i32), ("x_stride", _i64), ("dt_stride", _i64),
                ("b_stride", _i64), ("c_stride", _i64), ("gate_stride", _i64)]


class NormDims(ctypes.Structure):
    _fields_ = [("rows", _i64), ("d", _i32), ("dtype", _i32), ("residual_dtype", _i32),
                ("grad_dtype", _i32), ("eps", _f32), ("x_stride", _i64), ("gate_stride", _i64)]


def declare(L: ctypes.CDLL) -> None:
    """Argument types of this module's calls (lib() runs it once)."""
    cd, sd, nd = (ctypes.POINTER(t) for t in (ConvDims, ScanDims, NormDims))
    for name, restype, argtypes in (
            ("gdn2_short_conv_fwd", _i32, [_vp] * 7 + [cd, _vp]),
            ("gdn2_short_conv_bwd_workspace_bytes", _sz, [cd]),
            ("gdn2_short_conv_bwd", _i32, [_vp] * 11 + [cd, _vp, _sz, _vp]),
            ("gdn2_short_conv_step", _i32, [_vp] * 5 + [_i32, _vp, cd, _vp]),
            ("gdn2_selective_scan_fwd_workspace_bytes", _sz, [sd]),
            ("gdn2_selective_scan_fwd", _i32, [_vp] * 12 + [sd, _vp, _sz, _vp]),
            ("gdn2_selective_scan_bwd_workspace_bytes", _sz, [sd]),
            ("gdn2_selective_scan_bwd", _i32, [_vp] * 21 + [sd, _vp, _sz, _vp]),
            ("gdn2_selective_scan_step", _i32,
             [_vp] * 9 + [_i32, _vp, _i32, _vp, sd, _vp]),
            ("gdn2_block_norm_fwd", _i32, [_vp] * 8 + [nd, _vp]),
            ("gdn2_block_norm_bwd_workspace_bytes", _sz, [nd]),
            ("gdn2_block_norm_bwd", _i32, [_vp] * 14 + [nd, _vp, _sz, _vp])):
        f = getattr(L, name)
        f.restype, f.argtypes = restype, argtypes


def _call(dev: torch.device, f, *args) -> None:
    """f(*args, stream) on the device's current stream, with that device current."""
    index = dev.index
    if torch._C._cuda_getDevice() == index:
        st = f(*args, torch._C._cuda_getCurrentRawStream(index))
    else:
        with torch.cuda.device(dev):
            st = f(*args, torch._C._cuda_getCurrentRawStream(index))
    if st:
        _raise_on(st)


def _gpu_of(name: str, t: torch.Tensor) -> torch.device:
    """The GPU a call runs on: that of its first input."""
    if not t.is_cuda:
        raise ValueError(f"{name} must be a GPU tensor (the library has no CPU path)")
    return t.device


def _check(name: str, t: torch.Tensor, dev, dtype, shape) -> None:
    """Says what is wrong with a tensor's device, type or shape."""
    if not t.is_cuda:
        raise ValueError(f"{name} must be a GPU tensor (the library has no CPU path)")
    if t.device != dev:
        raise ValueError(f"{name} is on {t.device}, expected {dev}")
    if t.dtype != dtype:
        raise TypeError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must be {list(shape)}, not {list(t.shape)}")


def _tokens(name: str, t: torch.Tensor, dev, dtype, shape, row: int) -> int:
    """Checks a token input [B, T, ...] of `row` values per token that may be a column slice.
    Returns the elements from one token to the next."""
    if t.dtype != dtype or t.device != dev or t.shape != shape:
        _check(name, t, dev, dtype, shape)
    if t.is_contiguous():
        return row
    want = 1
    for d in range(t.dim() - 1, 1, -1):
        if t.shape[d] != 1 and t.stride(d) != want:
            raise ValueError(f"{name}: every token's values must be contiguous")
        want *= t.shape[d]
    B, T = shape[0], shape[1]
    if T > 1:
        step = t.stride(1)
        if B > 1 and t.stride(0) != T * step:
            raise ValueError(f"{name}: the sequences must follow each other at one token stride")
    else:
        step = t.stride(0) if B > 1 else row
    if step < row:
        raise ValueError(f"{name}: tokens overlap (stride {step}, {row} values)")
    return step


def _whole(name: str, t: Optional[torch.Tensor], dev, dtype, shape) -> Optional[int]:
    """Checks a contiguous tensor of one type and shape (None is let through); its pointer."""
    if t is None:
        return None
    if t.dtype != dtype or t.device != dev or t.shape != shape:
        _check(name, t, dev, dtype, shape)
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _grad_code(name: str, t: torch.Tensor, dtype) -> int:
    """The type of a call's token gradients: fp32 or the inputs' own."""
    if t.dtype != torch.float32 and t.dtype != dtype:
        raise TypeError(f"{name} has dtype {t.dtype}, expected {dtype} or torch.float32")
    return _dtype_code(t.dtype)


def _sequences(cu_seqlens, B: int, dev) -> Tuple[int, int]:
    """(number of sequences, num_seqs of the dims) of a dense or packed batch."""
    if cu_seqlens is None:
        return B, 0
    _need_gpu("cu_seqlens", cu_seqlens, dev)
    if cu_seqlens.dtype != torch.int32 or cu_seqlens.dim() != 1:
        raise TypeError("cu_seqlens must be a 1-D int32 tensor")
    N = _fits("the number of sequences", cu_seqlens.numel() - 1)
    if N < 1 or B != 1:
        raise ValueError("a packed batch is [1,T,..] with cu_seqlens of N+1 >= 2 offsets")
    return N, N


def _fits(name: str, value: int, limit: int = (1 << 31) - 1) -> int:
    """A size that the C structs hold in 32 bits; the C ABI checks everything smaller."""
    if value > limit:
        raise ValueError(f"{name} is {value}, at most {limit}")
    return value


def _workspace(workspace, need: int, dev) -> torch.Tensor:
    if workspace is None:
        return torch.empty(max(need, 256), dtype=torch.uint8, device=dev)
    _need_gpu("workspace", workspace, dev)
    return workspace


# ---- short convolution -------------------------------------------------------------------


def _conv_dims(x, weight, bias, cu_seqlens, silu, grad_code) -> Tuple[ConvDims, int]:
    """The checked dims of a prompt call, and the number of sequences."""
    dev = _gpu_of("x", x)
    if x.dim() != 3:
        raise ValueError("x must be [B,T,C]")
    B, T, C = x.shape
    _fits("the number of tokens", B * T)
    _fits("channels", C)
    code = _dtype_code(x.dtype)
    step = _tokens("x", x, dev, x.dtype, x.shape, C)
    if weight.dim() != 2 or weight.shape[0] != C:
        raise ValueError(f"weight must be fp32 [{C},W]")
    W = weight.shape[1]
    _whole("weight", weight, dev, torch.float32, (C, W))
    _whole("bias", bias, dev, torch.float32, (C,))
    N, num_seqs = _sequences(cu_seqlens, B, dev)
    return ConvDims(B, T, num_seqs, C, W, code, grad_code, 1 if silu else 0, step), N


def short_conv_fwd(x, weight, bias: Optional[torch.Tensor] = None,
                   state0: Optional[torch.Tensor] = None,
                   cu_seqlens: Optional[torch.Tensor] = None, silu: bool = False,
                   output_final_state: bool = True, out: Optional[torch.Tensor] = None,
                   final_state: Optional[torch.Tensor] = None
                   ) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """The short causal depthwise convolution over prompts. x [B,T,C] (may be a column slice);
    weight fp32 [C,W], W = 2..4, the last tap on the current token; bias fp32 [C]; state0 fp32
    [N,W-1,C], the inputs before each sequence (None: zeros); cu_seqlens int32 [N+1] for a
    packed batch. Returns (y [B,T,C], state_T fp32 [N,W-1,C] or None): state_T is what
    recurrent_fwd and short_conv_step keep in their conv_state. It must not be state0's own
    buffer."""
    d, N = _conv_dims(x, weight, bias, cu_seqlens, silu, 0)
    dev, shape = x.device, x.shape
    f32 = torch.float32
    st_shape = (N, d.width - 1, d.channels)
    s0 = _whole("state0", state0, dev, f32, st_shape)
    y = torch.empty(shape, dtype=x.dtype, device=dev) if out is None else out
    py = _whole("out", y, dev, x.dtype, shape)
    state_T = None
    if output_final_state:
        state_T = torch.empty(st_shape, dtype=f32, device=dev) if final_state is None else final_state
    ps = _whole("final_state", state_T, dev, f32, st_shape)
    _call(dev, lib().gdn2_short_conv_fwd, x.data_ptr(), weight.data_ptr(), _ptr(bias), s0,
          _ptr(cu_seqlens), py, ps, ctypes.byref(d))
    return y, state_T


def short_conv_bwd(x, weight, dy, bias: Optional[torch.Tensor] = None,
                   state0: Optional[torch.Tensor] = None,
                   cu_seqlens: Optional[torch.Tensor] = None, silu: bool = False,
                   dstate_T: Optional[torch.Tensor] = None,
                   workspace: Optional[torch.Tensor] = None) -> dict:
    """Gradients of short_conv_fwd given dy = dL/dy [B,T,C] (x's dtype or fp32) and dstate_T =
    dL/dstate_T (None: zero). Returns dx (dy's dtype), dweight fp32 [C,W], and dbias, dstate0
    where the call has a bias, a state0."""
    d, N = _conv_dims(x, weight, bias, cu_seqlens, silu, _grad_code("dy", dy, x.dtype))
    dev, shape = x.device, x.shape
    f32 = torch.float32
    st_shape = (N, d.width - 1, d.channels)
    s0 = _whole("state0", state0, dev, f32, st_shape)
    pdy = _whole("dy", dy, dev, dy.dtype, shape)
    pds = _whole("dstate_T", dstate_T, dev, f32, st_shape)
    out = {"dx": torch.empty(shape, dtype=dy.dtype, device=dev),
           "dweight": torch.empty(weight.shape, dtype=f32, device=dev)}
    if bias is not None:
        out["dbias"] = torch.empty(bias.shape, dtype=f32, device=dev)
    if state0 is not None:
        out["dstate0"] = torch.empty(st_shape, dtype=f32, device=dev)
    ws = _workspace(workspace, lib().gdn2_short_conv_bwd_workspace_bytes(ctypes.byref(d)), dev)
    _call(dev, lib().gdn2_short_conv_bwd, x.data_ptr(), weight.data_ptr(), _ptr(bias), s0,
          _ptr(cu_seqlens), pdy, pds, out["dx"].data_ptr(), out["dweight"].data_ptr(),
          _ptr(out.get("dbias")), _ptr(out.get("dstate0")), ctypes.byref(d), ws.data_ptr(),
          ws.numel())
    return out


def short_conv_bwd_workspace_bytes(batch: int, seqlen: int, channels: int, width: int,
                                   dtype: torch.dtype, num_seqs: int = 0) -> int:
    d = ConvDims(batch, seqlen, num_seqs, channels, width, _dtype_code(dtype), 0, 0, 0)
    return int(lib().gdn2_short_conv_bwd_workspace_bytes(ctypes.byref(d)))


def _state_idx(state_idx, N: int, dev) -> Optional[int]:
    if state_idx is None:
        return None
    _need_gpu("state_idx", state_idx, dev)
    if state_idx.dtype != torch.int32 or state_idx.shape != (N,):
        raise ValueError(f"state_idx must be int32 [{N}]")
    return state_idx.data_ptr()


def short_conv_step(x, weight, conv_state, bias: Optional[torch.Tensor] = None,
                    state_idx: Optional[torch.Tensor] = None, silu: bool = False,
                    out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """T tokens of each of N sequences, x [N,T,C], against a pool of conv states fp32
    [num_slots,W-1,C], updated in place. state_idx int32 [N]: the slot of each sequence (None:
    slot n); an entry outside the pool marks padding (zero y rows, no state touched). Returns
    y [N,T,C]."""
    d, N = _conv_dims(x, weight, bias, None, silu, 0)
    dev, shape = x.device, x.shape
    if conv_state.dim() != 3:
        raise ValueError(f"conv_state must be fp32 [num_slots,{d.width - 1},{d.channels}]")
    slots = _fits("the number of slots", conv_state.shape[0])
    ps = _whole("conv_state", conv_state, dev, torch.float32, (slots, d.width - 1, d.channels))
    y = torch.empty(shape, dtype=x.dtype, device=dev) if out is None else out
    py = _whole("out", y, dev, x.dtype, shape)
    _call(dev, lib().gdn2_short_conv_step, x.data_ptr(), weight.data_ptr(), _ptr(bias), ps,
          _state_idx(state_idx, N, dev), slots, py, ctypes.byref(d))
    return y


# ---- selective scan ----------------------------------------------------------------------


def _batch(x) -> int:
    if x.dim() != 3:
        raise ValueError("x must be [B,T,channels]")
    return x.shape[0]


def _scan_dims(x, dt, A, B, C, D, gate, dt_bias, dt_softplus, num_seqs, grad_code) -> ScanDims:
    """The checked dims of a scan call."""
    dev, dtype, shape = _gpu_of("x", x), x.dtype, x.shape
    _batch(x)
    if B.dim() != 4:
        raise ValueError("B and C must be [B,T,groups,d_state]")
    n, T, ch = shape
    G, M = B.shape[2], B.shape[3]
    _fits("the number of tokens", n * T)
    _fits("channels", max(ch, G * M))
    code, bc = _dtype_code(dtype), (n, T, G, M)
    strides = [_tokens("x", x, dev, dtype, shape, ch), _tokens("dt", dt, dev, dtype, shape, ch),
               _tokens("B", B, dev, dtype, bc, G * M), _tokens("C", C, dev, dtype, bc, G * M),
               0 if gate is None else _tokens("gate", gate, dev, dtype, shape, ch)]
    f32 = torch.float32
    _whole("A", A, dev, f32, (ch, M))
    _whole("D", D, dev, f32, (ch,))
    _whole("dt_bias", dt_bias, dev, f32, (ch,))
    return ScanDims(n, T, num_seqs, ch, M, G, code, grad_code, 1 if dt_softplus else 0,
                    *strides)


def _scan_ptrs(x, dt, A, B, C, D, gate, dt_bias):
    return (x.data_ptr(), dt.data_ptr(), A.data_ptr(), B.data_ptr(), C.data_ptr(), _ptr(D),
            _ptr(gate), _ptr(dt_bias))


def selective_scan_fwd(x, dt, A, B, C, D: Optional[torch.Tensor] = None,
                       gate: Optional[torch.Tensor] = None,
                       dt_bias: Optional[torch.Tensor] = None, dt_softplus: bool = False,
                       S0: Optional[torch.Tensor] = None,
                       cu_seqlens: Optional[torch.Tensor] = None,
                       output_final_state: bool = True, workspace: Optional[torch.Tensor] = None,
                       out: Optional[torch.Tensor] = None,
                       final_state: Optional[torch.Tensor] = None
                       ) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """The selective state space scan over prompts:
        h_t = exp(dt_t A) h_{t-1} + dt_t B_t x_t,  y_t = sum_n C_t h_t + D x_t,  o = y silu(gate)
    x, dt, gate [B,T,channels]; B, C [B,T,groups,d_state] (these five in one dtype, each may be
    a column slice); A fp32 [channels,d_state]; D, dt_bias fp32 [channels]; dt_softplus: the
    step is softplus(dt + dt_bias); S0 fp32 [N,channels,d_state]; cu_seqlens int32 [N+1] for a
    packed batch. Returns (o [B,T,channels], S_T fp32 [N,channels,d_state] or None)."""
    N, num_seqs = _sequences(cu_seqlens, _batch(x), _gpu_of("x", x))
    d = _scan_dims(x, dt, A, B, C, D, gate, dt_bias, dt_softplus, num_seqs, 0)
    dev, shape, f32 = x.device, x.shape, torch.float32
    st_shape = (N, d.channels, d.d_state)
    s0 = _whole("S0", S0, dev, f32, st_shape)
    o = torch.empty(shape, dtype=x.dtype, device=dev) if out is None else out
    po = _whole("out", o, dev, x.dtype, shape)
    S_T = None
    if output_final_state:
        S_T = torch.empty(st_shape, dtype=f32, device=dev) if final_state is None else final_state
    ps = _whole("final_state", S_T, dev, f32, st_shape)
    if workspace is None:
        need = lib().gdn2_selective_scan_fwd_workspace_bytes(ctypes.byref(d))
        workspace = torch.empty(need, dtype=torch.uint8, device=dev) if need else None
    else:
        _need_gpu("workspace", workspace, dev)
    pw, nw = (None, 0) if workspace is None else (workspace.data_ptr(), workspace.numel())
    _call(dev, lib().gdn2_selective_scan_fwd, *_scan_ptrs(x, dt, A, B, C, D, gate, dt_bias), s0,
          _ptr(cu_seqlens), po, ps, ctypes.byref(d), pw, nw)
    return o, S_T


def selective_scan_fwd_workspace_bytes(batch: int, seqlen: int, channels: int, d_state: int,
                                       groups: int, dtype: torch.dtype, num_seqs: int = 0) -> int:
    d = ScanDims(batch, seqlen, num_seqs, channels, d_state, groups, _dtype_code(dtype))
    return int(lib().gdn2_selective_scan_fwd_workspace_bytes(ctypes.byref(d)))


def selective_scan_bwd(x, dt, A, B, C, dO, D: Optional[torch.Tensor] = None,
                       gate: Optional[torch.Tensor] = None,
                       dt_bias: Optional[torch.Tensor] = None, dt_softplus: bool = False,
                       S0: Optional[torch.Tensor] = None,
                       cu_seqlens: Optional[torch.Tensor] = None,
                       dS_T: Optional[torch.Tensor] = None,
                       workspace: Optional[torch.Tensor] = None) -> dict:
    """Gradients of selective_scan_fwd given dO = dL/do [B,T,channels] (x's dtype or fp32) and
    dS_T = dL/dS_T (None: zero). Returns dx, ddt, dB, dC (and dgate) in dO's dtype, dA (and dD,
    ddt_bias, dS0) in fp32, each optional one for the argument given."""
    N, num_seqs = _sequences(cu_seqlens, _batch(x), _gpu_of("x", x))
    d = _scan_dims(x, dt, A, B, C, D, gate, dt_bias, dt_softplus, num_seqs,
                   _grad_code("dO", dO, x.dtype))
    dev, shape, f32 = x.device, x.shape, torch.float32
    st_shape = (N, d.channels, d.d_state)
    s0 = _whole("S0", S0, dev, f32, st_shape)
    pdo = _whole("dO", dO, dev, dO.dtype, shape)
    pds = _whole("dS_T", dS_T, dev, f32, st_shape)
    new = lambda like, dtype: None if like is None else torch.empty(  # noqa: E731
        like.shape, dtype=dtype, device=dev)
    gt = dO.dtype
    out = {"dx": new(x, gt), "ddt": new(dt, gt), "dA": new(A, f32), "dB": new(B, gt),
           "dC": new(C, gt), "dD": new(D, f32), "dgate": new(gate, gt),
           "ddt_bias": new(dt_bias, f32), "dS0": new(S0, f32)}
    ws = _workspace(workspace, lib().gdn2_selective_scan_bwd_workspace_bytes(ctypes.byref(d)), dev)
    _call(dev, lib().gdn2_selective_scan_bwd, *_scan_ptrs(x, dt, A, B, C, D, gate, dt_bias), s0,
          _ptr(cu_seqlens), pdo, pds, *(_ptr(t) for t in out.values()), ctypes.byref(d),
          ws.data_ptr(), ws.numel())
    return {n: t for n, t in out.items() if t is not None}


def selective_scan_bwd_workspace_bytes(batch: int, seqlen: int, channels: int, d_state: int,
                                       groups: int, dtype: torch.dtype, num_seqs: int = 0) -> int:
    d = ScanDims(batch, seqlen, num_seqs, channels, d_state, groups, _dtype_code(dtype))
    return int(lib().gdn2_selective_scan_bwd_workspace_bytes(ctypes.byref(d)))


def selective_scan_step(x, dt, A, B, C, state, D: Optional[torch.Tensor] = None,
                        gate: Optional[torch.Tensor] = None,
                        dt_bias: Optional[torch.Tensor] = None, dt_softplus: bool = False,
                        state_idx: Optional[torch.Tensor] = None,
                        out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """T tokens of each of N sequences (x [N,T,channels], the other inputs as in
    selective_scan_fwd) against a pool of states [num_slots,channels,d_state], fp32 or bf16,
    updated in place. state_idx int32 [N]: the slot of each sequence (None: slot n); an entry
    outside the pool marks padding (zero o rows, no state touched). Returns o [N,T,channels]."""
    d = _scan_dims(x, dt, A, B, C, D, gate, dt_bias, dt_softplus, 0, 0)
    dev, shape = x.device, x.shape
    if state.dim() != 3:
        raise ValueError(f"state must be [num_slots,{d.channels},{d.d_state}]")
    if state.dtype not in (torch.float32, torch.bfloat16):
        raise TypeError("state must be float32 or bfloat16")
    slots = _fits("the number of slots", state.shape[0])
    ps = _whole("state", state, dev, state.dtype, (slots, d.channels, d.d_state))
    o = torch.empty(shape, dtype=x.dtype, device=dev) if out is None else out
    po = _whole("out", o, dev, x.dtype, shape)
    _call(dev, lib().gdn2_selective_scan_step, *_scan_ptrs(x, dt, A, B, C, D, gate, dt_bias), ps,
          0 if state.dtype == torch.float32 else 1, _state_idx(state_idx, shape[0], dev), slots,
          po, ctypes.byref(d))
    return o


# ---- block norm --------------------------------------------------------------------------


def _rows(name: str, t: torch.Tensor, dev, dtype, shape) -> int:
    """Checks an input of rows that may be a column slice. Returns the elements between rows."""
    if t.dtype != dtype or t.device != dev or t.shape != shape:
        _check(name, t, dev, dtype, shape)
    d = shape[-1]
    if t.is_contiguous():
        return d
    if d > 1 and t.stride(-1) != 1:
        raise ValueError(f"{name}: every row's values must be contiguous")
    step, rows = None, 1
    for i in range(t.dim() - 2, -1, -1):
        if t.shape[i] == 1:
            continue
        if step is None:
            step = t.stride(i)
        elif t.stride(i) != rows * step:
            raise ValueError(f"{name}: the rows must follow each other at one stride")
        rows *= t.shape[i]
    step = d if step is None else step
    if step < d:
        raise ValueError(f"{name}: rows overlap (stride {step}, {d} values)")
    return step


def _norm_dims(x, gate, residual, norm_weight, scale, next_weight, eps, grad_code) -> NormDims:
    """The checked dims of a block norm call."""
    dev, dtype, shape = _gpu_of("x", x), x.dtype, x.shape
    if x.dim() < 1:
        raise ValueError("x must be [*rows,d]")
    d = _fits("d", shape[-1])
    code = _dtype_code(dtype)
    xs = _rows("x", x, dev, dtype, shape)
    gs = 0 if gate is None else _rows("gate", gate, dev, dtype, shape)
    rcode = code
    if residual is not None:
        rcode = _dtype_code(residual.dtype)
        if residual.dtype not in (dtype, torch.float32):
            raise TypeError(f"residual has dtype {residual.dtype}, expected {dtype} or torch.float32")
        _whole("residual", residual, dev, residual.dtype, shape)
    for name, t in (("norm_weight", norm_weight), ("scale", scale), ("next_weight", next_weight)):
        _whole(name, t, dev, torch.float32, (d,))
    rows = x.numel() // d if d else 0
    return NormDims(rows, d, code, rcode, grad_code, eps, xs, gs)


def block_norm_fwd(x, norm_weight: Optional[torch.Tensor] = None,
                   gate: Optional[torch.Tensor] = None, residual: Optional[torch.Tensor] = None,
                   scale: Optional[torch.Tensor] = None,
                   next_weight: Optional[torch.Tensor] = None, eps: float = 1e-5,
                   out: Optional[torch.Tensor] = None, next_out: Optional[torch.Tensor] = None
                   ) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """The norms after and before a block, with its gate, residual and scale:
        h = residual + scale (rms(x) norm_weight silu(gate)),   y = rms(h) next_weight
    where every stage but h is taken only if its argument is given. x, gate [*rows,d] (each may
    be a column slice); residual [*rows,d] in x's dtype or fp32; norm_weight, scale, next_weight
    fp32 [d]. Returns (h in residual's dtype, y in x's dtype or None). out may be residual."""
    d = _norm_dims(x, gate, residual, norm_weight, scale, next_weight, eps, 0)
    dev, shape = x.device, x.shape
    ht = x.dtype if residual is None else residual.dtype
    h = torch.empty(shape, dtype=ht, device=dev) if out is None else out
    ph = _whole("out", h, dev, ht, shape)
    y = None
    if next_weight is not None:
        y = torch.empty(shape, dtype=x.dtype, device=dev) if next_out is None else next_out
    py = _whole("next_out", y, dev, x.dtype, shape)
    _call(dev, lib().gdn2_block_norm_fwd, x.data_ptr(), _ptr(gate), _ptr(residual),
          _ptr(norm_weight), _ptr(scale), _ptr(next_weight), ph, py, ctypes.byref(d))
    return h, y


def block_norm_bwd(x, dh: Optional[torch.Tensor] = None, dy: Optional[torch.Tensor] = None,
                   norm_weight: Optional[torch.Tensor] = None,
                   gate: Optional[torch.Tensor] = None, residual: Optional[torch.Tensor] = None,
                   scale: Optional[torch.Tensor] = None,
                   next_weight: Optional[torch.Tensor] = None, eps: float = 1e-5,
                   grad_dtype: Optional[torch.dtype] = None,
                   workspace: Optional[torch.Tensor] = None) -> dict:
    """Gradients of block_norm_fwd given dh = dL/dh (None: zero, with next_weight only) and dy =
    dL/dy (with next_weight). grad_dtype, the type of the token gradients in and out, is x's or
    fp32 (None: dy's, else dh's, else x's); dh and dresidual have it too, and are fp32 with an
    fp32 residual. Returns dx, and dgate, dresidual, dnorm_weight,
    dscale, dnext_weight for the arguments given."""
    if (dy is None) != (next_weight is None):
        raise ValueError("dy and next_weight go together")
    if dh is None and dy is None:
        raise ValueError("without next_weight, dh is required")
    dev, shape = x.device, x.shape
    wide = residual is not None and residual.dtype == torch.float32 and x.dtype != torch.float32
    gt = grad_dtype
    if gt is None:      # with an fp32 residual dh says nothing about the other gradients' type
        gt = dy.dtype if dy is not None else x.dtype if wide else dh.dtype
    if gt not in (x.dtype, torch.float32):
        raise TypeError(f"gradients have dtype {gt}, expected {x.dtype} or torch.float32")
    d = _norm_dims(x, gate, residual, norm_weight, scale, next_weight, eps, _dtype_code(gt))
    ht = torch.float32 if wide else gt
    pdh = _whole("dh", dh, dev, ht, shape)
    pdy = _whole("dy", dy, dev, gt, shape)
    new = lambda like, dtype: None if like is None else torch.empty(  # noqa: E731
        like.shape, dtype=dtype, device=dev)
    f32 = torch.float32
    out = {"dx": new(x, gt), "dgate": new(gate, gt), "dresidual": new(residual, ht),
           "dnorm_weight": new(norm_weight, f32), "dscale": new(scale, f32),
           "dnext_weight": new(next_weight, f32)}
    ws = _workspace(workspace, lib().gdn2_block_norm_bwd_workspace_bytes(ctypes.byref(d)), dev)
    _call(dev, lib().gdn2_block_norm_bwd, x.data_ptr(), _ptr(gate), _ptr(residual),
          _ptr(norm_weight), _ptr(scale), _ptr(next_weight), pdh, pdy,
          *(_ptr(t) for t in out.values()), ctypes.byref(d), ws.data_ptr(), ws.numel())
    return {n: t for n, t in out.items() if t is not None}


def block_norm_bwd_workspace_bytes(rows: int, d: int) -> int:
    n = NormDims(rows, d, 0, 0, 0, 0.0, 0, 0)
    return int(lib().gdn2_block_norm_bwd_workspace_bytes(ctypes.byref(n)))
