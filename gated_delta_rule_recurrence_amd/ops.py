"""PyTorch-facing entry points with the same names as the C ABI.

PyTorch supplies device memory and the current HIP stream; the arithmetic all
happens in libgdr.so.  Tensors must be contiguous, on one GPU, and q, k, v,
g, beta, dy share one dtype (torch.float32 or torch.bfloat16); states are
torch.float32.  The operators around the recurrence (further down) take rows
with a stride too.
"""
from __future__ import annotations

import functools
import math
from dataclasses import dataclass
from typing import Optional

import torch

from . import _lib

DEFAULT_CHUNK = 64

_DTYPES = {torch.float32: _lib.GDR_F32, torch.bfloat16: _lib.GDR_BF16}


def _ptr(t: Optional[torch.Tensor]) -> int:
    return 0 if t is None else t.data_ptr()


def _check_tensor(name, t, shape, dtype, device):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if t.device.type != "cuda":
        raise ValueError(f"{name} must be a GPU tensor (the library has no CPU path)")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.dtype != dtype:
        raise ValueError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


@dataclass
class Saved:
    """What gdr_forward leaves for gdr_backward (opaque fp32 buffer), with
    the settings the backward must repeat."""

    ckpt: torch.Tensor
    chunk: int
    log_decay: bool = False
    mask: Optional[torch.Tensor] = None
    # the forward's v: the backward replays the tiles from it when chunk > 64
    v: Optional[torch.Tensor] = None


def shape_of(q, v, chunk, dtype, log_decay=False) -> _lib.GdrShape:
    B, T, Hk, Dk = q.shape
    Hv, Dv = v.shape[2], v.shape[3]
    decay = _lib.GDR_DECAY_LOG if log_decay else _lib.GDR_DECAY_G
    return _lib.make_shape(B, T, Hk, Hv, Dk, Dv, chunk, _DTYPES[dtype], decay)


def _as_mask(mask, B, T, device):
    if mask is None:
        return None
    if mask.dtype == torch.bool:
        mask = mask.to(torch.uint8)
    _check_tensor("mask", mask, (B, T), torch.uint8, device)
    return mask


def _stream(device) -> int:
    return torch.cuda.current_stream(device).cuda_stream


def gdr_forward(q, k, v, g, beta, S0=None, *, chunk=DEFAULT_CHUNK, save=True,
                out_state=True, y=None, S_T=None, ckpt=None, workspace=None,
                log_decay=False, mask=None):
    """Forward pass.  Returns (y, S_T or None, Saved or None).

    q, k [B,T,Hk,Dk]; v [B,T,Hv,Dv]; g, beta [B,T,Hv]; S0 [B,Hv,Dv,Dk] fp32
    or None.  Output and scratch buffers may be passed in to avoid allocation.
    log_decay: g holds the log of the decay (GDR_DECAY_LOG).
    mask: [B,T] torch.uint8 (or bool) or None; a step with mask 0 leaves the
    state unchanged (an identity step).  S_T may be S0 (in place).
    """
    if q.dtype not in _DTYPES:
        raise ValueError(f"unsupported dtype {q.dtype}")
    dev, dt = q.device, q.dtype
    B, T, Hk, Dk = q.shape
    Hv, Dv = v.shape[2], v.shape[3]
    _check_tensor("q", q, (B, T, Hk, Dk), dt, dev)
    _check_tensor("k", k, (B, T, Hk, Dk), dt, dev)
    _check_tensor("v", v, (B, T, Hv, Dv), dt, dev)
    _check_tensor("g", g, (B, T, Hv), dt, dev)
    _check_tensor("beta", beta, (B, T, Hv), dt, dev)
    if S0 is not None:
        _check_tensor("S0", S0, (B, Hv, Dv, Dk), torch.float32, dev)
    mask = _as_mask(mask, B, T, dev)
    shape = shape_of(q, v, chunk, dt, log_decay)
    if y is None:
        y = torch.empty((B, T, Hv, Dv), dtype=dt, device=dev)
    _check_tensor("y", y, (B, T, Hv, Dv), dt, dev)
    if out_state and S_T is None:
        S_T = torch.empty((B, Hv, Dv, Dk), dtype=torch.float32, device=dev)
    if not out_state:
        S_T = None
    saved = None
    if save:
        nbytes = _lib.checkpoint_bytes(shape)
        if ckpt is None:
            ckpt = torch.empty((max(nbytes, 1),), dtype=torch.uint8, device=dev)
        if ckpt.numel() * ckpt.element_size() < nbytes:
            raise ValueError("ckpt buffer too small")
        saved = Saved(ckpt, chunk, bool(log_decay), mask, v if chunk > 64 else None)
    wbytes = _lib.forward_workspace_bytes(shape)
    if wbytes > 0 and workspace is None:
        workspace = torch.empty((wbytes,), dtype=torch.uint8, device=dev)
    if wbytes > 0 and workspace.numel() * workspace.element_size() < wbytes:
        raise ValueError("forward workspace too small")
    st = _lib.forward_raw(shape, _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta),
                          _ptr(S0), _ptr(y), _ptr(S_T),
                          _ptr(saved.ckpt) if saved else 0,
                          _ptr(workspace) if wbytes > 0 else 0, wbytes, _stream(dev),
                          mask=_ptr(mask))
    _lib.check(st, "gdr_forward")
    return y, S_T, saved


def gdr_backward(q, k, g, beta, saved: Saved, dy, dS_T=None, *, want_dS0=True,
                 workspace=None, out=None):
    """Backward pass.  Returns (dq, dk, dv, dg, dbeta, dS0 or None).

    With a log-decay forward (saved.log_decay), dg is dL/d(log g).  For
    chunk > 64 the backward replays the forward tiles from saved.v, the
    forward's v."""
    dev, dt = q.device, q.dtype
    B, T, Hk, Dk = q.shape
    Hv, Dv = dy.shape[2], dy.shape[3]
    _check_tensor("q", q, (B, T, Hk, Dk), dt, dev)
    _check_tensor("k", k, (B, T, Hk, Dk), dt, dev)
    _check_tensor("g", g, (B, T, Hv), dt, dev)
    _check_tensor("beta", beta, (B, T, Hv), dt, dev)
    _check_tensor("dy", dy, (B, T, Hv, Dv), dt, dev)
    if dS_T is not None:
        _check_tensor("dS_T", dS_T, (B, Hv, Dv, Dk), torch.float32, dev)
    shape = shape_of(q, dy, saved.chunk, dt, saved.log_decay)
    if out is None:
        dq = torch.empty_like(q)
        dk = torch.empty_like(k)
        dv = torch.empty((B, T, Hv, Dv), dtype=dt, device=dev)
        dg = torch.empty_like(g)
        dbeta = torch.empty_like(beta)
        dS0 = (torch.empty((B, Hv, Dv, Dk), dtype=torch.float32, device=dev)
               if want_dS0 else None)
    else:
        dq, dk, dv, dg, dbeta, dS0 = out
    nbytes = _lib.backward_workspace_bytes(shape)
    if workspace is None:
        workspace = torch.empty((max(nbytes, 1),), dtype=torch.uint8, device=dev)
    st = _lib.backward_raw(shape, _ptr(q), _ptr(k), _ptr(g), _ptr(beta),
                           _ptr(saved.ckpt), _ptr(dy), _ptr(dS_T), _ptr(dq),
                           _ptr(dk), _ptr(dv), _ptr(dg), _ptr(dbeta), _ptr(dS0),
                           _ptr(workspace), workspace.numel() * workspace.element_size(),
                           _stream(dev), mask=_ptr(saved.mask), v=_ptr(saved.v))
    _lib.check(st, "gdr_backward")
    return dq, dk, dv, dg, dbeta, dS0


class GatedDeltaRule(torch.autograd.Function):
    """y, S_T = gated_delta_rule(q, k, v, g, beta, S0) with the library VJP."""

    @staticmethod
    def forward(ctx, q, k, v, g, beta, S0, chunk, log_decay=False, mask=None):
        y, S_T, saved = gdr_forward(q, k, v, g, beta, S0, chunk=chunk,
                                    log_decay=log_decay, mask=mask)
        ctx.has_S0 = S0 is not None
        # v is needed again only when the backward replays the tiles (chunk >
        # 64); it then goes through save_for_backward like the other inputs
        ctx.with_v = saved.v is not None
        saved.v = None
        ctx.saved = saved
        ctx.save_for_backward(q, k, g, beta, *((v,) if ctx.with_v else ()))
        return y, S_T

    @staticmethod
    def backward(ctx, dy, dS_T):
        q, k, g, beta, *rest = ctx.saved_tensors
        if ctx.with_v:
            ctx.saved.v = rest[0]
        # autograd materialises absent cotangents as zeros
        dy = dy.contiguous()
        dS_T = None if dS_T is None else dS_T.contiguous()
        dq, dk, dv, dg, dbeta, dS0 = gdr_backward(
            q, k, g, beta, ctx.saved, dy, dS_T, want_dS0=ctx.has_S0)
        return dq, dk, dv, dg, dbeta, (dS0 if ctx.has_S0 else None), None, None, None


def gated_delta_rule(q, k, v, g, beta, S0=None, chunk=DEFAULT_CHUNK, log_decay=False,
                     mask=None):
    """Autograd-enabled forward: returns (y, S_T).  With log_decay, g holds
    the log of the decay and its gradient is dL/d(log g); mask [B,T] marks
    identity steps with 0."""
    return GatedDeltaRule.apply(q, k, v, g, beta, S0, chunk, log_decay, mask)


# ---- the operators around the recurrence ----------------------------------------
#
# Activations are rows: [B, T, ...] or, with spans, [rows, ...] (any leading
# dimensions that collapse to one row stride, so slices of a wider projection
# pass as they are; the first row lies on a 16-byte boundary).  A T given
# without spans cuts all the rows into sequences of T, whatever their leading
# dimensions: rows [2, 5, ...] with T = 2 are five sequences.  spans is int32 [B, 2] on the device, the first row and
# the row past the last of each sequence, ascending and disjoint; T is then
# the longest sequence's length (by default the number of rows, which sizes
# grid and workspace for that).  Rows of no sequence are neither read nor
# written: buffers that a call allocates hold zeros there.

_ACTS = {None: _lib.GDR_ACT_NONE, "none": _lib.GDR_ACT_NONE, "silu": _lib.GDR_ACT_SILU}


def _act(act) -> int:
    if act not in _ACTS:
        raise ValueError(f"act must be None, 'none' or 'silu', got {act!r}")
    return _ACTS[act]


def _dense(name, t, shape, dtype, device):
    """_check_tensor, for the calls whose host time counts: one condition
    where all is well."""
    if not (isinstance(t, torch.Tensor) and t.shape == shape and t.dtype == dtype
            and t.device == device and t.is_contiguous()):
        _check_tensor(name, t, shape, dtype, device)


def _row_stride(name, t, tail, dtype, device, rows=None):
    """Checks a tensor of rows whose last dimensions are `tail` and dense;
    returns (rows, elements from one row to the next)."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if t.dtype != dtype:
        raise ValueError(f"{name} has dtype {t.dtype}, expected {dtype}")
    k = len(tail)
    shape = t.shape
    if len(shape) <= k or (shape[-1] != tail[0] if k == 1 else shape[-k:] != tail):
        raise ValueError(f"{name} has shape {tuple(shape)}, expected rows of {tuple(tail)}")
    width = tail[0] if k == 1 else math.prod(tail)
    if t.is_contiguous():
        n, step = (t.numel() // width if width else 0), width
    else:
        n, step = _collapse(name, shape, t.stride(), k, width)
    if rows is not None and n != rows:
        raise ValueError(f"{name} has {n} rows, expected {rows}")
    return n, step


def _row_stride_as(name, t, like, step, tail, dtype, device, rows):
    """_row_stride(..)[1] of rows laid out as `like`'s, checked before, as a
    rule: one condition then."""
    if (isinstance(t, torch.Tensor) and t.dtype == dtype and t.device == device
            and t.shape == like.shape and t.stride() == like.stride()):
        return step
    return _row_stride(name, t, tail, dtype, device, rows)[1]


def _collapse(name, shape, strides, k, width):
    """(rows, row stride) of a tensor that is not dense as a whole."""
    inner = 1
    for size, stride in zip(reversed(shape[-k:]), reversed(strides[-k:])):
        if size != 1 and stride != inner:
            raise ValueError(f"{name}: the elements of a row must be contiguous (got strides "
                             f"{strides})")
        inner *= size
    n, step = 1, width
    for size, stride in zip(reversed(shape[:-k]), reversed(strides[:-k])):
        if size == 0:
            return 0, width
        if size == 1:
            continue
        if n == 1:
            step = stride
        elif stride != step * n:
            raise ValueError(f"{name}: the rows must lie at one stride (got strides {strides})")
        n *= size
    if n > 1 and step < width:
        raise ValueError(f"{name}: the rows overlap (got strides {strides})")
    return n, step


def _gpu(x):
    if not isinstance(x, torch.Tensor):
        raise TypeError("the rows must be a torch.Tensor")
    if x.device.type != "cuda":
        raise ValueError("the rows must be a GPU tensor (the library has no CPU path)")
    if x.dtype not in _DTYPES:
        raise ValueError(f"unsupported dtype {x.dtype}")
    return x.device, x.dtype


def _sequences(x, rows, tail, spans, T, device):
    """(B, T) of rows x [..., *tail]."""
    if spans is not None:
        if spans.dim() != 2:
            raise ValueError(f"spans has shape {tuple(spans.shape)}, expected (B, 2)")
        _dense("spans", spans, (spans.shape[0], 2), torch.int32, device)
        return spans.shape[0], rows if T is None else int(T)
    batch = x.dim() == len(tail) + 2  # [B, T, ...]
    if T is None:
        if not batch:
            raise ValueError("T is needed where the rows are not [B, T, ...]")
        return x.shape[0], x.shape[1]
    T = int(T)
    if batch and x.shape[1] == T:
        return x.shape[0], T
    if T < 0 or (rows % T if T else rows):
        raise ValueError(f"{rows} rows are not sequences of {T}")
    return (rows // T if T else 0), T


def _weight_dtype(name, w):
    if w.dtype not in _DTYPES:
        raise ValueError(f"{name} has unsupported dtype {w.dtype}")
    return w.dtype


def _out(given, name, shape, dtype, device):
    if given is None:
        return torch.empty(shape, dtype=dtype, device=device)
    _dense(name, given, shape, dtype, device)
    return given


def _dense_like(t, spans=None):
    """A dense tensor of t's shape (an empty_like costs half of an empty)."""
    make = torch.empty_like if spans is None else torch.zeros_like
    return make(t, memory_format=torch.contiguous_format)


def _rows_out(given, name, like, spans=None):
    """The output rows of a call on rows `like`."""
    if given is None:
        return _dense_like(like, spans)
    _dense(name, given, like.shape, like.dtype, like.device)
    return given


def _scratch(workspace, nbytes, like, name="workspace"):
    if nbytes == 0:
        return None
    device = like.device
    if workspace is None:
        return like.new_empty(nbytes, dtype=torch.uint8)
    if workspace.numel() * workspace.element_size() < nbytes:
        raise ValueError(f"{name} too small")
    if workspace.device != device or not workspace.is_contiguous():
        raise ValueError(f"{name} must be contiguous and on {device}")
    return workspace


_current_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _raw_stream(device) -> int:
    """The current stream's handle without a Stream object around it (2 us
    of a call), where this PyTorch has that."""
    return _stream(device) if _current_raw_stream is None else _current_raw_stream(device.index)


def _launch(name, shape, tensors, device, workspace=None, nbytes=None):
    ptrs = [0 if t is None else t.data_ptr() for t in tensors]
    if nbytes is not None:
        ptrs.append(0 if workspace is None else workspace.data_ptr())
    if torch.cuda.current_device() == device.index:
        status = _lib.layer_raw(name, shape, ptrs, _raw_stream(device), nbytes)
    else:  # a stream's kernels are launched with its device current
        with torch.cuda.device(device):
            status = _lib.layer_raw(name, shape, ptrs, _raw_stream(device), nbytes)
    if status != 0:
        _lib.check(status, name)


def _gradient(t):
    """An incoming gradient as the library takes it: dense and on a 16-byte
    boundary (a dense view into the middle of another gradient may not be)."""
    t = t.contiguous()
    return t if t.data_ptr() % 16 == 0 else t.clone()


# The C structure of a call's sizes and the bytes of its buffers: they follow
# from the sizes alone, so that calls of the same sizes share them.

@functools.lru_cache(maxsize=1024)
def _conv_plan(*sizes):
    shape = _lib.GdrConvShape(*sizes, 0)
    return shape, _lib.size_of("gdr_conv_backward_workspace_bytes", shape)


@functools.lru_cache(maxsize=1024)
def _scan_plan(*sizes):
    shape = _lib.GdrScanShape(*sizes)
    return (shape, _lib.size_of("gdr_scan_checkpoint_bytes", shape),
            _lib.size_of("gdr_scan_forward_workspace_bytes", shape),
            _lib.size_of("gdr_scan_backward_workspace_bytes", shape))


@functools.lru_cache(maxsize=1024)
def _norm_plan(*sizes):
    shape = _lib.GdrNormShape(*sizes)
    return shape, _lib.size_of("gdr_norm_backward_workspace_bytes", shape)


@functools.lru_cache(maxsize=1024)
def _lin_plan(*sizes):
    shape = _lib.GdrLinShape(*sizes)
    return (shape, _lib.size_of("gdr_lin_checkpoint_bytes", shape),
            _lib.size_of("gdr_lin_forward_workspace_bytes", shape),
            _lib.size_of("gdr_lin_backward_workspace_bytes", shape))


@functools.lru_cache(maxsize=1024)
def _res_plan(*sizes):
    shape = _lib.GdrResShape(*sizes)
    return shape, _lib.size_of("gdr_res_backward_workspace_bytes", shape)


def _conv_sizes(x, weight, bias, state, spans, T, act):
    dev, dt = _gpu(x)
    if not isinstance(weight, torch.Tensor) or weight.dim() != 2:
        raise ValueError("weight must be a tensor [C, K]")
    C, K = weight.shape
    wdt = _weight_dtype("weight", weight)
    _dense("weight", weight, (C, K), wdt, dev)
    rows, xs = _row_stride("x", x, (C,), dt, dev)
    B, T = _sequences(x, rows, (C,), spans, T, dev)
    if bias is not None:
        _dense("bias", bias, (C,), wdt, dev)
    if state is not None:
        _dense("state", state, (B, K - 1, C), dt, dev)
    return _conv_plan(B, T, rows, C, K, xs, _DTYPES[dt], _DTYPES[wdt], _act(act))


def gdr_conv_forward(x, weight, bias=None, state=None, *, act="silu", spans=None, T=None,
                     out_state=True, y=None, state_out=None):
    """Short causal convolution.  Returns (y, state_out or None).

    x [B,T,C] (or rows, see above), weight [C,K], bias [C] or None, state
    [B,K-1,C] (the inputs before each sequence) or None.  state_out may be
    state (in place), and y may be x for at most 16 steps a sequence."""
    shape, _ = _conv_sizes(x, weight, bias, state, spans, T, act)
    dev, dt = x.device, x.dtype
    y = _rows_out(y, "y", x, spans)
    if not out_state:
        state_out = None
    else:
        state_out = _out(state_out, "state_out", (shape.B, shape.K - 1, shape.C), dt, dev)
    _launch("gdr_conv_forward", shape, (x, weight, bias, state, spans, y, state_out), dev)
    return y, state_out


def gdr_conv_backward(x, weight, bias, state, dy, dstate_out=None, *, act="silu", spans=None,
                      T=None, want_dstate=False, workspace=None):
    """Returns (dx, dweight, dbias or None, dstate or None)."""
    shape, nbytes = _conv_sizes(x, weight, bias, state, spans, T, act)
    dev, dt = x.device, x.dtype
    _dense("dy", dy, x.shape, dt, dev)
    window = (shape.B, shape.K - 1, shape.C)
    if dstate_out is not None:
        _dense("dstate_out", dstate_out, window, dt, dev)
    dx = _dense_like(x, spans)
    make = torch.empty_like if shape.B > 0 else torch.zeros_like
    dweight = make(weight)
    dbias = None if bias is None else make(bias)
    dstate = torch.empty(window, dtype=dt, device=dev) if want_dstate else None
    workspace = _scratch(workspace, nbytes, x)
    _launch("gdr_conv_backward", shape, (x, weight, bias, state, spans, dy, dstate_out, dx,
                                         dweight, dbias, dstate), dev, workspace, nbytes)
    return dx, dweight, dbias, dstate


@dataclass
class ScanSaved:
    """What gdr_scan_forward leaves for gdr_scan_backward (opaque fp32
    buffer), with the settings the backward must repeat."""

    ckpt: torch.Tensor
    spans: Optional[torch.Tensor]
    T: int
    softplus: bool


def _scan_sizes(u, dt, A, Bm, Cm, D, z, dt_bias, spans, T, softplus):
    dev, ty = _gpu(u)
    f32 = torch.float32
    if not isinstance(A, torch.Tensor) or A.dim() != 2:
        raise ValueError("A must be a tensor [C, N]")
    if not isinstance(Bm, torch.Tensor) or Bm.dim() < 3:
        raise ValueError("Bm must be a tensor [.., G, N]")
    C, N = A.shape
    G = Bm.shape[-2]
    rows, us = _row_stride("u", u, (C,), ty, dev)
    dts = _row_stride_as("dt", dt, u, us, (C,), ty, dev, rows)
    _, bs = _row_stride("Bm", Bm, (G, N), ty, dev, rows)
    cs = _row_stride_as("Cm", Cm, Bm, bs, (G, N), ty, dev, rows)
    zs = C if z is None else _row_stride_as("z", z, u, us, (C,), ty, dev, rows)
    _dense("A", A, (C, N), f32, dev)
    if D is not None:
        _dense("D", D, (C,), f32, dev)
    if dt_bias is not None:
        _dense("dt_bias", dt_bias, (C,), f32, dev)
    B, T = _sequences(u, rows, (C,), spans, T, dev)
    return _scan_plan(B, T, rows, C, N, G, us, dts, zs, bs, cs, _DTYPES[ty], 1 if softplus else 0)


def gdr_scan_forward(u, dt, A, Bm, Cm, D=None, z=None, dt_bias=None, S0=None, *, softplus=True,
                     spans=None, T=None, save=True, out_state=True, y=None, S_T=None, ckpt=None,
                     workspace=None):
    """Selective state space scan.  Returns (y, S_T or None, ScanSaved or None).

    u, dt, z [B,T,C] (or rows, see above); A [C,N], D, dt_bias [C] fp32; Bm,
    Cm [B,T,G,N]; S0 [B,C,N] fp32 or None.  S_T may be S0 (in place)."""
    shape, save_bytes, nbytes, _ = _scan_sizes(u, dt, A, Bm, Cm, D, z, dt_bias, spans, T, softplus)
    dev = u.device
    states = (shape.B, shape.C, shape.N)
    if S0 is not None:
        _dense("S0", S0, states, torch.float32, dev)
    y = _rows_out(y, "y", u, spans)
    S_T = _out(S_T, "S_T", states, torch.float32, dev) if out_state else None
    saved = None
    if save:
        ckpt = _scratch(ckpt, max(save_bytes, 1), u, "ckpt")
        saved = ScanSaved(ckpt, spans, shape.T, bool(softplus))
    workspace = _scratch(workspace, nbytes, u)
    _launch("gdr_scan_forward", shape, (u, dt, A, Bm, Cm, D, z, dt_bias, S0, spans, y, S_T,
                                        ckpt if save else None), dev, workspace, nbytes)
    return y, S_T, saved


def gdr_scan_backward(u, dt, A, Bm, Cm, D, z, dt_bias, saved: ScanSaved, dy, dS_T=None, *,
                      want_dS0=True, workspace=None):
    """Returns (du, ddt, dA, dBm, dCm, dD, dz, ddt_bias, dS0); None where the
    forward had no such input, and dS0 only where wanted."""
    spans = saved.spans
    shape, save_bytes, _, nbytes = _scan_sizes(u, dt, A, Bm, Cm, D, z, dt_bias, spans, saved.T,
                                               saved.softplus)
    dev, ty = u.device, u.dtype
    states = (shape.B, shape.C, shape.N)
    # (the kernel reads the states of as many rows as the inputs have)
    if not isinstance(saved.ckpt, torch.Tensor):
        raise TypeError("saved.ckpt must be a torch.Tensor")
    _scratch(saved.ckpt, save_bytes, u, "saved.ckpt")
    _dense("dy", dy, u.shape, ty, dev)
    if dS_T is not None:
        _dense("dS_T", dS_T, states, torch.float32, dev)
    du, ddt, dB, dC = [_dense_like(t, spans) for t in (u, dt, Bm, Cm)]
    dz = None if z is None else _dense_like(z, spans)
    make = torch.empty_like if shape.B > 0 else torch.zeros_like
    dA = make(A)
    dD = None if D is None else make(D)
    dbias = None if dt_bias is None else make(dt_bias)
    dS0 = torch.empty(states, dtype=torch.float32, device=dev) if want_dS0 else None
    workspace = _scratch(workspace, nbytes, u)
    _launch("gdr_scan_backward", shape, (u, dt, A, Bm, Cm, D, z, dt_bias, spans, saved.ckpt, dy,
                                         dS_T, du, ddt, dA, dB, dC, dD, dz, dbias, dS0), dev,
            workspace, nbytes)
    return du, ddt, dA, dB, dC, dD, dz, dbias, dS0


def _norm_sizes(x, weight, bias, z, groups, eps, center, act):
    dev, dt = _gpu(x)
    C = x.shape[-1]
    if groups < 1 or C % groups:
        raise ValueError(f"{C} channels are not {groups} groups")
    wdt, width = dt, C
    like = weight if weight is not None else bias
    if like is not None:  # weight and bias have one type and one shape
        wdt = _weight_dtype("weight" if weight is not None else "bias", like)
        width = C if like.numel() == C else C // groups
        if weight is not None:
            _dense("weight", weight, (width,), wdt, dev)
        if bias is not None:
            _dense("bias", bias, (width,), wdt, dev)
    rows, xs = _row_stride("x", x, (C,), dt, dev)
    zs = C
    if z is not None:
        if z.shape != x.shape:
            raise ValueError(f"z has shape {tuple(z.shape)}, expected {tuple(x.shape)}")
        zs = _row_stride_as("z", z, x, xs, (C,), dt, dev, rows)
    return _norm_plan(rows, C, groups, xs, zs, eps, _DTYPES[dt], _DTYPES[wdt], 1 if center else 0,
                      1 if width != C else 0, _act(act))


def gdr_norm_forward(x, weight=None, bias=None, z=None, *, groups, eps=1e-6, center=False,
                     act="silu", save=True, y=None, stats=None):
    """Group norm of the last dimension, in `groups` groups.  Returns (y,
    stats or None).  x, z [..., C]; weight, bias [C], or [C // groups] used by
    every group.  The activation takes z where there is one, else the normed
    rows."""
    shape, _ = _norm_sizes(x, weight, bias, z, groups, eps, center, act)
    dev = x.device
    y = _rows_out(y, "y", x)
    if save:
        stats = _out(stats, "stats", (shape.rows, shape.G, 2), torch.float32, dev)
    else:
        stats = None
    _launch("gdr_norm_forward", shape, (x, weight, bias, z, y, stats), dev)
    return y, stats


def gdr_norm_backward(x, weight, bias, z, stats, dy, *, groups, center=False, act="silu",
                      workspace=None):
    """Returns (dx, dweight, dbias, dz); None where the forward had no such
    input."""
    shape, nbytes = _norm_sizes(x, weight, bias, z, groups, 0.0, center, act)
    dev = x.device
    _dense("dy", dy, x.shape, x.dtype, dev)
    _dense("stats", stats, (shape.rows, shape.G, 2), torch.float32, dev)
    dx = _dense_like(x)
    dz = None if z is None else _dense_like(z)
    dweight = None if weight is None else torch.empty_like(weight)
    dbias = None if bias is None else torch.empty_like(bias)
    if weight is None and bias is None:
        nbytes = 0
    workspace = _scratch(workspace, nbytes, x)
    _launch("gdr_norm_backward", shape, (x, weight, bias, z, stats, dy, dx, dweight, dbias, dz),
            dev, workspace, nbytes)
    return dx, dweight, dbias, dz


@dataclass
class LinSaved:
    """What gdr_lin_forward leaves for gdr_lin_backward (opaque fp32 buffer),
    with the settings the backward must repeat."""

    ckpt: torch.Tensor
    spans: Optional[torch.Tensor]
    T: int
    scale: float


def _lin_sizes(q, k, v, log_g, scale, spans, T):
    dev, ty = _gpu(q)
    if q.dim() < 3:
        raise ValueError("q must be a tensor [.., Hk, Dk]")
    if not isinstance(v, torch.Tensor) or v.dim() < 3:
        raise ValueError("v must be a tensor [.., Hv, Dv]")
    heads, wide = tuple(q.shape[-2:]), tuple(v.shape[-2:])
    rows, qs = _row_stride("q", q, heads, ty, dev)
    ks = _row_stride_as("k", k, q, qs, heads, ty, dev, rows)
    _, vs = _row_stride("v", v, wide, ty, dev, rows)
    Hv = wide[0]
    gs, gt, per_head = Hv, torch.float32, 0
    if log_g is not None:
        if not isinstance(log_g, torch.Tensor):
            raise TypeError("log_g must be a torch.Tensor")
        gt = _weight_dtype("log_g", log_g)
        if log_g.dim() == 1:
            _dense("log_g", log_g, (Hv,), gt, dev)
            per_head = 1
        else:
            _, gs = _row_stride("log_g", log_g, (Hv,), gt, dev, rows)
    B, T = _sequences(q, rows, heads, spans, T, dev)
    return _lin_plan(B, T, rows, heads[0], Hv, heads[1], wide[1], qs, ks, vs, gs, float(scale),
                     _DTYPES[ty], _DTYPES[gt], per_head)


def gdr_lin_forward(q, k, v, log_g=None, S0=None, *, scale=1.0, spans=None, T=None, save=True,
                    out_state=True, y=None, S_T=None, ckpt=None, workspace=None):
    """Linear attention with a decay for each head.  Returns (y, S_T or None,
    LinSaved or None).

    q, k [B,T,Hk,Dk], v [B,T,Hv,Dv] (or rows, see above); log_g [B,T,Hv], or
    [Hv] for one decay per head, of either type, or None (no decay); S0
    [B,Hv,Dv,Dk] fp32 or None.  S_T may be S0 (in place)."""
    shape, save_bytes, nbytes, _ = _lin_sizes(q, k, v, log_g, scale, spans, T)
    dev = q.device
    states = (shape.B, shape.Hv, shape.Dv, shape.Dk)
    if S0 is not None:
        _dense("S0", S0, states, torch.float32, dev)
    y = _rows_out(y, "y", v, spans)
    S_T = _out(S_T, "S_T", states, torch.float32, dev) if out_state else None
    saved = None
    if save:
        ckpt = _scratch(ckpt, max(save_bytes, 1), q, "ckpt")
        saved = LinSaved(ckpt, spans, shape.T, float(scale))
    workspace = _scratch(workspace, nbytes, q)
    _launch("gdr_lin_forward", shape, (q, k, v, log_g, S0, spans, y, S_T, ckpt if save else None),
            dev, workspace, nbytes)
    return y, S_T, saved


def gdr_lin_backward(q, k, v, log_g, saved: LinSaved, dy, dS_T=None, *, want_dlog_g=True,
                     want_dS0=True, workspace=None):
    """Returns (dq, dk, dv, dlog_g, dS0); dlog_g and dS0 None where not
    wanted, dlog_g also where the forward had no log_g."""
    spans = saved.spans
    shape, save_bytes, _, nbytes = _lin_sizes(q, k, v, log_g, saved.scale, spans, saved.T)
    dev, ty = q.device, q.dtype
    states = (shape.B, shape.Hv, shape.Dv, shape.Dk)
    # (the kernel reads the states of as many rows as the inputs have)
    if not isinstance(saved.ckpt, torch.Tensor):
        raise TypeError("saved.ckpt must be a torch.Tensor")
    _scratch(saved.ckpt, save_bytes, q, "saved.ckpt")
    _dense("dy", dy, v.shape, ty, dev)
    if dS_T is not None:
        _dense("dS_T", dS_T, states, torch.float32, dev)
    dq, dk, dv = [_dense_like(t, spans) for t in (q, k, v)]
    dlog_g = None
    if log_g is not None and want_dlog_g:
        dlog_g = _dense_like(log_g, spans if shape.B > 0 else True)
    dS0 = torch.empty(states, dtype=torch.float32, device=dev) if want_dS0 else None
    workspace = _scratch(workspace, nbytes, q)
    _launch("gdr_lin_backward", shape, (q, k, v, log_g, spans, saved.ckpt, dy, dS_T, dq, dk, dv,
                                        dlog_g, dS0), dev, workspace, nbytes)
    return dq, dk, dv, dlog_g, dS0


def _res_sizes(x, residual, gate, post_weight, post_bias, pre_weight, pre_bias, alpha, eps, post,
               pre, center, weight_offset):
    dev, dt = _gpu(x)
    if x.dim() < 2:
        raise ValueError("x must be a tensor [.., C]")
    C = x.shape[-1]
    if not isinstance(residual, torch.Tensor):
        raise TypeError("residual must be a torch.Tensor")
    rdt = _weight_dtype("residual", residual)
    if residual.shape != x.shape:
        raise ValueError(f"residual has shape {tuple(residual.shape)}, expected {tuple(x.shape)}")
    rows, xs = _row_stride("x", x, (C,), dt, dev)
    _, rs = _row_stride("residual", residual, (C,), rdt, dev, rows)
    wdt = None
    for name, w, used in (("post_weight", post_weight, post), ("post_bias", post_bias, post),
                          ("pre_weight", pre_weight, pre), ("pre_bias", pre_bias, pre)):
        if w is None:
            continue
        if not used:
            raise ValueError(f"{name} is given for a norm that is not taken")
        if not isinstance(w, torch.Tensor):
            raise TypeError(f"{name} must be a torch.Tensor")
        wdt = _weight_dtype(name, w) if wdt is None else wdt  # they have one type
        _dense(name, w, (C,), wdt, dev)
    gate_rows, gdt, gs = 0, dt, C
    if gate is not None:
        if not isinstance(gate, torch.Tensor):
            raise TypeError("gate must be a torch.Tensor")
        gdt = _weight_dtype("gate", gate)
        lead = x.shape[:-1]
        if gate.dim() == 1:
            _dense("gate", gate, (C,), gdt, dev)
        elif gate.shape == x.shape:
            gate_rows, gs = 1, _row_stride("gate", gate, (C,), gdt, dev, rows)[1]
        elif gate.shape in ((*lead[:-1], C), (*lead[:-1], 1, C)):
            gate_rows = lead[-1]
            _, gs = _row_stride("gate", gate, (C,), gdt, dev)
        else:
            raise ValueError(f"gate has shape {tuple(gate.shape)}, expected (C,), that of x, or "
                             f"one row for each sequence [B, C]")
        gate_rows = max(gate_rows, 0)
    return _res_plan(rows, C, gate_rows, xs, rs, gs, float(alpha), float(eps),
                     float(weight_offset), _DTYPES[dt], _DTYPES[rdt], _DTYPES[wdt or dt],
                     _DTYPES[gdt], 1 if post else 0, 1 if pre else 0, 1 if center else 0)


def gdr_res_forward(x, residual, gate=None, post_weight=None, post_bias=None, pre_weight=None,
                    pre_bias=None, *, alpha=1.0, eps=1e-6, post=True, pre=True, center=False,
                    weight_offset=0.0, save=True, y=None, h=None, stats=None):
    """The norms around a block: h = residual + alpha gate N(x; post), y =
    N(h; pre).  Returns (y or None, h, stats or None).

    x [..., C] is what the block made, residual the sum so far (x's shape; fp32
    or x's type).  gate is [C], of x's shape, or [B, C] with one row for each
    sequence of x [B, T, C]; of either type.  The weights [C] are used as
    weight + weight_offset; post and pre say which of the norms are taken.
    h may be residual (in place)."""
    shape, _ = _res_sizes(x, residual, gate, post_weight, post_bias, pre_weight, pre_bias, alpha,
                          eps, post, pre, center, weight_offset)
    dev = x.device
    y = _rows_out(y, "y", x) if pre else None
    h = _rows_out(h, "h", residual)
    stats = _out(stats, "stats", (shape.rows, 4), torch.float32, dev) if save else None
    _launch("gdr_res_forward", shape, (x, residual, gate, post_weight, post_bias, pre_weight,
                                       pre_bias, y, h, stats), dev)
    return y, h, stats


def gdr_res_backward(x, residual, gate, post_weight, post_bias, pre_weight, pre_bias, stats, dy,
                     dh=None, *, alpha=1.0, eps=1e-6, post=True, pre=True, center=False,
                     weight_offset=0.0, workspace=None):
    """Returns (dx, dresidual, dgate, dpost_weight, dpost_bias, dpre_weight,
    dpre_bias); None where the forward had no such input.  residual is the
    forward's input, not h; dy is None without the pre norm."""
    shape, nbytes = _res_sizes(x, residual, gate, post_weight, post_bias, pre_weight, pre_bias,
                               alpha, eps, post, pre, center, weight_offset)
    dev = x.device
    if pre:
        _dense("dy", dy, x.shape, x.dtype, dev)
    if dh is not None:
        _dense("dh", dh, residual.shape, residual.dtype, dev)
    elif not pre:
        raise ValueError("dh is needed without the pre norm")
    _dense("stats", stats, (shape.rows, 4), torch.float32, dev)
    dx, dr = _dense_like(x), _dense_like(residual)
    make = torch.empty_like if shape.rows > 0 else torch.zeros_like
    dgate = None if gate is None else make(gate, memory_format=torch.contiguous_format)
    dw = [None if w is None else make(w) for w in (post_weight, post_bias, pre_weight, pre_bias)]
    workspace = _scratch(workspace, nbytes, x)
    _launch("gdr_res_backward", shape, (x, residual, gate, post_weight, post_bias, pre_weight,
                                        pre_bias, stats, dy if pre else None, dh, dx, dr, dgate,
                                        *dw), dev, workspace, nbytes)
    return (dx, dr, dgate, *dw)


def _wanted(args):
    """Whether a gradient of any of them will be asked for."""
    return torch.is_grad_enabled() and any(t is not None and t.requires_grad for t in args)


class CausalConv(torch.autograd.Function):
    """y, state_out = causal_conv(x, weight, bias, state) with the library VJP."""

    @staticmethod
    def forward(ctx, x, weight, bias, state, act, spans, T):
        y, state_out = gdr_conv_forward(x, weight, bias, state, act=act, spans=spans, T=T)
        ctx.settings = (act, T)
        ctx.save_for_backward(x, weight, bias, state, spans)
        return y, state_out

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dy, dstate_out):
        x, weight, bias, state, spans = ctx.saved_tensors
        act, T = ctx.settings
        dx, dw, db, ds = gdr_conv_backward(
            x, weight, bias, state, _gradient(dy), _gradient(dstate_out), act=act, spans=spans, T=T,
            want_dstate=state is not None)
        return dx, dw, db, ds, None, None, None


def causal_conv(x, weight, bias=None, state=None, *, act="silu", spans=None, T=None):
    """Autograd-enabled short causal convolution: returns (y, state_out)."""
    return CausalConv.apply(x, weight, bias, state, act, spans, T)


class SelectiveScan(torch.autograd.Function):
    """y, S_T = selective_scan(...) with the library VJP."""

    @staticmethod
    def forward(ctx, u, dt, A, Bm, Cm, D, z, dt_bias, S0, softplus, spans, T, save):
        y, S_T, ctx.saved = gdr_scan_forward(u, dt, A, Bm, Cm, D, z, dt_bias, S0,
                                             softplus=softplus, spans=spans, T=T, save=save)
        ctx.has_S0 = S0 is not None
        # (spans too, so that a change of theirs in between is noticed)
        ctx.save_for_backward(u, dt, A, Bm, Cm, D, z, dt_bias, spans)
        return y, S_T

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dy, dS_T):
        grads = gdr_scan_backward(*ctx.saved_tensors[:8], ctx.saved, _gradient(dy),
                                  _gradient(dS_T), want_dS0=ctx.has_S0)
        return (*grads, None, None, None, None)


def selective_scan(u, dt, A, Bm, Cm, D=None, z=None, dt_bias=None, S0=None, *, softplus=True,
                   spans=None, T=None):
    """Autograd-enabled selective state space scan: returns (y, S_T).  The
    states for the backward are saved only where a gradient is wanted."""
    args = (u, dt, A, Bm, Cm, D, z, dt_bias, S0)
    return SelectiveScan.apply(*args, softplus, spans, T, _wanted(args))


class GroupNorm(torch.autograd.Function):
    """y = group_norm(x, weight, bias, z) with the library VJP."""

    @staticmethod
    def forward(ctx, x, weight, bias, z, groups, eps, center, act, save):
        y, stats = gdr_norm_forward(x, weight, bias, z, groups=groups, eps=eps, center=center,
                                    act=act, save=save)
        ctx.settings = dict(groups=groups, center=center, act=act)
        ctx.save_for_backward(x, weight, bias, z, stats)
        return y

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dy):
        dx, dw, db, dz = gdr_norm_backward(*ctx.saved_tensors, _gradient(dy), **ctx.settings)
        return dx, dw, db, dz, None, None, None, None, None


def group_norm(x, weight=None, bias=None, z=None, *, groups, eps=1e-6, center=False, act="silu"):
    """Autograd-enabled group norm of the last dimension (see
    gdr_norm_forward): returns y."""
    return GroupNorm.apply(x, weight, bias, z, groups, eps, center, act,
                           _wanted((x, weight, bias, z)))


class LinearAttention(torch.autograd.Function):
    """y, S_T = linear_attention(...) with the library VJP."""

    @staticmethod
    def forward(ctx, q, k, v, log_g, S0, scale, spans, T, save):
        y, S_T, ctx.saved = gdr_lin_forward(q, k, v, log_g, S0, scale=scale, spans=spans, T=T,
                                            save=save)
        ctx.has_S0 = S0 is not None
        # (spans too, so that a change of theirs in between is noticed)
        ctx.save_for_backward(q, k, v, log_g, spans)
        return y, S_T

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dy, dS_T):
        q, k, v, log_g, _ = ctx.saved_tensors
        grads = gdr_lin_backward(q, k, v, log_g, ctx.saved, _gradient(dy), _gradient(dS_T),
                                 want_dlog_g=ctx.needs_input_grad[3], want_dS0=ctx.has_S0)
        return (*grads, None, None, None, None)


def linear_attention(q, k, v, log_g=None, S0=None, *, scale=1.0, spans=None, T=None):
    """Autograd-enabled linear attention with a decay for each head (see
    gdr_lin_forward): returns (y, S_T).  The states for the backward are saved
    only where a gradient is wanted."""
    return LinearAttention.apply(q, k, v, log_g, S0, scale, spans, T,
                                 _wanted((q, k, v, log_g, S0)))


class ResidualNorm(torch.autograd.Function):
    """y, h = residual_norm(...) with the library VJP."""

    @staticmethod
    def forward(ctx, x, residual, gate, post_weight, post_bias, pre_weight, pre_bias, how, save):
        y, h, stats = gdr_res_forward(x, residual, gate, post_weight, post_bias, pre_weight,
                                      pre_bias, save=save, **how)
        ctx.how = how
        ctx.save_for_backward(x, residual, gate, post_weight, post_bias, pre_weight, pre_bias,
                              stats)
        return y, h

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dy, dh):
        dy = None if dy is None else _gradient(dy)
        grads = gdr_res_backward(*ctx.saved_tensors, dy, _gradient(dh), **ctx.how)
        return (*grads, None, None)


def residual_norm(x, residual, gate=None, post_weight=None, post_bias=None, pre_weight=None,
                  pre_bias=None, *, alpha=1.0, eps=1e-6, post=True, pre=True, center=False,
                  weight_offset=0.0):
    """Autograd-enabled norms around a block (see gdr_res_forward): returns
    (y or None, h)."""
    args = (x, residual, gate, post_weight, post_bias, pre_weight, pre_bias)
    how = dict(alpha=alpha, eps=eps, post=post, pre=pre, center=center,
               weight_offset=weight_offset)
    return ResidualNorm.apply(*args, how, _wanted(args))
