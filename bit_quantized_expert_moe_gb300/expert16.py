"""The 16-bit expert operators: products grouped by expert with their gradients,
the gated activation with the routing weight, and the norms around a block.

Argument marshalling only, as in the rest of the binding: shapes and types are
checked here, everything else by the library.  The checks and pointers are
spelled out in place: a small call takes a few microseconds on the GPU, and
helper calls on the host would take longer than that.  `offsets` and `row_map` are the
`offsets` and `sorted` of permute().
"""
from __future__ import annotations

import torch

from . import _check, _ptr, _stream, lib, workspace

_DTYPES = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}
_I32, _F32 = torch.int32, torch.float32
_empty = torch.empty
_raw_stream, _device = torch._C._cuda_getCurrentRawStream, torch._C._cuda_getDevice  # as _stream(None)


def _dtype(dt: torch.dtype) -> int:
    d = _DTYPES.get(dt)
    if d is None:
        raise ValueError(f"bfloat16, float16 or float32 tensor expected, not {dt}")
    return d


def _bad(t: torch.Tensor):
    raise ValueError("contiguous tensor expected" if t.is_cuda else "device tensor expected")


def _refuse(what: str, t: torch.Tensor, shape: tuple, dtype: torch.dtype):
    raise ValueError(f"{what}: shape {tuple(shape)} of {dtype} expected, not {tuple(t.shape)} of {t.dtype}")


# ---------------------------------------------------------------------------
def grouped_mm_workspace_size(R: int, E: int, N: int, K: int) -> int:
    return lib().moe_grouped_mm_workspace_size(R, E, N, K)


def _grouped(fn, what: str, dt, a, b, offsets, R: int, E: int, N: int, K: int, out, ws, stream):
    if offsets.shape != (E + 1,) or offsets.dtype is not _I32:
        _refuse("offsets", offsets, (E + 1,), _I32)
    if ws is None:
        ws = workspace(grouped_mm_workspace_size(R, E, N, K), offsets.device)
    st = fn(_DTYPES.get(dt, -1), a.data_ptr() if a.is_cuda and a.is_contiguous() else _bad(a),
            b.data_ptr() if b.is_cuda and b.is_contiguous() else _bad(b),
            offsets.data_ptr() if offsets.is_cuda and offsets.is_contiguous() else _bad(offsets), R, E, N, K,
            out.data_ptr() if out.is_cuda and out.is_contiguous() else _bad(out),
            ws.data_ptr() if ws.is_cuda and ws.is_contiguous() else _bad(ws), ws.numel(),
            _raw_stream(_device()) if stream is None else stream.cuda_stream)
    if st:
        _check(st, what)
    return out


def grouped_mm(x: torch.Tensor, w: torch.Tensor, offsets: torch.Tensor, y: torch.Tensor | None = None,
               ws: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """y[r] = w[e] x[r] for the rows r of every expert e: x [R, K], w [E, N, K]."""
    (R, K), (E, N, Kw), dt = x.shape, w.shape, x.dtype
    if Kw != K or w.dtype is not dt:
        _refuse("w", w, (E, N, K), dt)
    if y is None:
        y = _empty((R, N), dtype=dt, device=x.device)
    elif y.shape != (R, N) or y.dtype is not dt:
        _refuse("y", y, (R, N), dt)
    return _grouped(lib().moe_grouped_mm, "moe_grouped_mm", dt, x, w, offsets, R, E, N, K, y, ws, stream)


def grouped_mm_dx(dy: torch.Tensor, w: torch.Tensor, offsets: torch.Tensor, dx: torch.Tensor | None = None,
                  ws: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Gradient of grouped_mm in x: dx[r] = dy[r] w[e]."""
    (R, N), (E, Nw, K), dt = dy.shape, w.shape, dy.dtype
    if Nw != N or w.dtype is not dt:
        _refuse("w", w, (E, N, K), dt)
    if dx is None:
        dx = _empty((R, K), dtype=dt, device=dy.device)
    elif dx.shape != (R, K) or dx.dtype is not dt:
        _refuse("dx", dx, (R, K), dt)
    return _grouped(lib().moe_grouped_mm_dx, "moe_grouped_mm_dx", dt, dy, w, offsets, R, E, N, K, dx, ws, stream)


def grouped_mm_dw(dy: torch.Tensor, x: torch.Tensor, offsets: torch.Tensor, dw: torch.Tensor | None = None,
                  ws: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Gradient of grouped_mm in w: dw[e] = sum of dy[r]^T x[r] over the expert's rows."""
    (R, N), (Rx, K), E, dt = dy.shape, x.shape, offsets.numel() - 1, dy.dtype
    if Rx != R or x.dtype is not dt:
        _refuse("x", x, (R, K), dt)
    if dw is None:
        dw = _empty((E, N, K), dtype=dt, device=dy.device)
    elif dw.shape != (E, N, K) or dw.dtype is not dt:
        _refuse("dw", dw, (E, N, K), dt)
    return _grouped(lib().moe_grouped_mm_dw, "moe_grouped_mm_dw", dt, dy, x, offsets, R, E, N, K, dw, ws, stream)


# ---------------------------------------------------------------------------
def _check_row_weights(R: int, F2: int, row_w, row_map) -> None:
    if F2 & 1:
        raise ValueError("gu holds the gate and the up half of every row")
    if row_w is not None and (row_w.shape != (R,) or row_w.dtype is not _F32):
        _refuse("row_w", row_w, (R,), _F32)
    if row_map is not None and (row_map.shape != (R,) or row_map.dtype is not _I32):
        _refuse("row_map", row_map, (R,), _I32)


def swiglu(gu: torch.Tensor, row_w: torch.Tensor | None = None, row_map: torch.Tensor | None = None,
           h: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """h[r] = row_w[row_map[r]] SiLU(gate) up for gu [R, 2F], gate then up."""
    (R, F2), dt = gu.shape, gu.dtype
    _check_row_weights(R, F2, row_w, row_map)
    F = F2 >> 1
    if h is None:
        h = _empty((R, F), dtype=dt, device=gu.device)
    elif h.shape != (R, F) or h.dtype is not dt:
        _refuse("h", h, (R, F), dt)
    st = lib().moe_swiglu(_dtype(dt), gu.data_ptr() if gu.is_cuda and gu.is_contiguous() else _bad(gu),
                          None if row_w is None else row_w.data_ptr() if row_w.is_cuda and row_w.is_contiguous() else _bad(row_w),
                          None if row_map is None else row_map.data_ptr() if row_map.is_cuda and row_map.is_contiguous() else _bad(row_map), R, F,
                          h.data_ptr() if h.is_cuda and h.is_contiguous() else _bad(h),
                          _raw_stream(_device()) if stream is None else stream.cuda_stream)
    if st:
        _check(st, "moe_swiglu")
    return h


def swiglu_backward(dh: torch.Tensor, gu: torch.Tensor, row_w: torch.Tensor | None = None,
                    row_map: torch.Tensor | None = None, dgu: torch.Tensor | None = None,
                    drow_w: torch.Tensor | None = None, stream=None):
    """Gradients of swiglu: (dgu [R, 2F], drow_w [R] fp32, or None without row_w)."""
    (R, F2), dt = gu.shape, gu.dtype
    _check_row_weights(R, F2, row_w, row_map)
    F = F2 >> 1
    if dh.shape != (R, F) or dh.dtype is not dt:
        _refuse("dh", dh, (R, F), dt)
    if dgu is None:
        dgu = _empty((R, F2), dtype=dt, device=gu.device)
    elif dgu.shape != gu.shape or dgu.dtype is not dt:
        _refuse("dgu", dgu, gu.shape, dt)
    if drow_w is not None:
        if drow_w.shape != (R,) or drow_w.dtype is not _F32:
            _refuse("drow_w", drow_w, (R,), _F32)
    elif row_w is not None:
        drow_w = _empty((R,), dtype=_F32, device=gu.device)
    st = lib().moe_swiglu_backward(_dtype(dt), _ptr(dh), _ptr(gu), _ptr(row_w), _ptr(row_map), R, F, _ptr(dgu),
                                   _ptr(drow_w), _stream(stream))
    if st:
        _check(st, "moe_swiglu_backward")
    return dgu, drow_w


# ---------------------------------------------------------------------------
def _norm_params(T: int, D: int, dt, gamma_post, gate, gamma_pre) -> tuple[int, int]:
    """(gate rows, parameter type); dt where there is no parameter."""
    G, pt = 1, None
    if gate is not None:
        pt = gate.dtype
        G = gate.shape[0] if gate.dim() == 2 else 0
        if G < 1 or T % G or gate.shape[1] != D:
            raise ValueError(f"gate: [G, {D}] with G a divisor of {T} rows expected, not {tuple(gate.shape)}")
    if gamma_post is not None:
        pt = pt or gamma_post.dtype
        if gamma_post.shape != (D,) or gamma_post.dtype is not pt:
            _refuse("gamma_post", gamma_post, (D,), pt)
    if gamma_pre is not None:
        pt = pt or gamma_pre.dtype
        if gamma_pre.shape != (D,) or gamma_pre.dtype is not pt:
            _refuse("gamma_pre", gamma_pre, (D,), pt)
    return G, _dtype(pt or dt)


def block_norm(x: torch.Tensor, y: torch.Tensor | None = None, gamma_post: torch.Tensor | None = None,
               gate: torch.Tensor | None = None, gamma_pre: torch.Tensor | None = None, alpha: float = 1.0,
               eps: float = 1e-6, x_out: torch.Tensor | None = None, h: torch.Tensor | None = None, stream=None):
    """x_out = x + alpha gate norm(y) gamma_post and h = norm(x_out) gamma_pre.

    Returns (x_out, h): x_out is None without y, h is None without gamma_pre.
    gamma_post None: y enters unnormalised; gate [G, D] None: 1; x_out may be x."""
    shape, dt = x.shape, x.dtype
    T, D = shape
    G, pt = _norm_params(T, D, dt, gamma_post, gate, gamma_pre)
    if y is not None and (y.shape != shape or y.dtype is not dt):
        _refuse("y", y, shape, dt)
    if x_out is not None:
        if x_out.shape != shape or x_out.dtype is not dt:
            _refuse("x_out", x_out, shape, dt)
    elif y is not None:
        x_out = _empty(shape, dtype=dt, device=x.device)
    if h is not None:
        if h.shape != shape or h.dtype is not dt:
            _refuse("h", h, shape, dt)
    elif gamma_pre is not None:
        h = _empty(shape, dtype=dt, device=x.device)
    st = lib().moe_block_norm(_dtype(dt), pt, T, D, G, alpha, eps,
                              None if gamma_post is None else gamma_post.data_ptr() if gamma_post.is_cuda and gamma_post.is_contiguous() else _bad(gamma_post),
                              None if gate is None else gate.data_ptr() if gate.is_cuda and gate.is_contiguous() else _bad(gate),
                              None if gamma_pre is None else gamma_pre.data_ptr() if gamma_pre.is_cuda and gamma_pre.is_contiguous() else _bad(gamma_pre),
                              x.data_ptr() if x.is_cuda and x.is_contiguous() else _bad(x),
                              None if y is None else y.data_ptr() if y.is_cuda and y.is_contiguous() else _bad(y),
                              None if x_out is None else x_out.data_ptr() if x_out.is_cuda and x_out.is_contiguous() else _bad(x_out),
                              None if h is None else h.data_ptr() if h.is_cuda and h.is_contiguous() else _bad(h),
                              _raw_stream(_device()) if stream is None else stream.cuda_stream)
    if st:
        _check(st, "moe_block_norm")
    return x_out, h


def block_norm_backward_workspace_size(T: int, D: int, G: int = 1) -> int:
    return lib().moe_block_norm_backward_workspace_size(T, D, G)


def block_norm_backward(x_out: torch.Tensor, y: torch.Tensor | None = None, dx_out: torch.Tensor | None = None,
                        dh: torch.Tensor | None = None, gamma_post: torch.Tensor | None = None,
                        gate: torch.Tensor | None = None, gamma_pre: torch.Tensor | None = None, alpha: float = 1.0,
                        eps: float = 1e-6, ws: torch.Tensor | None = None, stream=None):
    """Gradients of block_norm at the stored x_out (x, where there is no y):
    (dx, dy, dgamma_post, dgate, dgamma_pre), None for what was not there."""
    shape, dt = x_out.shape, x_out.dtype
    T, D = shape
    G, pt = _norm_params(T, D, dt, gamma_post, gate, gamma_pre)
    if dx_out is not None and (dx_out.shape != shape or dx_out.dtype is not dt):
        _refuse("dx_out", dx_out, shape, dt)
    if dh is not None and (dh.shape != shape or dh.dtype is not dt):
        _refuse("dh", dh, shape, dt)
    dev = x_out.device
    dx, dy = _empty(shape, dtype=dt, device=dev), None
    if y is not None:
        if y.shape != shape or y.dtype is not dt:
            _refuse("y", y, shape, dt)
        dy = _empty(shape, dtype=dt, device=dev)
    dpost = None if gamma_post is None else _empty((D,), dtype=gamma_post.dtype, device=dev)
    dgate = None if gate is None else _empty((G, D), dtype=gate.dtype, device=dev)
    dpre = None if gamma_pre is None else _empty((D,), dtype=gamma_pre.dtype, device=dev)
    if ws is None:
        ws = workspace(block_norm_backward_workspace_size(T, D, G), x_out.device)
    st = lib().moe_block_norm_backward(
        _dtype(dt), pt, T, D, G, alpha, eps,
        None if gamma_post is None else gamma_post.data_ptr() if gamma_post.is_cuda and gamma_post.is_contiguous() else _bad(gamma_post),
        None if gate is None else gate.data_ptr() if gate.is_cuda and gate.is_contiguous() else _bad(gate),
        None if gamma_pre is None else gamma_pre.data_ptr() if gamma_pre.is_cuda and gamma_pre.is_contiguous() else _bad(gamma_pre),
        x_out.data_ptr() if x_out.is_cuda and x_out.is_contiguous() else _bad(x_out),
        None if y is None else y.data_ptr() if y.is_cuda and y.is_contiguous() else _bad(y),
        None if dx_out is None else dx_out.data_ptr() if dx_out.is_cuda and dx_out.is_contiguous() else _bad(dx_out),
        None if dh is None else dh.data_ptr() if dh.is_cuda and dh.is_contiguous() else _bad(dh),
        dx.data_ptr(), None if dy is None else dy.data_ptr(), None if dpost is None else dpost.data_ptr(),
        None if dgate is None else dgate.data_ptr(), None if dpre is None else dpre.data_ptr(),
        ws.data_ptr() if ws.is_cuda and ws.is_contiguous() else _bad(ws), ws.numel(),
        _raw_stream(_device()) if stream is None else stream.cuda_stream)
    if st:
        _check(st, "moe_block_norm_backward")
    return dx, dy, dpost, dgate, dpre
