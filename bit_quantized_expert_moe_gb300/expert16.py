"""The 16-bit expert operators: products grouped by expert with their gradients,
the gated activation with the routing weight, and the norms around a block.

Argument marshalling only, as in the rest of the binding: shapes and types are
checked here, everything else by the library.  `offsets` and `row_map` are the
`offsets` and `sorted` of permute().
"""
from __future__ import annotations

import torch

from . import _check, _ptr, _stream, lib, workspace

_DTYPES = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}


def _dtype(t: torch.Tensor) -> int:
    d = _DTYPES.get(t.dtype)
    if d is None:
        raise ValueError(f"bfloat16, float16 or float32 tensor expected, not {t.dtype}")
    return d


def _same_type(first: torch.Tensor, *others: torch.Tensor | None) -> None:
    for t in others:
        if t is not None and (t.dtype != first.dtype or t.device != first.device):
            raise ValueError("tensors of one type on one device expected")


def _want(t: torch.Tensor | None, what: str, *shape: int, dtype: torch.dtype | None = None) -> None:
    if t is not None and (tuple(t.shape) != shape or (dtype is not None and t.dtype != dtype)):
        raise ValueError(f"{what}: shape {shape}" + (f" of {dtype}" if dtype else "") +
                         f" expected, not {tuple(t.shape)} of {t.dtype}")


# ---------------------------------------------------------------------------
def grouped_mm_workspace_size(R: int, E: int, N: int, K: int) -> int:
    return lib().moe_grouped_mm_workspace_size(R, E, N, K)


def _grouped(fn: str, a, b, offsets, R: int, E: int, N: int, K: int, out, ws, stream):
    _want(offsets, "offsets", E + 1, dtype=torch.int32)
    if ws is None:
        ws = workspace(grouped_mm_workspace_size(R, E, N, K), offsets.device)
    _check(getattr(lib(), fn)(_dtype(a), _ptr(a), _ptr(b), _ptr(offsets), R, E, N, K, _ptr(out), _ptr(ws), ws.numel(),
                              _stream(stream)), fn)
    return out


def grouped_mm(x: torch.Tensor, w: torch.Tensor, offsets: torch.Tensor, y: torch.Tensor | None = None,
               ws: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """y[r] = w[e] x[r] for the rows r of every expert e: x [R, K], w [E, N, K]."""
    (R, K), (E, N, _) = x.shape, w.shape
    _want(w, "w", E, N, K)
    if y is None:
        y = torch.empty((R, N), dtype=x.dtype, device=x.device)
    _want(y, "y", R, N)
    _same_type(x, w, y)
    return _grouped("moe_grouped_mm", x, w, offsets, R, E, N, K, y, ws, stream)


def grouped_mm_dx(dy: torch.Tensor, w: torch.Tensor, offsets: torch.Tensor, dx: torch.Tensor | None = None,
                  ws: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Gradient of grouped_mm in x: dx[r] = dy[r] w[e]."""
    (R, N), (E, _, K) = dy.shape, w.shape
    _want(w, "w", E, N, K)
    if dx is None:
        dx = torch.empty((R, K), dtype=dy.dtype, device=dy.device)
    _want(dx, "dx", R, K)
    _same_type(dy, w, dx)
    return _grouped("moe_grouped_mm_dx", dy, w, offsets, R, E, N, K, dx, ws, stream)


def grouped_mm_dw(dy: torch.Tensor, x: torch.Tensor, offsets: torch.Tensor, dw: torch.Tensor | None = None,
                  ws: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Gradient of grouped_mm in w: dw[e] = sum of dy[r]^T x[r] over the expert's rows."""
    (R, N), K, E = dy.shape, x.shape[1], offsets.numel() - 1
    _want(x, "x", R, K)
    if dw is None:
        dw = torch.empty((E, N, K), dtype=dy.dtype, device=dy.device)
    _want(dw, "dw", E, N, K)
    _same_type(dy, x, dw)
    return _grouped("moe_grouped_mm_dw", dy, x, offsets, R, E, N, K, dw, ws, stream)


# ---------------------------------------------------------------------------
def _check_swiglu(gu, row_w, row_map) -> tuple[int, int]:
    R, F2 = gu.shape
    if F2 % 2:
        raise ValueError("gu holds the gate and the up half of every row")
    _want(row_w, "row_w", R, dtype=torch.float32)
    _want(row_map, "row_map", R, dtype=torch.int32)
    return R, F2 // 2


def swiglu(gu: torch.Tensor, row_w: torch.Tensor | None = None, row_map: torch.Tensor | None = None,
           h: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """h[r] = row_w[row_map[r]] SiLU(gate) up for gu [R, 2F], gate then up."""
    R, F = _check_swiglu(gu, row_w, row_map)
    if h is None:
        h = torch.empty((R, F), dtype=gu.dtype, device=gu.device)
    _want(h, "h", R, F, dtype=gu.dtype)
    _check(lib().moe_swiglu(_dtype(gu), _ptr(gu), _ptr(row_w), _ptr(row_map), R, F, _ptr(h), _stream(stream)),
           "moe_swiglu")
    return h


def swiglu_backward(dh: torch.Tensor, gu: torch.Tensor, row_w: torch.Tensor | None = None,
                    row_map: torch.Tensor | None = None, dgu: torch.Tensor | None = None,
                    drow_w: torch.Tensor | None = None, stream=None):
    """Gradients of swiglu: (dgu [R, 2F], drow_w [R] fp32, or None without row_w)."""
    R, F = _check_swiglu(gu, row_w, row_map)
    _want(dh, "dh", R, F, dtype=gu.dtype)
    if dgu is None:
        dgu = torch.empty_like(gu)
    if drow_w is None and row_w is not None:
        drow_w = torch.empty_like(row_w)
    _want(dgu, "dgu", R, 2 * F, dtype=gu.dtype)
    _want(drow_w, "drow_w", R, dtype=torch.float32)
    _check(lib().moe_swiglu_backward(_dtype(gu), _ptr(dh), _ptr(gu), _ptr(row_w), _ptr(row_map), R, F, _ptr(dgu),
                                     _ptr(drow_w), _stream(stream)), "moe_swiglu_backward")
    return dgu, drow_w


# ---------------------------------------------------------------------------
def _norm_params(x, gamma_post, gate, gamma_pre) -> tuple[int, int, int, int]:
    """(rows, width, gate rows, parameter type)"""
    T, D = x.shape
    G, given = 1, None
    if gate is not None:
        G = gate.shape[0] if gate.dim() == 2 else 0
        given = gate
    if G < 1 or T % G:
        raise ValueError("gate: [G, D] with G a divisor of the rows expected")
    _want(gate, "gate", G, D)
    _want(gamma_post, "gamma_post", D)
    _want(gamma_pre, "gamma_pre", D)
    for t in (gamma_post, gamma_pre):
        if t is not None:
            given = t if given is None else given
            _same_type(given, t)
    return T, D, G, _dtype(given if given is not None else x)


def block_norm(x: torch.Tensor, y: torch.Tensor | None = None, gamma_post: torch.Tensor | None = None,
               gate: torch.Tensor | None = None, gamma_pre: torch.Tensor | None = None, alpha: float = 1.0,
               eps: float = 1e-6, x_out: torch.Tensor | None = None, h: torch.Tensor | None = None, stream=None):
    """x_out = x + alpha gate norm(y) gamma_post and h = norm(x_out) gamma_pre.

    Returns (x_out, h): x_out is None without y, h is None without gamma_pre.
    gamma_post None: y enters unnormalised; gate [G, D] None: 1; x_out may be x."""
    T, D, G, pt = _norm_params(x, gamma_post, gate, gamma_pre)
    if x_out is None and y is not None:
        x_out = torch.empty_like(x)
    if h is None and gamma_pre is not None:
        h = torch.empty_like(x)
    for t, what in ((y, "y"), (x_out, "x_out"), (h, "h")):
        _want(t, what, T, D, dtype=x.dtype)
    _check(lib().moe_block_norm(_dtype(x), pt, T, D, G, alpha, eps, _ptr(gamma_post), _ptr(gate), _ptr(gamma_pre),
                                _ptr(x), _ptr(y), _ptr(x_out), _ptr(h), _stream(stream)), "moe_block_norm")
    return x_out, h


def block_norm_backward_workspace_size(T: int, D: int, G: int = 1) -> int:
    return lib().moe_block_norm_backward_workspace_size(T, D, G)


def block_norm_backward(x_out: torch.Tensor, y: torch.Tensor | None = None, dx_out: torch.Tensor | None = None,
                        dh: torch.Tensor | None = None, gamma_post: torch.Tensor | None = None,
                        gate: torch.Tensor | None = None, gamma_pre: torch.Tensor | None = None, alpha: float = 1.0,
                        eps: float = 1e-6, ws: torch.Tensor | None = None, stream=None):
    """Gradients of block_norm at the stored x_out (x, where there is no y):
    (dx, dy, dgamma_post, dgate, dgamma_pre), None for what was not there."""
    T, D, G, pt = _norm_params(x_out, gamma_post, gate, gamma_pre)
    for t, what in ((y, "y"), (dx_out, "dx_out"), (dh, "dh")):
        _want(t, what, T, D, dtype=x_out.dtype)
    dx = torch.empty_like(x_out)
    dy = torch.empty_like(y) if y is not None else None
    dpost, dgate, dpre = (torch.empty_like(t) if t is not None else None for t in (gamma_post, gate, gamma_pre))
    if ws is None:
        ws = workspace(block_norm_backward_workspace_size(T, D, G), x_out.device)
    _check(lib().moe_block_norm_backward(
        _dtype(x_out), pt, T, D, G, alpha, eps, _ptr(gamma_post), _ptr(gate), _ptr(gamma_pre), _ptr(x_out), _ptr(y),
        _ptr(dx_out), _ptr(dh), _ptr(dx), _ptr(dy), _ptr(dpost), _ptr(dgate), _ptr(dpre), _ptr(ws), ws.numel(),
        _stream(stream)), "moe_block_norm_backward")
    return dx, dy, dpost, dgate, dpre
