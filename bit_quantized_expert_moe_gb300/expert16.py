"""The 16-bit expert operators: products grouped by expert with their gradients,
the gated activation with the routing weight, and the norms around a block; and
the operators of expert blocks in 8 and 16 bits: the layer norm before a block with
its gradients, rows to 8-bit codes, the 8-bit products grouped by expert, and the
whole layer of 16-bit experts for a few tokens.

    grouped_mm(x, w, offsets, y=None, ws=None, stream=None)
    grouped_mm_dx(dy, w, offsets, dx=None, ws=None, stream=None)
    grouped_mm_dw(dy, x, offsets, dw=None, ws=None, stream=None)
    swiglu(gu, row_w=None, row_map=None, h=None, stream=None)
    swiglu_backward(dh, gu, row_w=None, row_map=None, dgu=None, drow_w=None, stream=None)
    block_norm(x, y=None, gamma_post=None, gate=None, gamma_pre=None, alpha=1.0, eps=1e-6, x_out=None, h=None,
               stream=None)
    block_norm_backward(x_out, y=None, dx_out=None, dh=None, gamma_post=None, gate=None, gamma_pre=None, alpha=1.0,
                        eps=1e-6, ws=None, stream=None)
    layer_norm(x, y=None, gamma=None, beta=None, eps=1e-5, x_out=None, h=None, stream=None)
    layer_norm_backward(x_out, dh, dx_out=None, gamma=None, beta=None, eps=1e-5, ws=None, stream=None)
    quantize_rows(x, row_map=None, k=1, codes=None, scales=None, ws=None, stream=None)
    grouped_mm_i8(x, x_scale, w, w_scale, offsets, y=None, dtype=torch.bfloat16, ws=None, stream=None)
    expert_layer(x, logits, w13, w2, k, out=None, ids=None, ws=None, stream=None)

`offsets` and `row_map` are the `offsets` and `sorted` of permute().  Offsets
out of order or range set the error word of the `ws` that was given, which
get_device_error(ws) reads; without one nobody learns of them.  Outputs and
workspaces that are not given belong to the call's stream; operands that belong to
another have to outlast the call there (record_stream).  No call records an
autograd graph (operands that require gradients draw a warning where autograd
records): gradients come from grouped_mm_dx, grouped_mm_dw and the calls named
_backward; quantize_rows, grouped_mm_i8 and expert_layer have none.  The functions
are compiled (csrc/expert16_binding.cpp, argument marshalling only); this module
loads them at their first use.
"""
from __future__ import annotations

import importlib

from . import _check, lib

NAMES = ("grouped_mm", "grouped_mm_dx", "grouped_mm_dw", "swiglu", "swiglu_backward", "block_norm",
         "block_norm_backward", "layer_norm", "layer_norm_backward", "quantize_rows", "grouped_mm_i8",
         "expert_layer")


def load(name: str):
    """One of the compiled functions; raises if the library has not been built."""
    lib()
    try:
        m = importlib.import_module("bit_quantized_expert_moe_gb300._expert16")
    except ImportError as e:
        raise RuntimeError(f"the compiled binding cannot be loaded ({e}): build it with "
                           "`python -m bit_quantized_expert_moe_gb300.build`") from e
    m._init(_check)
    return getattr(m, name)


def unbuilt(name: str):
    """Stands for one of the functions while there is no library: like the others
    of the package it is there, and a call raises until the library is."""
    def call(*args, **kwargs):
        return load(name)(*args, **kwargs)
    call.__name__ = call.__qualname__ = name
    return call


def grouped_mm_workspace_size(R: int, E: int, N: int, K: int) -> int:
    return lib().moe_grouped_mm_workspace_size(R, E, N, K)


def block_norm_backward_workspace_size(T: int, D: int, G: int = 1) -> int:
    return lib().moe_block_norm_backward_workspace_size(T, D, G)


def layer_norm_backward_workspace_size(T: int, D: int) -> int:
    return lib().moe_layer_norm_backward_workspace_size(T, D)


def quantize_rows_workspace_size(T: int, R: int, D: int) -> int:
    return lib().moe_quantize_rows_workspace_size(T, R, D)


def grouped_mm_i8_workspace_size(R: int, E: int, N: int, K: int) -> int:
    return lib().moe_grouped_mm_i8_workspace_size(R, E, N, K)


def expert_layer_workspace_size(T: int, k: int, E: int, d: int, f: int) -> int:
    return lib().moe_expert_layer_workspace_size(T, k, E, d, f)
