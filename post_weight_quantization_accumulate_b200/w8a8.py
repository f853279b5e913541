"""Linears of 8-bit tokens and 8-bit weights.

The consumer of `LayerQuantizer(..., bits=8, group_size=-1)`: its codes, laid
out once as a `Weight`, are multiplied with activations that are quantized a
token at a time, by themselves (`quantize_tokens`), after a gated activation
(`gate`) or as the output of the norm between two blocks (`block_norm`).  All
arithmetic happens in libgptq.so; the calls here allocate their outputs, run
on the current stream of the inputs' device and can be captured into graphs.
They go through _calls.so, which does in C++ what the gptq_* functions of
`binding` (for outputs of one's own, in place, or on a stream by argument) do
in Python; while a call allocates and launches, other Python threads run.
Nothing here is differentiated: outputs carry no gradient, whatever the inputs
require, so that what is trained must not pass through these calls.
"""
from __future__ import annotations

import os
from dataclasses import dataclass

import torch

from . import binding as B


_native = None


def _calls():
    """The loaded _calls module (raises if it has not been built)."""
    global _native
    if _native is None:
        B.lib()
        if not os.path.exists(os.path.join(os.path.dirname(os.path.abspath(__file__)), "_calls.so")):
            raise RuntimeError("_calls.so is missing: build it with "
                               "python -m post_weight_quantization_accumulate_b200.build")
        from . import _calls as native
        native.set_check(B._check)
        _native = native
    return _native


@dataclass
class Tokens:
    codes: torch.Tensor | None         # int8 [M, K], row pitch a multiple of 16
    scales: torch.Tensor               # float32 [M]
    sums: torch.Tensor | None = None   # int32 [M]: row sums of the codes
    hat: torch.Tensor | None = None    # [M, K]: the values the codes stand for


@dataclass
class Weight:
    codes: torch.Tensor                # int8 [N, K], row pitch a multiple of 16
    scales: torch.Tensor               # float32 [N]
    zeros: torch.Tensor | None = None  # int32 [N], or None for symmetric codes


def empty_codes(rows: int, cols: int, device) -> torch.Tensor:
    """int8 [rows, cols] at the pitch the 8-bit calls take."""
    codes = torch.empty(rows, (cols + 15) // 16 * 16, dtype=torch.int8, device=device)
    return codes if cols % 16 == 0 else codes[:, :cols]


def pack(layer) -> Weight:
    """The `Weight` of a `QuantizedLayer` with 8-bit codes and one scale a row."""
    if layer.codes is None or layer.scales.shape[1] != 1:
        raise ValueError("the 8-bit linear needs the layer's codes and one group a row (group_size=-1)")
    N, K = layer.codes.shape
    w = Weight(empty_codes(N, K, layer.codes.device), layer.scales[:, 0].clone(),
               torch.empty(N, dtype=torch.int32, device=layer.codes.device))
    B.gptq_w8a8_pack(w.codes, w.zeros, layer.codes, layer.zeros[:, 0].contiguous())
    return w


def quantize_tokens(x: torch.Tensor, gate: torch.Tensor | None = None, codes: bool = True,
                    hat: bool = False) -> Tokens:
    """The 8-bit tokens of x [M, K], or of silu(gate) * x; with `hat` also the
    values they stand for, in x's type."""
    return Tokens(*(_native or _calls()).quantize_tokens(x, gate, codes, hat))


def block_norm(block: torch.Tensor | None, residual: torch.Tensor | None, pre_weight: torch.Tensor | None = None, *,
               post_norm: bool = False, post_weight: torch.Tensor | None = None, gate: torch.Tensor | None = None,
               gate_rows: int = 0, scale: float = 1.0, eps: float = 1e-6, quantize: bool = False, keep_stream: bool = True,
               keep_out: bool = True):
    """(r', out) with r' = residual + scale * gate * norm(block) and out =
    norm(r'); with `quantize` out is `Tokens`, of its float32 values up to their
    rounding (beside a border between two codes either may be taken).  Without `keep_stream` r', and
    without `keep_out` out, is None and not stored.  See gptq_block_norm."""
    r, out, codes, scales, sums = (_native or _calls()).block_norm(
        block, residual, pre_weight, post_norm, post_weight, gate, gate_rows, scale, eps, quantize, keep_stream, keep_out)
    return r, (Tokens(codes, scales, sums) if codes is not None else out)


def linear(tokens: Tokens, weight: Weight, bias: torch.Tensor | None = None,
           dtype: torch.dtype = torch.bfloat16) -> torch.Tensor:
    """Y [M, N] of the given type: the tokens times the weights transposed."""
    return (_native or _calls()).linear(tokens.codes, tokens.scales, tokens.sums, weight.codes, weight.scales, weight.zeros,
                                        bias, dtype)
