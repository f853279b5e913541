"""Linears of 8-bit tokens and 8-bit weights.

The consumer of `LayerQuantizer(..., bits=8, group_size=-1)`: its codes, laid
out once as a `Weight`, are multiplied with activations that are quantized a
token at a time, by themselves (`quantize_tokens`), after a gated activation
(`gate`) or as the output of the norm between two blocks (`block_norm`).  All
arithmetic happens in libgptq.so; this module allocates the outputs.
"""
from __future__ import annotations

from dataclasses import dataclass

import torch

from . import binding as B


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
    M, K = x.shape
    t = Tokens(empty_codes(M, K, x.device) if codes else None,
               torch.empty(M, dtype=torch.float32, device=x.device),
               torch.empty(M, dtype=torch.int32, device=x.device),
               torch.empty(M, K, dtype=x.dtype, device=x.device) if hat else None)
    B.gptq_quantize_tokens(t.codes, t.scales, t.sums, x, gate, t.hat)
    return t


def block_norm(block: torch.Tensor | None, residual: torch.Tensor | None, pre_weight: torch.Tensor | None = None, *,
               post_norm: bool = False, post_weight: torch.Tensor | None = None, gate: torch.Tensor | None = None,
               gate_rows: int = 0, scale: float = 1.0, eps: float = 1e-6, quantize: bool = False, keep_stream: bool = True,
               keep_out: bool = True):
    """(r', out) with r' = residual + scale * gate * norm(block) and out =
    norm(r'); with `quantize` out is `Tokens`.  Without `keep_stream` r', and
    without `keep_out` out, is None and not stored.  See gptq_block_norm."""
    x = block if block is not None else residual
    M, D = x.shape
    stream_out = torch.empty(M, D, dtype=x.dtype, device=x.device) if keep_stream else None
    t, outs = None, {}
    if keep_out and quantize:
        t = Tokens(empty_codes(M, D, x.device), torch.empty(M, dtype=torch.float32, device=x.device),
                   torch.empty(M, dtype=torch.int32, device=x.device))
        outs = {"q": t.codes, "q_scales": t.scales, "q_sums": t.sums}
    elif keep_out:
        t = torch.empty(M, D, dtype=x.dtype, device=x.device)
        outs = {"out": t}
    B.gptq_block_norm(block, residual, pre_weight, stream_out=stream_out, post_norm=post_norm, post_weight=post_weight,
                      gate=gate, gate_rows=gate_rows, scale=scale, eps=eps, **outs)
    return stream_out, t


def linear(tokens: Tokens, weight: Weight, bias: torch.Tensor | None = None,
           dtype: torch.dtype = torch.bfloat16) -> torch.Tensor:
    """Y [M, N] of the given type: the tokens times the weights transposed."""
    y = torch.empty(tokens.codes.shape[0], weight.codes.shape[0], dtype=dtype, device=tokens.codes.device)
    B.gptq_w8a8_gemm(y, tokens.codes, tokens.scales, weight.codes, weight.scales, tokens.sums, weight.zeros, bias)
    return y
