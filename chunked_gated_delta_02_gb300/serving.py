"""The serving operators: public signatures over their native binding (csrc/binding.cpp).

``step`` continues a KDA forward by one token per request on states kept in a pool; ``la_fwd``
and ``la_step`` are linear attention with one decay per head, over prompts and by single tokens
(the fixed-decay linear attention of the cuLA README mirror, section "Quick Start", and its form
with a decay per token); ``norm_gate`` and ``add_norm`` are the norms of a layer around them. All
compute runs in libkda.so on the caller's current CUDA stream (include/kda.h has the formulas).

Unlike ``fwd``, these take token tensors with strides, as long as the last dimension is
contiguous: q, k and v may be views of one projection. Arguments are checked before anything runs;
a refused one raises TypeError or ValueError, a failed library call KDAError.
"""
from __future__ import annotations

import os
from typing import Optional, Tuple

import torch

from ._lib import lib

__all__ = ["step", "la_fwd", "la_step", "la_workspace_size", "norm_gate", "add_norm"]

_native = None


def _load():
    """The native binding; like libkda.so it is loaded by the first call, and there is no fallback."""
    global _native
    if _native is None:
        path = os.path.join(os.path.dirname(os.path.abspath(__file__)), "_serving.so")
        if not os.path.exists(path):
            raise OSError(f"_serving.so not found at {path}; build it first "
                          "(python -m chunked_gated_delta_02_gb300.build)")
        lib()
        from . import _serving
        _native = _serving
    return _native


def _kv(layout) -> bool:
    if layout == "vk":
        return False
    if layout == "kv":
        return True
    raise ValueError("state_layout must be 'vk' (rows [V,K]) or 'kv' (rows [K,V])")


def _scale(scale, q):
    if scale is None:
        return q.shape[-1] ** -0.5 if isinstance(q, torch.Tensor) and q.dim() and q.shape[-1] else 1.0
    return scale


def step(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, g: torch.Tensor, beta: torch.Tensor,
         A_log: torch.Tensor, state: torch.Tensor, dt_bias: Optional[torch.Tensor] = None,
         lower_bound: float = -5.0, scale: Optional[float] = None,
         state_indices: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
         state_layout: str = "vk") -> torch.Tensor:
    """One token of the KDA recurrence for each of N requests; ``state`` is updated in place.

    q, k: bf16 [N,H,K]; v: bf16 [N,H,V]; g: bf16 [N,H,K], or [N,H] for one decay per head (then
    dt_bias is [H]); beta: bf16 or fp32 [N,H] logits; A_log, dt_bias, lower_bound, scale as in
    ``fwd``. state: a pool [rows,H,V,K] (state_layout "vk") or [rows,H,K,V] ("kv"), fp32 or bf16,
    contiguous. state_indices: int32 [N], the pool row of each request (None: row n); a negative
    index is a padding entry (its output is 0, no state is touched), one past the pool is reported by
    ``device_status()``, and no row may occur twice. Returns o, bf16 [N,H,V].
    """
    return (_native or _load()).step(q, k, v, g, beta, A_log, state, dt_bias, lower_bound, _scale(scale, q),
                                     state_indices, out, _kv(state_layout))


def la_step(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, log_decay: torch.Tensor, state: torch.Tensor,
            state_indices: Optional[torch.Tensor] = None, scale: Optional[float] = None,
            out: Optional[torch.Tensor] = None, state_layout: str = "vk") -> torch.Tensor:
    """One token of linear attention with a decay per head for each of N requests.

    q, k: bf16 [N,Hk,K], Hk dividing the H heads of v (value head h reads head h // (H / Hk));
    v: bf16 [N,H,V]; log_decay: fp32 [H], or [N,H] for a decay per token; state, state_indices,
    out and state_layout as in ``step``. Returns o, bf16 [N,H,V]; ``state`` is updated in place.
    """
    return (_native or _load()).la_step(q, k, v, log_decay, state, state_indices, _scale(scale, q), out,
                                        _kv(state_layout))


def la_workspace_size(B: int, T: int, H: int, K: int, V: int, num_seqs: int, varlen: bool = False) -> int:
    """Scratch bytes of an ``la_fwd`` call on the current device (kda_la_workspace_size); 0 when it needs none."""
    return int(lib().kda_la_workspace_size(B, T, H, K, V, num_seqs, int(bool(varlen))))


def la_fwd(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, log_decay: torch.Tensor,
           scale: Optional[float] = None, initial_state: Optional[torch.Tensor] = None,
           output_final_state: bool = False, cu_seqlens: Optional[torch.Tensor] = None,
           workspace: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
           final_state: Optional[torch.Tensor] = None, state_layout: str = "vk",
           state_dtype: Optional[torch.dtype] = None) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """Linear attention with a decay per head over prompts, chunked.

    q, k: bf16 [B,T,Hk,K], Hk dividing the H heads of v; v: bf16 [B,T,H,V]; log_decay: fp32 [H], or
    [B,T,H] for a decay per token, <= 0 (or positive where no run of up to 128 tokens sums to more
    than 44). initial_state: [N,H,V,K] ("vk") or [N,H,K,V] ("kv"), fp32 or bf16, or None;
    cu_seqlens: int32 [N+1] of packed sequences (then B must be 1) or None. state_dtype: dtype of the
    final state when there is no initial_state (default fp32; with an initial_state, its dtype).
    Strides of q, k and v must be multiples of 8 elements and their bases 16-byte aligned. Returns
    (o bf16 [B,T,H,V], final_state or None). The call can be captured in a
    CUDA graph when a `workspace` tensor is passed.
    """
    if state_dtype not in (None, torch.float32, torch.bfloat16):
        raise TypeError("the state must be float32 or bfloat16")
    return (_native or _load()).la_fwd(q, k, v, log_decay, _scale(scale, q), initial_state, bool(output_final_state),
                                       cu_seqlens, workspace, out, final_state, _kv(state_layout),
                                       state_dtype is torch.bfloat16)


def norm_gate(x: torch.Tensor, gate: torch.Tensor, weight: Optional[torch.Tensor] = None, eps: float = 1e-6,
              activation: str = "sigmoid", out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """RMS norm over the last dimension, times weight and act(gate): the norm of the heads' outputs.

    x, gate: bf16 [..., D], contiguous or [rows,D], [rows,heads,D] or [B,T,heads,D] with strides;
    weight: fp32 [D] or None; activation: "sigmoid" or "silu". Returns bf16 [..., D]; `out` may be x.
    """
    if activation not in ("sigmoid", "silu"):
        raise ValueError("activation must be 'sigmoid' or 'silu'")
    return (_native or _load()).norm_gate(x, gate, weight, eps, activation == "silu", out)


def add_norm(x: torch.Tensor, residual: torch.Tensor, weight: Optional[torch.Tensor] = None,
             post_weight: Optional[torch.Tensor] = None, gate: Optional[torch.Tensor] = None,
             residual_scale=1.0, eps: float = 1e-6, out: Optional[torch.Tensor] = None,
             residual_out: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, torch.Tensor]:
    """The norms around a residual addition, with the block's gate and scale, in one pass.

    z = x; with post_weight, z = rms_norm(x) * post_weight; with gate, z = z * sigmoid(gate);
    h = residual + residual_scale * z; y = rms_norm(h) * weight. Returns (y, h).

    x, gate: bf16 [..., D]; residual: bf16 or fp32 [..., D] (h has its dtype); weight, post_weight: fp32
    [D] or None; residual_scale: a number, or fp32 [D]. x, residual and gate are contiguous, or
    [rows,D] with a row stride. out: y's buffer; residual_out: h's, which may be `residual` itself.
    """
    return (_native or _load()).add_norm(x, residual, weight, post_weight, gate, residual_scale, eps, out, residual_out)
