"""Python binding of the serving operators (argument marshalling only).

``step`` continues a KDA forward by one token per request on states kept in a pool; ``la_fwd``
and ``la_step`` are linear attention with one decay per head, over prompts and by single tokens
(the fixed-decay linear attention of the cuLA README mirror, section "Quick Start", and its form
with a decay per token); ``norm_gate`` and ``add_norm`` are the norms of a layer around them. All
compute runs in libkda.so on the caller's current CUDA stream (include/kda.h has the formulas).

Unlike ``fwd``, these take token tensors with strides, as long as the last dimension is
contiguous: q, k and v may be views of one projection.
"""
from __future__ import annotations

import ctypes
from typing import Optional, Tuple

import torch

from ._lib import check, lib
from .kda import BETA_F32, GATE_PER_HEAD, STATE_BF16, STATE_KV

__all__ = ["step", "la_fwd", "la_step", "la_workspace_size", "norm_gate", "add_norm"]

LA_TOKEN_DECAY = 0x10000
NORM_SILU = 0x1
NORM_RESIDUAL_F32 = 0x1

_Strides4, _Strides10, _Strides12 = ctypes.c_int64 * 4, ctypes.c_int64 * 10, ctypes.c_int64 * 12


def _tensor(t, name, dtype, shape, device, contiguous=False):
    """Type, device, dtype, shape and layout of one tensor argument (shape None: not checked)."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.device != device:
        raise ValueError(f"{name} must be on {device}, got {t.device}")
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if contiguous:
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
    elif t.shape[-1] > 1 and t.stride(-1) != 1:
        raise ValueError(f"{name} must be contiguous in its last dimension")


def _need_dims(t, name, dims, text):
    if not isinstance(t, torch.Tensor) or t.dim() != dims:
        raise ValueError(f"{name} must be a {dims}-D torch.Tensor {text}")


def _on_gpu(t, name):
    if t.device.type != "cuda":
        raise ValueError(f"{name} must be a CUDA tensor (there is no CPU path)")


def _call(name, device, *args):
    """One library call on the current stream of `device`; the stream is the last argument."""
    fn = getattr(lib(), name)
    if device.index == torch.cuda.current_device():
        rc = fn(*args, torch.cuda.current_stream(device).cuda_stream)
    else:
        with torch.cuda.device(device):
            rc = fn(*args, torch.cuda.current_stream(device).cuda_stream)
    if rc:
        check(name, rc)


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def _state_flags(layout, dtype):
    if layout not in ("vk", "kv"):
        raise ValueError("state_layout must be 'vk' (rows [V,K]) or 'kv' (rows [K,V])")
    if dtype not in (torch.float32, torch.bfloat16):
        raise TypeError("the state must be float32 or bfloat16")
    return (STATE_KV if layout == "kv" else 0) | (STATE_BF16 if dtype is torch.bfloat16 else 0)


def _pool(state, state_indices, layout, N, H, K, V, device):
    """Checks of a pool of states; returns (rows, flags)."""
    _need_dims(state, "state", 4, "[rows,H,V,K] or [rows,H,K,V]")
    flags = _state_flags(layout, state.dtype)
    rows = state.shape[0]
    _tensor(state, "state", state.dtype, (rows, H, V, K) if layout == "vk" else (rows, H, K, V), device, True)
    if state_indices is not None:
        _tensor(state_indices, "state_indices", torch.int32, (N,), device, True)
    elif rows < N:
        raise ValueError(f"state must hold {N} rows, or state_indices say which it uses; got {rows}")
    return rows, flags


def _out(out, shape, device):
    if out is None:
        return torch.empty(shape, dtype=torch.bfloat16, device=device)
    _tensor(out, "out", torch.bfloat16, shape, device, True)
    return out


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
    _need_dims(q, "q", 3, "[N,H,K]")
    _need_dims(v, "v", 3, "[N,H,V]")
    N, H, K = q.shape
    V, dev, bf16 = v.shape[2], q.device, torch.bfloat16
    _tensor(q, "q", bf16, None, dev)
    _tensor(k, "k", bf16, (N, H, K), dev)
    _tensor(v, "v", bf16, (N, H, V), dev)
    rows, flags = _pool(state, state_indices, state_layout, N, H, K, V, dev)
    if isinstance(g, torch.Tensor) and g.dim() == 2:
        flags |= GATE_PER_HEAD
        _tensor(g, "g", bf16, (N, H), dev, True)
        gs = (H, 1)
    else:
        _tensor(g, "g", bf16, (N, H, K), dev)
        gs = g.stride()
    if isinstance(beta, torch.Tensor) and beta.dtype is torch.float32:
        flags |= BETA_F32
        _tensor(beta, "beta", torch.float32, (N, H), dev)
    else:
        _tensor(beta, "beta", bf16, (N, H), dev)
    _tensor(A_log, "A_log", torch.float32, (H,), dev)
    if dt_bias is not None:
        _tensor(dt_bias, "dt_bias", torch.float32, None, dev, True)
        if dt_bias.numel() != (H if flags & GATE_PER_HEAD else H * K):
            raise ValueError(f"dt_bias must hold {H if flags & GATE_PER_HEAD else H * K} values")
    o = _out(out, (N, H, V), dev)
    _on_gpu(q, "q")
    qs, ks, vs, bs = q.stride(), k.stride(), v.stride(), beta.stride()
    strides = _Strides10(qs[0], qs[1], ks[0], ks[1], vs[0], vs[1], gs[0], gs[1], bs[0], bs[1])
    _call("kda_step", dev, q.data_ptr(), k.data_ptr(), v.data_ptr(), g.data_ptr(), beta.data_ptr(),
          A_log.data_ptr(), _ptr(dt_bias), lower_bound, K ** -0.5 if scale is None else scale, state.data_ptr(),
          _ptr(state_indices), N, H, K, V, rows, strides, flags, o.data_ptr())
    return o


def _decay(log_decay, H, lead, device):
    """(flags, strides) of a log decay: [H], or [*lead, H]."""
    if isinstance(log_decay, torch.Tensor) and log_decay.dim() == 1:
        _tensor(log_decay, "log_decay", torch.float32, (H,), device)
        return 0, (0,) * (len(lead) + 1)
    _tensor(log_decay, "log_decay", torch.float32, (*lead, H), device)
    return LA_TOKEN_DECAY, log_decay.stride()


def _heads(q, k, v, tokens):
    """Checks the token tensors of linear attention; returns (Hk, H, K, V)."""
    dims = len(tokens) + 2
    Hk, K = q.shape[-2:]
    H, V = v.shape[-2:]
    dev = q.device
    _tensor(q, "q", torch.bfloat16, None, dev)
    _tensor(k, "k", torch.bfloat16, (*tokens, Hk, K), dev)
    _tensor(v, "v", torch.bfloat16, (*tokens, H, V), dev)
    if Hk < 1 or H % Hk:
        raise ValueError(f"the {H} heads of v must be a multiple of the {Hk} heads of q and k")
    return Hk, H, K, V


def la_step(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, log_decay: torch.Tensor, state: torch.Tensor,
            state_indices: Optional[torch.Tensor] = None, scale: Optional[float] = None,
            out: Optional[torch.Tensor] = None, state_layout: str = "vk") -> torch.Tensor:
    """One token of linear attention with a decay per head for each of N requests.

    q, k: bf16 [N,Hk,K], Hk dividing the H heads of v (value head h reads head h // (H / Hk));
    v: bf16 [N,H,V]; log_decay: fp32 [H], or [N,H] for a decay per token; state, state_indices,
    out and state_layout as in ``step``. Returns o, bf16 [N,H,V]; ``state`` is updated in place.
    """
    _need_dims(q, "q", 3, "[N,Hk,K]")
    _need_dims(v, "v", 3, "[N,H,V]")
    N, dev = q.shape[0], q.device
    Hk, H, K, V = _heads(q, k, v, (N,))
    rows, flags = _pool(state, state_indices, state_layout, N, H, K, V, dev)
    token, gs = _decay(log_decay, H, (N,), dev)
    o = _out(out, (N, H, V), dev)
    _on_gpu(q, "q")
    qs, ks, vs = q.stride(), k.stride(), v.stride()
    strides = _Strides10(qs[0], qs[1], ks[0], ks[1], vs[0], vs[1], gs[0], gs[1], 0, 0)
    _call("kda_la_step", dev, q.data_ptr(), k.data_ptr(), v.data_ptr(), log_decay.data_ptr(),
          K ** -0.5 if scale is None else scale, state.data_ptr(), _ptr(state_indices), N, Hk, H, K, V, rows, strides,
          flags | token, o.data_ptr())
    return o


def la_workspace_size(B: int, T: int, H: int, K: int, V: int, num_seqs: int, varlen: bool = False) -> int:
    """Scratch bytes of an ``la_fwd`` call (kda_la_workspace_size); 0 when it needs none."""
    return int(lib().kda_la_workspace_size(B, T, H, K, V, num_seqs, int(bool(varlen))))


def la_fwd(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, log_decay: torch.Tensor,
           scale: Optional[float] = None, initial_state: Optional[torch.Tensor] = None,
           output_final_state: bool = False, cu_seqlens: Optional[torch.Tensor] = None,
           workspace: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
           final_state: Optional[torch.Tensor] = None, state_layout: str = "vk",
           state_dtype: Optional[torch.dtype] = None) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """Linear attention with a decay per head over prompts, chunked.

    q, k: bf16 [B,T,Hk,K], Hk dividing the H heads of v; v: bf16 [B,T,H,V]; log_decay: fp32 [H], or
    [B,T,H] for a decay per token, <= 0. initial_state: [N,H,V,K] ("vk") or [N,H,K,V] ("kv"), fp32
    or bf16, or None; cu_seqlens: int32 [N+1] of packed sequences (then B must be 1) or None.
    state_dtype: dtype of the final state when there is no initial_state (default fp32; with an
    initial_state, its dtype). Strides of q, k and v must be multiples of 8 elements and their bases
    16-byte aligned. Returns (o bf16 [B,T,H,V], final_state or None). The call can be captured in a
    CUDA graph when a `workspace` tensor is passed.
    """
    _need_dims(q, "q", 4, "[B,T,Hk,K]")
    _need_dims(v, "v", 4, "[B,T,H,V]")
    B, T = q.shape[:2]
    dev = q.device
    Hk, H, K, V = _heads(q, k, v, (B, T))
    sdt = initial_state.dtype if initial_state is not None else (state_dtype or torch.float32)
    flags = _state_flags(state_layout, sdt)
    token, ds = _decay(log_decay, H, (B, T), dev)
    N = B
    if cu_seqlens is not None:
        _tensor(cu_seqlens, "cu_seqlens", torch.int32, None, dev, True)
        if cu_seqlens.dim() != 1 or cu_seqlens.numel() < 1:
            raise ValueError("cu_seqlens must be a 1-D tensor of N + 1 offsets")
        if B != 1:
            raise ValueError("packed sequences (cu_seqlens) need B = 1")
        N = cu_seqlens.numel() - 1
    sshape = (N, H, V, K) if state_layout == "vk" else (N, H, K, V)
    if initial_state is not None:
        _tensor(initial_state, "initial_state", sdt, sshape, dev, True)
    fs = None
    if output_final_state:
        if final_state is not None:
            _tensor(final_state, "final_state", sdt, sshape, dev, True)
            fs = final_state
        else:
            fs = torch.empty(sshape, dtype=sdt, device=dev)
    o = _out(out, (B, T, H, V), dev)
    _on_gpu(q, "q")
    need = la_workspace_size(B, T, H, K, V, N, cu_seqlens is not None)
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=dev) if need else None
    else:
        _tensor(workspace, "workspace", workspace.dtype, None, dev, True)
        if workspace.numel() * workspace.element_size() < need:
            raise ValueError(f"workspace too small: need {need} bytes")
    qs, ks, vs = q.stride(), k.stride(), v.stride()
    strides = _Strides12(*qs[:3], *ks[:3], *vs[:3], *ds)
    _call("kda_la_fwd", dev, q.data_ptr(), k.data_ptr(), v.data_ptr(), log_decay.data_ptr(),
          K ** -0.5 if scale is None else scale, _ptr(initial_state), _ptr(fs), _ptr(cu_seqlens), B, T, Hk, H, K, V, N,
          strides, flags | token, o.data_ptr(), _ptr(workspace),
          0 if workspace is None else workspace.numel() * workspace.element_size())
    return o, fs


def _rows(t, name):
    """(outer rows, inner rows, outer stride, inner stride) of a tensor [..., D] as rows of D values."""
    if t.is_contiguous():
        D = t.shape[-1]
        return t.numel() // D if D else 0, 1, D, D
    if t.dim() == 2:
        return t.shape[0], 1, t.stride(0), t.stride(0)
    if t.dim() == 3:
        return t.shape[0], t.shape[1], t.stride(0), t.stride(1)
    if t.dim() == 4 and (t.shape[0] == 1 or t.shape[1] == 1 or t.stride(0) == t.shape[1] * t.stride(1)):
        return t.shape[0] * t.shape[1], t.shape[2], t.stride(0 if t.shape[1] == 1 else 1), t.stride(2)
    raise ValueError(f"{name} must be contiguous, or a strided tensor [rows,D], [rows,heads,D] or [B,T,heads,D] "
                     "whose B and T are one dimension")


_ACTIVATIONS = {"sigmoid": 0, "silu": NORM_SILU}


def norm_gate(x: torch.Tensor, gate: torch.Tensor, weight: Optional[torch.Tensor] = None, eps: float = 1e-6,
              activation: str = "sigmoid", out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """RMS norm over the last dimension, times weight and act(gate): the norm of the heads' outputs.

    x, gate: bf16 [..., D], contiguous or [rows,D], [rows,heads,D] or [B,T,heads,D] with strides;
    weight: fp32 [D] or None; activation: "sigmoid" or "silu". Returns bf16 [..., D]; `out` may be x.
    """
    if not isinstance(x, torch.Tensor) or x.dim() < 1 or x.shape[-1] < 1:
        raise ValueError("x must be a torch.Tensor [..., D]")
    dev, D = x.device, x.shape[-1]
    _tensor(x, "x", torch.bfloat16, None, dev)
    _tensor(gate, "gate", torch.bfloat16, x.shape, dev)
    if weight is not None:
        _tensor(weight, "weight", torch.float32, (D,), dev)
    if activation not in _ACTIVATIONS:
        raise ValueError("activation must be 'sigmoid' or 'silu'")
    xo, xi, xs0, xs1 = _rows(x, "x")
    go, gi, gs0, gs1 = _rows(gate, "gate")
    if xi != gi:   # one of them contiguous, with its rows not split yet: the other's split
        if xi == 1:
            xo, xi, xs0, xs1 = go, gi, gi * xs1, xs1
        else:
            gs0, gs1 = xi * gs1, gs1
    y = _out(out, x.shape, dev)
    _on_gpu(x, "x")
    _call("kda_norm_gate", dev, x.data_ptr(), gate.data_ptr(), _ptr(weight), eps, xo, max(xi, 1), D,
          _Strides4(xs0, xs1, gs0, gs1), _ACTIVATIONS[activation], y.data_ptr())
    return y


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
    if not isinstance(x, torch.Tensor) or x.dim() < 1 or x.shape[-1] < 1:
        raise ValueError("x must be a torch.Tensor [..., D]")
    dev, D = x.device, x.shape[-1]
    _tensor(x, "x", torch.bfloat16, None, dev)
    rdt = residual.dtype if isinstance(residual, torch.Tensor) and residual.dtype is torch.float32 else torch.bfloat16
    _tensor(residual, "residual", rdt, x.shape, dev)
    strides = []
    for t, name in ((x, "x"), (residual, "residual"), (gate, "gate")):
        if t is None:
            strides.append(0)
            continue
        if t is gate:
            _tensor(gate, "gate", torch.bfloat16, x.shape, dev)
        if not t.is_contiguous() and t.dim() != 2:
            raise ValueError(f"{name} must be contiguous, or [rows,D] with a row stride")
        strides.append(D if t.is_contiguous() else t.stride(0))
    for t, name in ((weight, "weight"), (post_weight, "post_weight")):
        if t is not None:
            _tensor(t, name, torch.float32, (D,), dev)
    number, vec = 1.0, None
    if isinstance(residual_scale, torch.Tensor):
        vec = residual_scale
        _tensor(vec, "residual_scale", torch.float32, (D,), dev)
    else:
        number = float(residual_scale)
    y = _out(out, x.shape, dev)
    if residual_out is None:
        h = torch.empty(x.shape, dtype=rdt, device=dev)
    else:
        _tensor(residual_out, "residual_out", rdt, x.shape, dev, True)
        h = residual_out
    _on_gpu(x, "x")
    _call("kda_add_norm", dev, x.data_ptr(), residual.data_ptr(), _ptr(gate), _ptr(post_weight), _ptr(weight),
          _ptr(vec), number, eps, x.numel() // D, D, _Strides4(*strides, 0),
          NORM_RESIDUAL_F32 if rdt is torch.float32 else 0, y.data_ptr(), h.data_ptr())
    return y, h
