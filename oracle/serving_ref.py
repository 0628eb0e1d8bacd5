"""fp64 definitions of the serving operators (numpy), token by token.

TEST INFRASTRUCTURE ONLY, like kda_ref: nothing in the product path imports it.

  la_ref       S_t = exp(a_t) S_{t-1} + k_t v_t^T,  o_t = scale S_t^T q_t           (S is K x V)
  kda_step_ref one token of the KDA recurrence (kda_ref's definition)
  norm_gate_ref, add_norm_ref
"""
from __future__ import annotations

import numpy as np
import torch

MIN_LOG_DECAY = -126.0 * np.log(2.0)   # smaller log decays count as this one (include/kda.h)


def f64(x):
    """A tensor or array as float64, exactly."""
    if isinstance(x, torch.Tensor):
        x = x.detach().cpu()
        return x.to(torch.float64).numpy() if x.is_floating_point() else x.numpy()
    return np.asarray(x, np.float64)


def sigmoid(x):
    x = f64(x)
    with np.errstate(over="ignore"):
        return 1.0 / (1.0 + np.exp(-x))


def la_tokens(q, k, v, a, S, scale):
    """Tokens of one batch of sequences of equal length. q, k [n,T,H,K], v [n,T,H,V], a [n,T,H],
    S [n,H,K,V] (changed in place). Returns o [n,T,H,V]."""
    o = np.empty(v.shape)
    decay = np.exp(a)
    for t in range(q.shape[1]):
        S *= decay[:, t, :, None, None]
        S += k[:, t, :, :, None] * v[:, t, :, None, :]
        o[:, t] = scale * np.matmul(q[:, t, :, None, :], S)[:, :, 0]
    return o


def la_ref(q, k, v, log_decay, scale, init=None, cu=None):
    """init: [N,H,K,V] or None. Returns (o [B,T,H,V], final [N,H,K,V])."""
    q, k, v, a = f64(q), f64(k), f64(v), f64(log_decay)
    B, T, Hk, K = q.shape
    H, V = v.shape[2:]
    q, k = np.repeat(q, H // Hk, 2), np.repeat(k, H // Hk, 2)
    a = np.broadcast_to(np.maximum(a, MIN_LOG_DECAY), (B, T, H))
    if cu is None:
        S = np.zeros((B, H, K, V)) if init is None else f64(init).copy()
        return la_tokens(q, k, v, a, S, scale), S
    cu = [int(x) for x in cu]
    S = np.zeros((len(cu) - 1, H, K, V)) if init is None else f64(init).copy()
    o = np.zeros((1, T, H, V))
    for s in range(len(cu) - 1):
        sl = slice(cu[s], cu[s + 1])
        o[:, sl] = la_tokens(q[:, sl], k[:, sl], v[:, sl], a[:, sl], S[s:s + 1], scale)
    return o, S


def kda_step_ref(q, k, v, g, beta, A_log, dt_bias, lower_bound, scale, S):
    """S [N,H,K,V] before the token. Returns (o [N,H,V], S after it)."""
    q, k, v, g, S = f64(q), f64(k), f64(v), f64(g), f64(S)
    g = g[..., None] if g.ndim == 2 else g
    dt = 0.0 if dt_bias is None else f64(dt_bias).reshape(q.shape[1], -1)
    alpha = np.exp(lower_bound * sigmoid(np.exp(f64(A_log))[:, None] * (g + dt)))
    qh = q / np.sqrt((q * q).sum(-1, keepdims=True) + 1e-6)
    kh = k / np.sqrt((k * k).sum(-1, keepdims=True) + 1e-6)
    S = S * np.broadcast_to(alpha, q.shape)[..., None]
    u = sigmoid(beta)[..., None] * (v - np.einsum("nhk,nhkv->nhv", kh, S))
    S = S + kh[..., None] * u[:, :, None, :]
    return scale * np.einsum("nhk,nhkv->nhv", qh, S), S


def rms(x, eps):
    return x / np.sqrt((x * x).mean(-1, keepdims=True) + eps)


def norm_gate_ref(x, gate, weight, eps, activation):
    g = f64(gate)
    act = sigmoid(g) * (g if activation == "silu" else 1.0)
    return rms(f64(x), eps) * (1.0 if weight is None else f64(weight)) * act


def add_norm_ref(x, residual, weight, post_weight, gate, scale, eps):
    z = f64(x)
    if post_weight is not None:
        z = rms(z, eps) * f64(post_weight)
    if gate is not None:
        z = z * sigmoid(gate)
    h = f64(residual) + (f64(scale) if isinstance(scale, torch.Tensor) else scale) * z
    return rms(h, eps) * (1.0 if weight is None else f64(weight)), h
