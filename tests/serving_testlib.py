"""Tolerances and inputs shared by the tests of the serving operators.

Tolerances, from the operators' roundings. Rounding to bf16 errs by up to 2^-8 relative, 1.66e-3 in RMS
over evenly spread mantissas; fp32 sums and the hardware's base-2 exponential and reciprocal stay
below 2^-21 per operation.
  * o of a single-token step: one rounding to bf16, 2e-3 rel-L2;
  * o of la_fwd: P (or the copy of S) and o are rounded to bf16, two independent errors, sqrt(2) 1.66e-3
    = 2.35e-3 rel-L2, taken as 3e-3;
  * fp32 states: products of 24-bit operands added in fp32 and decays of a few exponentials: 2e-6;
  * bf16 states: one rounding per call, 2e-3 rel-L2.
"""
from __future__ import annotations

import numpy as np
import torch

TOL_O_STEP = 2.0e-3
TOL_O_FWD = 3.0e-3
TOL_S32 = 2.0e-6
TOL_S16 = 2.0e-3


def rel_l2(x, y):
    x = x.detach().cpu().double().numpy() if isinstance(x, torch.Tensor) else np.asarray(x, np.float64)
    y = np.asarray(y, np.float64)
    assert x.shape == y.shape, (x.shape, y.shape)
    den = np.linalg.norm(y)
    num = np.linalg.norm(x - y)
    return float(num / den) if den > 0 else float(num)


def close(x, y, tol, what):
    assert bool(torch.isfinite(x).all()), f"{what}: not finite"
    e = rel_l2(x, y)
    assert e <= tol, f"{what}: rel-L2 {e:.3e} (<= {tol})"
    return e


def state_tol(dtype):
    return TOL_S16 if dtype == torch.bfloat16 else TOL_S32


def randn(gen, *shape, dtype=torch.bfloat16, scale=1.0):
    return (scale * torch.randn(*shape, generator=gen)).to(dtype).cuda()


def as_kv(state, layout):
    """A state [.., V, K] or [.., K, V] as [.., K, V]."""
    return state if layout == "kv" else state.transpose(-1, -2)


def in_layout(state_kv, layout):
    return (state_kv if layout == "kv" else state_kv.transpose(-1, -2)).contiguous()
