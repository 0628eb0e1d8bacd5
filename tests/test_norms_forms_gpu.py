"""norm_gate and add_norm in the forms that the row length chooses, against fp64.

The bounds are those of test_norms_gpu.py.
"""
from __future__ import annotations

import pytest
import torch

import chunked_gated_delta_02_gb300 as kda
from serving_testlib import randn
from test_norms_gpu import check_add, check_gate

pytestmark = pytest.mark.gpu

# Both ends and the middle of the row lengths of 384 threads with two chunks each, of 384 with four and of 448 with
# four, and the lengths next to them.
LENGTHS = [5120, 5128, 5640, 6144, 6152, 10240, 10248, 11272, 12288, 12296, 13320, 14336, 14344]


@pytest.mark.parametrize("D", LENGTHS)
@pytest.mark.parametrize("activation", ["sigmoid", "silu"])
def test_norm_gate_long_rows(D, activation):
    gen = torch.Generator().manual_seed(D)
    x, g, w = randn(gen, 7, D, scale=3.0), randn(gen, 7, D, scale=2.0), randn(gen, D, dtype=torch.float32)
    check_gate(x, g, w, activation, what=f"D={D}")
    check_gate(x, g, None, activation, what=f"D={D}, no weight")


@pytest.mark.parametrize("D", LENGTHS)
@pytest.mark.parametrize("rdt", [torch.bfloat16, torch.float32])
def test_add_norm_long_rows(D, rdt):
    gen = torch.Generator().manual_seed(D)
    x, r, g = randn(gen, 7, D), randn(gen, 7, D, dtype=torch.float32, scale=4.0).to(rdt), randn(gen, 7, D)
    w, post, vec = (randn(gen, D, dtype=torch.float32) for _ in range(3))
    check_add(x, r, w, post, g, vec, what=f"D={D}, everything")
    check_add(x, r, None, None, None, 1.0, what=f"D={D}, plain")


@pytest.mark.parametrize("rdt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("D", [512, 1000, 5640, 11272, 13320])
def test_add_norm_rows_past_the_prefetch(D, rdt):
    """More rows than lie between a row and the one that is prefetched for it, 15 MB later."""
    rows = int(15e6 / (2 * D)) + 50
    gen = torch.Generator().manual_seed(D)
    x, r = randn(gen, rows, D), randn(gen, rows, D, dtype=torch.float32).to(rdt)
    w = randn(gen, D, dtype=torch.float32)
    y, h = kda.add_norm(x, r, w, residual_scale=0.5)
    for part in (slice(0, 40), slice(rows - 90, rows)):
        one_y, one_h = check_add(x[part], r[part], w, None, None, 0.5, what=f"{rows} x {D}")
        assert torch.equal(y[part], one_y) and torch.equal(h[part], one_h)
