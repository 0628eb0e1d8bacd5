"""norm_gate and add_norm in each form that the row length and the number of rows choose, against fp64.

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


def within(y, ref):
    """test_norms_gpu.within for a bf16 result, on the GPU, with terms of the size of the result."""
    assert bool(torch.isfinite(y).all())
    size = ref.abs()
    arith = 2.0 ** -20 * size
    _, exponent = torch.frexp((size + arith).clamp(min=2.0 ** -126))
    bound = torch.ldexp(torch.ones_like(size), exponent - 9) + arith
    worst = float(((y.double() - ref).abs() / bound).max())
    assert worst <= 1.0, f"{worst:.2f} of the bound"


@pytest.mark.parametrize("D,groups", [(40, 32), (64, 32), (104, 16), (128, 16), (200, 8), (256, 8)])
@pytest.mark.parametrize("past", [-1, 0, 1, "ragged"])
@pytest.mark.parametrize("weight,activation,views", [(True, "silu", True), (False, "sigmoid", False), (True, "sigmoid", True)])
def test_norm_gate_row_counts_around_the_four_row_form(D, groups, past, weight, activation, views):
    """Groups of threads take four rows each from 24 blocks of `groups` such groups per multiprocessor on. Every row is
    compared; x and the gate are views of one tensor, or contiguous."""
    heads = 3
    rows = torch.cuda.get_device_properties(0).multi_processor_count * 24 * groups * 4
    rows += 2 * groups + groups // 2 + 1 if past == "ragged" else past
    if views:
        rows = -(-rows // heads) * heads if past != -1 else (rows // heads) * heads
    gen = torch.Generator(device="cuda").manual_seed(rows)

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device="cuda")

    if views:
        x, gate = normal(rows // heads, 2, heads, D).bfloat16().unbind(1)
    else:
        x, gate = normal(rows, D).bfloat16(), normal(rows, D).bfloat16()
    w = normal(D) if weight else None
    y = kda.norm_gate(x, gate, w, activation=activation)
    assert y.shape == x.shape
    for part in torch.arange(x.shape[0], device="cuda").chunk(8):
        a, g = x[part].double(), gate[part].double()
        ref = a * torch.rsqrt(a.square().mean(-1, keepdim=True) + 1e-6) * torch.sigmoid(g)
        if activation == "silu":
            ref = ref * g
        within(y[part], ref if w is None else ref * w.double())
