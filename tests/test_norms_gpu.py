"""norm_gate and add_norm against fp64.

Bounds per element: one rounding of the result to its type, which is half the spacing of that type at
the result, and fp32 arithmetic of a few operations on terms no larger than those added (2^-20 of them).
"""
from __future__ import annotations

import numpy as np
import pytest
import torch

import chunked_gated_delta_02_gb300 as kda
from oracle.serving_ref import add_norm_ref, f64, norm_gate_ref, rms, sigmoid
from serving_testlib import randn

pytestmark = pytest.mark.gpu

FRACTION_BITS = {torch.bfloat16: 7, torch.float32: 23}


def half_spacing(x, dtype):
    """Half the distance between neighbouring numbers of a type at |x|."""
    return np.exp2(np.floor(np.log2(np.maximum(x, 2.0 ** -126))) - FRACTION_BITS[dtype] - 1)


def within(x, ref, terms, what):
    """|x - ref| <= rounding of ref to x's type + fp32 arithmetic on terms of size `terms`."""
    g = f64(x)
    assert np.isfinite(g).all(), f"{what}: not finite"
    arith = 2.0 ** -20 * terms
    bound = half_spacing(np.abs(ref) + arith, x.dtype) + arith
    worst = float((np.abs(g - ref) / bound).max()) if g.size else 0.0
    assert worst <= 1.0, f"{what}: {worst:.2f} of the bound"


def check_gate(x, gate, w, activation="sigmoid", eps=1e-6, what="", out=None):
    ref = norm_gate_ref(x, gate, w, eps, activation)
    y = kda.norm_gate(x, gate, w, eps=eps, activation=activation, out=out)
    assert y.shape == x.shape and y.is_contiguous()
    within(y, ref, np.abs(ref), what)
    return y


DIMS = [1, 2, 7, 8, 24, 64, 100, 128, 129, 136, 256, 264, 512, 520, 1000, 1023, 1024, 1032, 2048, 2056, 2880, 4096,
        4104, 8192, 8200, 16384, 16392, 20001, 32768]


@pytest.mark.parametrize("D", DIMS)
@pytest.mark.parametrize("activation", ["sigmoid", "silu"])
def test_norm_gate_row_lengths(D, activation):
    gen = torch.Generator().manual_seed(D)
    x, g = randn(gen, 5, D, scale=3.0), randn(gen, 5, D, scale=2.0)
    check_gate(x, g, randn(gen, D, dtype=torch.float32), activation, what=f"D={D}")


@pytest.mark.parametrize("rows", [0, 1, 2, 15, 16, 17, 63, 64, 65, 1000, 80000])
def test_norm_gate_row_counts(rows):
    """80000 rows of 128 take the four-row form of the kernel, with a ragged end."""
    gen = torch.Generator().manual_seed(rows)
    x, g = randn(gen, rows, 128), randn(gen, rows, 128)
    check_gate(x, g, None, what=f"{rows} rows")


@pytest.mark.parametrize("D", [64, 100, 128, 520])
def test_norm_gate_views(D):
    gen = torch.Generator().manual_seed(1)
    wide = randn(gen, 2, 6, 4 * D * 3)
    a, b, c = (t.unflatten(-1, (4, D)) for t in torch.split(wide, 4 * D, -1))
    plain = randn(gen, 2, 6, 4, D)
    w = randn(gen, D, dtype=torch.float32)
    check_gate(a, b, w, what="two views")
    check_gate(plain, c, w, what="contiguous x, view gate")
    check_gate(b, plain, w, what="view x, contiguous gate")
    check_gate(wide[0, :, :D], wide[1, :, D:2 * D], w, what="2-D views")
    check_gate(a[1], plain[0], w, what="3-D view")
    check_gate(plain.transpose(1, 2)[:1], plain[:1].transpose(1, 2), w, what="one batch row, heads first")
    assert torch.equal(check_gate(plain, plain, w, out=plain.clone()), kda.norm_gate(plain, plain, w))
    x = plain.clone()
    ref = kda.norm_gate(x, plain, w)
    assert torch.equal(kda.norm_gate(x, plain, w, out=x), ref)


def test_norm_gate_unaligned_bases_and_odd_strides():
    gen = torch.Generator().manual_seed(2)
    flat = randn(gen, 4000)
    x = flat[1:1 + 6 * 128].view(6, 128)
    g = flat[1001:1001 + 6 * 131].view(6, 131)[:, :128]
    w = randn(gen, 200, dtype=torch.float32)[3:131]
    check_gate(x, g, w, what="unaligned")
    check_gate(x, g, None, eps=0.0, what="no weight, no eps")


def test_norm_gate_zero_rows_and_extreme_gates():
    gen = torch.Generator().manual_seed(3)
    x, g = randn(gen, 8, 128), randn(gen, 8, 128)
    x[0] = 0
    g[1], g[2] = float("inf"), float("-inf")
    g[3], g[4] = 300.0, -300.0
    x[5] = 2.0 ** 60
    x[6] = 2.0 ** -60
    ref = norm_gate_ref(x, g, None, 1e-6, "sigmoid")
    y = kda.norm_gate(x, g)
    within(y, ref, np.abs(ref), "extremes")
    assert not y[0].any() and not y[2].any()


def check_add(x, r, w, post, g, scale, eps=1e-6, what="", **out):
    ref_y, ref_h = add_norm_ref(x, r, w, post, g, scale, eps)
    y, h = kda.add_norm(x, r, w, post_weight=post, gate=g, residual_scale=scale, eps=eps, **out)
    assert h.dtype == r.dtype and y.dtype == torch.bfloat16 and y.shape == h.shape == x.shape
    z = ref_h - f64(r)
    terms = np.abs(f64(r)) + np.abs(z)
    within(h, ref_h, terms, f"{what} h")
    factor = np.abs(ref_y) / np.where(ref_h == 0, 1.0, np.abs(ref_h))
    within(y, ref_y, np.abs(ref_y) + factor * terms, f"{what} y")
    return y, h


@pytest.mark.parametrize("D", DIMS)
@pytest.mark.parametrize("rdt", [torch.bfloat16, torch.float32])
def test_add_norm_row_lengths(D, rdt):
    gen = torch.Generator().manual_seed(D)
    x, r, g = randn(gen, 5, D), randn(gen, 5, D, dtype=torch.float32, scale=4.0).to(rdt), randn(gen, 5, D)
    w, post, vec = (randn(gen, D, dtype=torch.float32) for _ in range(3))
    check_add(x, r, w, post, g, vec, what=f"D={D}, everything")
    check_add(x, r, None, None, None, 1.0, what=f"D={D}, plain")


@pytest.mark.parametrize("post", [False, True])
@pytest.mark.parametrize("gate", [False, True])
@pytest.mark.parametrize("scale", [1.0, -0.25, 0, "vector"])
def test_add_norm_parts(post, gate, scale):
    gen = torch.Generator().manual_seed(4)
    D = 256
    vec = randn(gen, D, dtype=torch.float32)
    check_add(randn(gen, 3, 7, D), randn(gen, 3, 7, D), randn(gen, D, dtype=torch.float32),
              randn(gen, D, dtype=torch.float32) if post else None, randn(gen, 3, 7, D) if gate else None,
              vec if scale == "vector" else scale, what=f"post {post} gate {gate} scale {scale}")


@pytest.mark.parametrize("rows", [0, 1, 9, 33, 3000])
@pytest.mark.parametrize("D", [64, 4096])
def test_add_norm_row_counts(rows, D):
    gen = torch.Generator().manual_seed(rows)
    check_add(randn(gen, rows, D), randn(gen, rows, D), randn(gen, D, dtype=torch.float32), None, None, 0.5,
              what=f"{rows} x {D}")


@pytest.mark.parametrize("D", [128, 1000, 1001])
def test_add_norm_strides_and_in_place(D):
    gen = torch.Generator().manual_seed(6)
    wide = randn(gen, 6, 3 * D + 8)
    w = randn(gen, D, dtype=torch.float32)
    check_add(wide[:, :D], wide[:, D:2 * D], w, w, wide[:, 2 * D:3 * D], 1.0, what="row strides")
    x = randn(gen, 6, D)
    for rdt in (torch.bfloat16, torch.float32):
        r = randn(gen, 6, D, dtype=torch.float32).to(rdt)
        y, h = check_add(x, r, w, None, None, 2.0, what="fresh")
        y2, h2 = kda.add_norm(x, r, w, residual_scale=2.0, residual_out=r)
        assert h2.data_ptr() == r.data_ptr() and torch.equal(r, h) and torch.equal(y2, y)
    x2 = x.clone()
    y3, _ = kda.add_norm(x2, wide[:, :D], w, residual_scale=2.0, out=x2)
    assert y3.data_ptr() == x2.data_ptr()
    assert torch.equal(x2, kda.add_norm(x, wide[:, :D], w, residual_scale=2.0)[0])


def test_norms_on_another_stream_and_in_a_graph():
    gen = torch.Generator().manual_seed(7)
    x, r, g = randn(gen, 40, 512), randn(gen, 40, 512), randn(gen, 40, 512)
    ref = (*kda.add_norm(x, r, gate=g), kda.norm_gate(x, g))
    out = [torch.empty_like(t) for t in ref]

    def call():
        kda.add_norm(x, r, gate=g, out=out[0], residual_out=out[1])
        kda.norm_gate(x, g, out=out[2])

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(out, ref))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for t in out:
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(out, ref))


def test_many_rows_past_32_bit_offsets():
    """Rows whose elements lie past 2^31: the last ones are checked."""
    rows, D = (1 << 31) // 128 + 100, 128
    x = torch.ones(rows, D, dtype=torch.bfloat16, device="cuda")
    gen = torch.Generator().manual_seed(8)
    x[-50:] = randn(gen, 50, D)
    y = kda.norm_gate(x, x)
    tail = f64(x[-50:])
    within(y[-50:], rms(tail, 1e-6) * sigmoid(tail), np.abs(tail), "last rows")
