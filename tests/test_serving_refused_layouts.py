"""Refusals of layouts that a serving operator cannot read, by the Python binding and by the argument's name. No GPU is needed."""
from __future__ import annotations

import pytest
import torch

import chunked_gated_delta_02_gb300 as kda
from test_serving_boundary import bf, f32, la_fwd_args, la_step_args, lib, step_args  # noqa: F401


def off(t):
    """The same tensor, one element past a boundary."""
    return torch.empty(t.numel() + 1, dtype=t.dtype, device="meta")[1:].view(t.shape)


@pytest.mark.parametrize("name,shape", [("q", (1, 9, 2, 64)), ("k", (1, 9, 2, 64)), ("v", (1, 9, 4, 128))])
def test_la_fwd_names_tensors_it_cannot_read(lib, name, shape):  # noqa: F811
    B, T, H, D = shape
    for t in (bf(B, T, 1, D).expand(shape), bf(B, 1, H, D).expand(shape), bf(B, T, H, D + 4)[..., :D],
              bf(B, T, H * D + 2)[..., :H * D].unflatten(-1, (H, D))):
        with pytest.raises(ValueError, match=f"^{name} must have strides that are positive multiples of 8"):
            kda.la_fwd(**la_fwd_args(**{name: t}))
    with pytest.raises(ValueError, match=f"^{name} must begin on a 16-byte boundary"):
        kda.la_fwd(**la_fwd_args(**{name: off(bf(*shape))}))


def test_la_fwd_takes_any_stride_of_a_dimension_of_one(lib):  # noqa: F811
    q, k = bf(1, 2, 64)[:, None].expand(1, 1, 2, 64), bf(1, 1, 1, 64).expand(1, 1, 2, 64)
    with pytest.raises(ValueError, match="^k must have strides"):
        kda.la_fwd(**la_fwd_args(q=q, k=k, v=bf(1, 1, 4, 128)))
    with pytest.raises(ValueError, match="CUDA tensor"):
        kda.la_fwd(**la_fwd_args(q=q, k=torch.empty_strided((1, 1, 2, 64), (3, 5, 64, 1), dtype=torch.bfloat16, device="meta"),
                                 v=bf(1, 1, 4, 128)))


@pytest.mark.parametrize("name", ["initial_state", "final_state"])
def test_la_fwd_names_states_off_a_boundary(lib, name):  # noqa: F811
    with pytest.raises(ValueError, match=f"^{name} must begin on a 16-byte boundary"):
        kda.la_fwd(**la_fwd_args(**{name: off(f32(1, 4, 128, 64))}, output_final_state=True))


def test_la_fwd_names_an_output_off_a_boundary(lib):  # noqa: F811
    with pytest.raises(ValueError, match="^out must begin on a 16-byte boundary"):
        kda.la_fwd(**la_fwd_args(out=off(bf(1, 9, 4, 128))))


def test_steps_name_pools_off_a_boundary(lib):  # noqa: F811
    pool = off(f32(3, 4, 128, 64))
    with pytest.raises(ValueError, match="^state must begin on a 16-byte boundary"):
        kda.step(**step_args(state=pool))
    with pytest.raises(ValueError, match="^state must begin on a 16-byte boundary"):
        kda.la_step(**la_step_args(state=pool))
