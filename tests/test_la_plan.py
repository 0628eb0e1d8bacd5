"""la_fwd's plan of a call as its workspace shows it: no memory for segments that the call cannot have. No GPU is needed."""
from __future__ import annotations

import os

import pytest

import chunked_gated_delta_02_gb300 as kda

STATE = 128 * 128 * 4   # bytes of one fp32 state


@pytest.fixture(scope="module", autouse=True)
def built():
    from chunked_gated_delta_02_gb300 import build
    if not (os.path.exists(build.LIB) and os.path.exists(build.BINDING)):
        build.build()


@pytest.mark.parametrize("T,H,N", [(1024, 64, 1), (8192, 64, 512), (0, 8, 3), (1, 8, 1), (127, 64, 64)])
def test_packed_calls_without_a_second_segment_need_a_schedule_alone(T, H, N):
    """One sequence of all tokens fits one segment of these calls, so that nothing is formed ahead."""
    assert kda.la_workspace_size(1, T, H, 128, 128, N, True) < STATE + 64 * N


@pytest.mark.parametrize("T,H,N,blocks", [(70000, 64, 512, 2), (200000, 8, 4000, 16), (9000, 32, 2000, 0)])
def test_packed_calls_hold_no_states_of_sequences_in_one_segment(T, H, N, blocks):
    """However many sequences there are: `blocks` states per head are what the tokens can fill segments with, twice."""
    size = kda.la_workspace_size(1, T, H, 128, 128, N, True)
    assert size < blocks * H * (STATE + 4) + 64 * (N + 16)
    assert size >= blocks // 2 * H * STATE
