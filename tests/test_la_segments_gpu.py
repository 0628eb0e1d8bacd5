"""la_fwd on sequences that are cut into segments: states in place, and a workspace of the size asked for."""
from __future__ import annotations

import pytest
import torch

import chunked_gated_delta_02_gb300 as kda
from test_la_fwd_gpu import check, make

pytestmark = pytest.mark.gpu


def calls(d):
    """(call into given buffers, fresh ones for it): o, the start states' buffer and another for the final states."""
    st = d["initial_state"]
    B, T, H, V = d["v"].shape

    def call(o, init, final):
        return kda.la_fwd(d["q"], d["k"], d["v"], d["log_decay"], initial_state=init, output_final_state=True,
                          cu_seqlens=d["cu_seqlens"], state_layout=d["state_layout"], out=o, final_state=final)

    return call, lambda: (torch.full_like(d["v"], 7.0), st.clone(), torch.full_like(st, 7.0))


def is_cut(d):
    """Whether a call has room for two segment states of each sequence and head, or, packed, of one sequence."""
    B, T, H, V = d["v"].shape
    N, K, packed = d["initial_state"].shape[0], d["q"].shape[3], d["cu_seqlens"] is not None
    return kda.la_workspace_size(B, T, H, K, V, N, packed) >= 2 * (1 if packed else N) * H * K * V * 4


# rows, tokens, heads; the third has more (sequence, head, segment) items than SMs, which also share some of them
FIXED = [(1, 8000, 2), (2, 903, 8), (2, 3200, 30), (1, 20000, 5)]
PACKED = [([6000, 0, 1, 129, 640], 2), ([2500, 2500, 2500], 2), ([3000, 0, 2047, 1, 5130, 1400, 130, 1664, 2700, 1025], 24),
          ([9000] + [700, 20] * 12, 20)]


@pytest.mark.parametrize("shape", FIXED + PACKED)
@pytest.mark.parametrize("init,layout,K,V", [(torch.float32, "vk", 128, 128), (torch.float32, "kv", 64, 128),
                                             (torch.bfloat16, "vk", 128, 64), (torch.bfloat16, "kv", 128, 128)])
def test_final_state_in_place_of_the_initial_state(shape, init, layout, K, V):
    """The same bits as with a buffer of its own for the final state, which are right."""
    if len(shape) == 3:
        B, T, H = shape
        d = make(B, T, H, H, K, V, seed=T, init=init, layout=layout)
    else:
        lens, H = shape
        d = make(1, 0, H, H, K, V, seed=len(lens), lens=lens, init=init, layout=layout, token=True)
    assert is_cut(d)
    call, buffers = calls(d)
    if d["v"].shape[1] * H <= 16000:
        want = check(d, f"{shape}")
    else:
        want = call(*buffers())
    for _ in range(3):
        o, st, _ = buffers()
        got = call(o, st, st)
        assert got[1].data_ptr() == st.data_ptr()
        assert torch.equal(o, want[0]) and torch.equal(st, want[1])


@pytest.mark.parametrize("shape", [(2, 3200, 30), (2, 903, 8), ([3000, 0, 2047, 1, 5130, 1400, 130, 1664, 2700, 1025], 24)])
def test_final_state_in_place_while_some_multiprocessors_are_taken(shape):
    """Calls on another stream hold 28 multiprocessors at a time, so that some of the call's blocks start late: the
    first segments of sequences whose last ones are done, it may be."""
    if len(shape) == 3:
        B, T, H = shape
        d = make(B, T, H, H, 128, 128, seed=1)
    else:
        lens, H = shape
        d = make(1, 0, H, H, 128, 128, seed=1, lens=lens, token=True)
    assert is_cut(d)
    call, buffers = calls(d)
    want = call(*buffers())
    other = make(1, 1024, 28, 28, 128, 128, seed=2, init=None)
    assert kda.la_workspace_size(1, 1024, 28, 128, 128, 1) == 0   # 28 blocks, eight chunks each
    got = [buffers() for _ in range(40)]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for o, st, _ in got:
        with torch.cuda.stream(side):
            for _ in range(3):
                kda.la_fwd(other["q"], other["k"], other["v"], other["log_decay"])
        call(o, st, st)
    torch.cuda.synchronize()
    for o, st, _ in got:
        assert torch.equal(o, want[0]) and torch.equal(st, want[1])
    assert kda.device_status() == 0


LONG_AND_SHORT = [9000] + [0, 1, 40, 300] * 60 + [128 * 9 + 1, 5000] + [17] * 1100 + [4000]   # more than one tile of the schedule


@pytest.mark.parametrize("lens,H", PACKED + [(LONG_AND_SHORT, 4), ([1024], 16), ([1025], 64), ([5, 1020], 64)])
def test_a_workspace_of_exactly_the_size_asked_for(lens, H):
    """4 KB of guard bytes around it; the bits of a call that allocates its own, and of the next call in the same one."""
    d = make(1, 0, 1, H, 64, 128, seed=7, lens=lens, token=True)
    call, buffers = calls(d)
    want = check(d, "own workspace") if sum(lens) * H < 100000 else call(*buffers())
    size = kda.la_workspace_size(1, sum(lens), H, 64, 128, len(lens), True)
    buf = torch.full((size + 8192,), 0xA5, dtype=torch.uint8, device="cuda")
    for _ in range(2):
        o, init, final = buffers()
        kda.la_fwd(d["q"], d["k"], d["v"], d["log_decay"], initial_state=init, output_final_state=True,
                   cu_seqlens=d["cu_seqlens"], out=o, final_state=final, workspace=buf[4096:4096 + size])
        assert torch.equal(o, want[0]) and torch.equal(final, want[1])
        assert bool((buf[:4096] == 0xA5).all()) and bool((buf[-4096:] == 0xA5).all())
    assert kda.device_status() == 0
