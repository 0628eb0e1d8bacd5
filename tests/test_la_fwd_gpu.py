"""la_fwd (linear attention with a decay per head, chunked) against its fp64 definition."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import chunked_gated_delta_02_gb300 as kda
from oracle.serving_ref import f64, la_ref
from serving_testlib import TOL_O_FWD, as_kv, close, in_layout, randn, state_tol

pytestmark = pytest.mark.gpu

BAD_CU_SEQLENS = 1


def head_decay(H):
    return -torch.exp2(-8.0 * torch.arange(1, H + 1) / H)


def make(B, T, Hk, H, K, V, seed=0, token=False, init=torch.float32, layout="vk", lens=None, fused=False, decay=None):
    gen = torch.Generator().manual_seed(seed)
    N = B
    cu = None
    if lens is not None:
        B, T, N = 1, sum(lens), len(lens)
        cu = torch.tensor([0] + list(lens)).cumsum(0).to(torch.int32).cuda()
    if fused:
        x = randn(gen, B, T, 2 * Hk * K + H * V)
        q, k, v = torch.split(x, [Hk * K, Hk * K, H * V], -1)
        q, k, v = q.unflatten(-1, (Hk, K)), k.unflatten(-1, (Hk, K)), v.unflatten(-1, (H, V))
    else:
        q, k, v = randn(gen, B, T, Hk, K), randn(gen, B, T, Hk, K), randn(gen, B, T, H, V)
    if decay is None:
        decay = torch.nn.functional.logsigmoid(1.5 * torch.randn(B, T, H, generator=gen) + 3) if token else head_decay(H)
    st = None if init is None else in_layout(randn(gen, N, H, K, V, dtype=torch.float32, scale=0.5), layout).to(init)
    return dict(q=q, k=k, v=v, log_decay=decay.float().cuda(), initial_state=st, cu_seqlens=cu, state_layout=layout)


def check(d, what="", scale=None, state_dtype=None, **kw):
    o, fs = kda.la_fwd(d["q"], d["k"], d["v"], d["log_decay"], scale=scale, initial_state=d["initial_state"],
                       output_final_state=True, cu_seqlens=d["cu_seqlens"], state_layout=d["state_layout"],
                       state_dtype=state_dtype, **kw)
    init = None if d["initial_state"] is None else as_kv(d["initial_state"], d["state_layout"])
    K = d["q"].shape[-1]
    ref_o, ref_s = la_ref(d["q"], d["k"], d["v"], d["log_decay"], K ** -0.5 if scale is None else scale, init,
                          None if d["cu_seqlens"] is None else d["cu_seqlens"].tolist())
    close(o, ref_o, TOL_O_FWD, f"{what} o")
    close(as_kv(fs, d["state_layout"]).float(), ref_s, state_tol(fs.dtype), f"{what} state")
    assert kda.device_status() == 0
    return o, fs


@pytest.mark.parametrize("T", [1, 2, 31, 32, 63, 64, 65, 127, 128, 129, 255, 256, 257, 384, 700])
@pytest.mark.parametrize("token", [False, True])
def test_lengths(T, token):
    check(make(2, T, 3, 3, 128, 128, seed=T, token=token), f"T={T}")


@pytest.mark.parametrize("K,V", [(64, 64), (64, 128), (128, 64), (128, 128)])
@pytest.mark.parametrize("layout", ["vk", "kv"])
@pytest.mark.parametrize("init", [None, torch.float32, torch.bfloat16])
def test_head_dims_states_and_layouts(K, V, layout, init):
    check(make(2, 300, 2, 2, K, V, seed=K + V, init=init, layout=layout, token=True), f"K{K} V{V} {layout}",
          state_dtype=torch.bfloat16 if init is None and K == 64 else None)


@pytest.mark.parametrize("Hk,H", [(1, 1), (1, 5), (2, 8), (3, 3), (4, 8), (1, 64)])
@pytest.mark.parametrize("fused", [False, True])
def test_shared_heads_and_fused_projections(Hk, H, fused):
    check(make(2, 200, Hk, H, 64, 128, seed=H, fused=fused, token=H == 8), f"Hk{Hk} H{H} fused={fused}")


def test_strides_of_every_dimension():
    """Heads before tokens, a slice of a wider head dimension, a strided token decay."""
    gen = torch.Generator().manual_seed(3)
    d = make(2, 150, 2, 4, 64, 64, token=True)
    d["q"] = randn(gen, 2, 2, 150, 64).transpose(1, 2)
    d["k"] = randn(gen, 2, 150, 2, 192)[..., 64:128]
    d["v"] = randn(gen, 150, 2, 4, 64).transpose(0, 1)
    d["log_decay"] = (-0.1 * torch.rand(2, 4, 150, generator=gen)).cuda().transpose(1, 2)
    check(d, "strides")


LENS = [[5], [0, 1, 63, 64, 65, 127, 128, 129, 0, 300], [1] * 40, [700, 0, 0, 3], [128, 256, 128], [0, 0, 7]]


@pytest.mark.parametrize("lens", LENS)
@pytest.mark.parametrize("token", [False, True])
def test_packed_sequences(lens, token):
    check(make(1, 0, 2, 4, 128, 64, seed=len(lens), lens=lens, token=token, fused=token), f"lens {lens[:6]}")


def test_many_packed_sequences():
    """More sequences than the schedule's threads, so its scan runs over several tiles."""
    rng = np.random.default_rng(0)
    check(make(1, 0, 1, 1, 64, 64, lens=[int(x) for x in rng.integers(0, 5, 2500)]), "2500 sequences")


@pytest.mark.parametrize("lens", [None, [6000, 0, 1, 129, 640], [2500, 2500, 2500]])
@pytest.mark.parametrize("init", [None, torch.bfloat16])
def test_segments_of_long_sequences(lens, init):
    """Few long sequences run as segments (a workspace for their states shows it)."""
    T = 8000 if lens is None else sum(lens)
    d = make(1, T, 1, 2, 128, 128, seed=9, lens=lens, init=init, layout="kv" if init else "vk", token=lens is not None)
    n = 1 if lens is None else len(lens)
    assert kda.la_workspace_size(1, T, 2, 128, 128, n, lens is not None) > 2 * 2 * 128 * 128 * 4
    check(d, f"segments {lens}")


@pytest.mark.parametrize("K,V", [(64, 64), (64, 128), (128, 64), (128, 128)])
@pytest.mark.parametrize("lens,H,packed", [
    ([1250] * 5, 40, False), ([1250] * 51, 3, False), ([1250] * 5, 40, True), ([600] * 40 + [3000, 512], 5, True),
    ([900, 0, 2047, 1, 513, 1400, 130, 1664, 700, 1025], 24, True),
    ([3000, 0, 2047, 1, 5130, 1400, 130, 1664, 2700, 1025], 24, True), ([9000] + [700, 20] * 12, 20, True),
])
def test_more_sequences_than_blocks(lens, H, packed, K, V):
    """More sequences and heads than SMs, and not a multiple: to even out the blocks' shares, a block goes on
    with the state of another."""
    if packed:
        d = make(1, 0, H, H, K, V, seed=H + K, lens=lens, token=True)
    else:
        d = make(len(lens), lens[0], H, H, K, V, seed=H + K, init=None)
    first = check(d, f"{len(lens)} x {H}")
    for _ in range(3):
        again = kda.la_fwd(d["q"], d["k"], d["v"], d["log_decay"], initial_state=d["initial_state"],
                           output_final_state=True, cu_seqlens=d["cu_seqlens"])
        assert all(torch.equal(x, y) for x, y in zip(first, again))


@pytest.mark.parametrize("decay", [0.0, -1e-4, -0.7, -5.0, -60.0, float("-inf")])
@pytest.mark.parametrize("T", [200, 4500])
def test_constant_decays(decay, T):
    """From no decay at all to a state that lasts one token; 4500 tokens run as segments."""
    check(make(1, T, 2, 2, 64, 64, seed=7, decay=torch.full((2,), decay)), f"decay {decay}")


def test_decays_of_all_sizes_in_one_chunk():
    """Weak, strong and total decays mixed over the tokens, which takes both forms of the decay mask."""
    gen = torch.Generator().manual_seed(11)
    T, H = 640, 3
    a = -torch.exp(4 * torch.randn(1, T, H, generator=gen) - 4)
    a[0, [0, 64, 127, 128, 300], 0] = float("-inf")
    a[0, 200:230, 1] = float("-inf")
    a[0, :128, 2] = -1e-3                       # a weak chunk between strong ones
    a[0, 128:256, 2] = -30.0
    check(make(1, T, 3, 3, 128, 128, seed=12, decay=a), "mixed decays")


def test_slow_decay_keeps_the_state_accurate():
    """An almost undamped state of 6000 tokens: the sums of many chunks and segments stay fp32-accurate."""
    check(make(1, 6000, 1, 1, 128, 128, seed=4, decay=torch.full((1,), -1e-5)), "slow decay")


def test_other_sequences_never_reach_a_sequence():
    """Infinities and NaN in the neighbours of a packed sequence, and in nothing of its own."""
    lens = [70, 130, 0, 90]
    d = make(1, 0, 2, 2, 128, 128, seed=5, lens=lens, token=True)
    clean = check(d, "clean")
    for name, bad in (("q", float("nan")), ("k", float("inf")), ("v", float("nan")), ("log_decay", float("nan"))):
        d[name] = d[name].clone()
        d[name][0, :70] = bad
        d[name][0, 200:] = bad
    o, fs = kda.la_fwd(d["q"], d["k"], d["v"], d["log_decay"], initial_state=d["initial_state"], output_final_state=True,
                       cu_seqlens=d["cu_seqlens"])
    assert torch.equal(o[:, 70:200], clean[0][:, 70:200])
    assert torch.equal(fs[1:3], clean[1][1:3])
    assert kda.device_status() == 0


def test_nan_decay_is_not_hidden():
    d = make(1, 100, 1, 1, 64, 64, token=True)
    d["log_decay"][0, 50] = float("nan")
    o, fs = kda.la_fwd(d["q"], d["k"], d["v"], d["log_decay"], output_final_state=True)
    assert bool(torch.isnan(o[0, 50:]).all()) and bool(torch.isnan(fs).all())
    assert bool(torch.isfinite(o[0, :50]).all())


def test_empty_calls():
    d = make(2, 0, 2, 2, 64, 64)
    o, fs = kda.la_fwd(d["q"], d["k"], d["v"], d["log_decay"], initial_state=d["initial_state"], output_final_state=True)
    assert o.shape == (2, 0, 2, 64) and torch.equal(fs, d["initial_state"])
    o, fs = kda.la_fwd(d["q"], d["k"], d["v"], d["log_decay"], output_final_state=True)
    assert not fs.any()
    cu = torch.zeros(1, dtype=torch.int32, device="cuda")
    o, fs = kda.la_fwd(d["q"][:1], d["k"][:1], d["v"][:1], d["log_decay"], output_final_state=True, cu_seqlens=cu)
    assert fs.shape == (0, 2, 64, 64)


def test_in_place_state_given_buffers_and_no_final_state():
    d = make(2, 333, 2, 4, 128, 128, seed=21)
    o, fs = check(d, "fresh buffers")
    st, out = d["initial_state"].clone(), torch.full_like(o, 7.0)
    o2, fs2 = kda.la_fwd(d["q"], d["k"], d["v"], d["log_decay"], initial_state=st, output_final_state=True, out=out,
                         final_state=st)
    assert o2.data_ptr() == out.data_ptr() and fs2.data_ptr() == st.data_ptr()
    assert torch.equal(out, o) and torch.equal(st, fs)
    o3, none = kda.la_fwd(d["q"], d["k"], d["v"], d["log_decay"], initial_state=d["initial_state"])
    assert none is None and torch.equal(o3, o)
    o4, _ = kda.la_fwd(d["q"], d["k"], d["v"], d["log_decay"], initial_state=d["initial_state"], scale=-0.25)
    ref = (-0.25 * 128 ** 0.5) * o.double()
    assert float((o4.double() - ref).norm() / ref.norm()) < 2 ** -8


@pytest.mark.parametrize("lens", [None, [900, 0, 77, 1300]])
def test_graph_stream_and_repeatability(lens):
    """Captured, replayed and run on another stream, the call gives the bits of the first."""
    d = make(1, 5000, 2, 2, 128, 128, seed=31, lens=lens, token=True)
    B, T, H, V = d["v"].shape
    N = 1 if lens is None else len(lens)
    ws = torch.empty(max(1, kda.la_workspace_size(B, T, H, 128, V, N, lens is not None)), dtype=torch.uint8, device="cuda")
    o = torch.empty(B, T, H, V, dtype=torch.bfloat16, device="cuda")
    fs = torch.empty_like(d["initial_state"])

    def call():
        kda.la_fwd(d["q"], d["k"], d["v"], d["log_decay"], initial_state=d["initial_state"], output_final_state=True,
                   cu_seqlens=d["cu_seqlens"], workspace=ws, out=o, final_state=fs)

    call()
    torch.cuda.synchronize()
    ref = o.clone(), fs.clone()
    side = torch.cuda.Stream()
    for buf in (o, fs, ws):
        buf.zero_()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    side.synchronize()
    assert torch.equal(o, ref[0]) and torch.equal(fs, ref[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for _ in range(2):
        o.zero_()
        fs.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, ref[0]) and torch.equal(fs, ref[1])
    assert kda.device_status() == 0


@pytest.mark.parametrize("lens", [None, [100, 130, 3]])
def test_nothing_outside_the_buffers_is_written(lens):
    """4 KB of guard bytes around o, the final state and a workspace of exactly the size asked for."""
    d = make(1, 4400, 1, 2, 64, 128, seed=41, lens=lens)
    B, T, H, V = d["v"].shape
    N = 1 if lens is None else len(lens)

    def guarded(nbytes):
        buf = torch.full((nbytes + 8192,), 0xA5, dtype=torch.uint8, device="cuda")
        return buf, buf[4096:4096 + nbytes]

    bufs, views = zip(*[guarded(n) for n in (B * T * H * V * 2, N * H * V * 64 * 4,
                                             max(256, kda.la_workspace_size(B, T, H, 64, V, N, lens is not None)))])
    o, fs = views[0].view(torch.bfloat16).view(B, T, H, V), views[1].view(torch.float32).view(N, H, V, 64)
    kda.la_fwd(d["q"], d["k"], d["v"], d["log_decay"], initial_state=d["initial_state"], output_final_state=True,
               cu_seqlens=d["cu_seqlens"], out=o, final_state=fs, workspace=views[2])
    torch.cuda.synchronize()
    for b in bufs:
        assert bool((b[:4096] == 0xA5).all()) and bool((b[-4096:] == 0xA5).all())
    ref_o, ref_s = la_ref(d["q"], d["k"], d["v"], d["log_decay"], 64 ** -0.5, as_kv(d["initial_state"], "vk"),
                          None if lens is None else d["cu_seqlens"].tolist())
    close(o, ref_o, TOL_O_FWD, "guarded o")


@pytest.mark.parametrize("cu", [[1, 5, 100], [0, 60, 50, 100], [0, 50, 99], [0, 101]])
def test_bad_cu_seqlens_is_reported_and_nothing_is_written(cu):
    d = make(1, 100, 1, 1, 64, 64)
    o = torch.full((1, 100, 1, 64), 3.0, dtype=torch.bfloat16, device="cuda")
    fs = torch.full((len(cu) - 1, 1, 64, 64), 3.0, device="cuda")
    kda.la_fwd(d["q"], d["k"], d["v"], d["log_decay"], output_final_state=True, out=o, final_state=fs,
               cu_seqlens=torch.tensor(cu, dtype=torch.int32, device="cuda"))
    assert kda.device_status() == BAD_CU_SEQLENS
    assert bool((o == 3).all()) and bool((fs == 3).all())
    check(d, "after the error")


def test_same_as_single_tokens():
    """A prompt, then the same prompt's tokens one at a time, give the same states."""
    d = make(2, 140, 2, 4, 128, 64, seed=51, token=True)
    o, fs = check(d, "prompt")
    pool = d["initial_state"].clone()
    steps = [kda.la_step(d["q"][:, t], d["k"][:, t], d["v"][:, t], d["log_decay"][:, t], pool) for t in range(140)]
    close(pool, f64(fs), 4e-6, "states")
    close(torch.stack(steps, 1), f64(o), 2 * TOL_O_FWD, "outputs")
