"""Single-token steps over a pool of states (step: KDA, la_step: decay per head) against fp64."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import chunked_gated_delta_02_gb300 as kda
from chunked_gated_delta_02_gb300.workloads import custom, make_inputs
from kda_testlib import TOL_S_REL, to_dev
from oracle.serving_ref import f64, kda_step_ref, la_tokens
from serving_testlib import TOL_O_STEP, as_kv, close, in_layout, randn, state_tol

pytestmark = pytest.mark.gpu

BAD_STATE_INDEX = 4


def make(op, N, H, K, V, seed=0, Hk=None, dtype=torch.float32, layout="vk", rows=None, per_head=False, f32=False,
         fused=False):
    gen = torch.Generator().manual_seed(seed)
    Hk = Hk or H
    if fused:
        q, k, v = torch.split(randn(gen, N, 2 * Hk * K + H * V + 3), [Hk * K, Hk * K, H * V, 3], -1)[:3]
        q, k, v = q.unflatten(-1, (Hk, K)), k.unflatten(-1, (Hk, K)), v.unflatten(-1, (H, V))
    else:
        q, k, v = randn(gen, N, Hk, K), randn(gen, N, Hk, K), randn(gen, N, H, V)
    rows = rows or N + 3
    d = dict(q=q, k=k, v=v, layout=layout, op=op,
             state=in_layout(randn(gen, rows, H, K, V, dtype=torch.float32, scale=0.5), layout).to(dtype),
             idx=torch.randperm(rows, generator=gen)[:N].to(torch.int32).cuda())
    if op == "kda":
        d["g"] = randn(gen, N, H) if per_head else randn(gen, N, H, K)
        d["beta"] = randn(gen, N, H, dtype=torch.float32 if f32 else torch.bfloat16)
        d["A_log"] = randn(gen, H, dtype=torch.float32, scale=0.3)
        d["dt_bias"] = randn(gen, H, dtype=torch.float32) if per_head else randn(gen, H, K, dtype=torch.float32)
    else:
        d["decay"] = -(torch.rand(N, H, generator=gen) if f32 else torch.rand(H, generator=gen)).cuda()
    return d


def run(d, idx="given", lower_bound=-3.0, scale=None, out=None):
    idx = d["idx"] if isinstance(idx, str) else idx
    if d["op"] == "kda":
        return kda.step(d["q"], d["k"], d["v"], d["g"], d["beta"], d["A_log"], d["state"], dt_bias=d["dt_bias"],
                        lower_bound=lower_bound, scale=scale, state_indices=idx, state_layout=d["layout"], out=out)
    return kda.la_step(d["q"], d["k"], d["v"], d["decay"], d["state"], state_indices=idx, scale=scale,
                       state_layout=d["layout"], out=out)


def reference(d, idx, lower_bound=-3.0, scale=None):
    """(o, the pool after the call [rows,H,K,V]) for valid rows `idx`."""
    K, H = d["q"].shape[-1], d["v"].shape[1]
    scale = K ** -0.5 if scale is None else scale
    pool = f64(as_kv(d["state"], d["layout"])).copy()
    S = pool[idx]
    if d["op"] == "kda":
        o, S = kda_step_ref(d["q"], d["k"], d["v"], d["g"], d["beta"], d["A_log"], d["dt_bias"], lower_bound, scale, S)
    else:
        group = H // d["q"].shape[1]
        a = np.broadcast_to(f64(d["decay"]), (len(idx), H))
        o = la_tokens(np.repeat(f64(d["q"]), group, 1)[:, None], np.repeat(f64(d["k"]), group, 1)[:, None],
                      f64(d["v"])[:, None], a[:, None], S, scale)[:, 0]
    pool[idx] = S
    return o, pool


def check(d, what="", **kw):
    idx = d["idx"].cpu().numpy()
    ref_o, ref_pool = reference(d, idx, **kw)
    before = d["state"].clone()
    o = run(d, **kw)
    close(o, ref_o, TOL_O_STEP, f"{what} o")
    close(as_kv(d["state"], d["layout"]).float(), ref_pool, state_tol(d["state"].dtype), f"{what} pool")
    others = np.setdiff1d(np.arange(before.shape[0]), idx)
    assert torch.equal(d["state"][others], before[others]), f"{what}: a row that no request names changed"
    assert kda.device_status() == 0
    return o


@pytest.mark.parametrize("op", ["kda", "la"])
@pytest.mark.parametrize("K,V", [(64, 64), (64, 128), (128, 64), (128, 128)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("layout", ["vk", "kv"])
def test_head_dims_dtypes_layouts(op, K, V, dtype, layout):
    check(make(op, 5, 3, K, V, seed=K + V, dtype=dtype, layout=layout), f"{op} K{K} V{V} {dtype} {layout}")


@pytest.mark.parametrize("op", ["kda", "la"])
@pytest.mark.parametrize("N", [1, 2, 3, 17, 64, 301])
@pytest.mark.parametrize("H", [1, 5, 32])
def test_batch_sizes(op, N, H):
    if N * H > 3000:
        H = 4
    check(make(op, N, H, 128, 128, seed=N), f"{op} N{N} H{H}")


@pytest.mark.parametrize("layout", ["vk", "kv"])
def test_kda_gate_per_head_fp32_beta_and_strided_views(layout):
    check(make("kda", 7, 4, 128, 64, seed=1, per_head=True, f32=True, layout=layout, fused=True), "per head, fp32 beta")
    d = make("kda", 7, 4, 64, 128, seed=2, layout=layout, fused=True)
    gen = torch.Generator().manual_seed(8)
    d["g"] = randn(gen, 4, 7, 64).transpose(0, 1)
    d["beta"] = randn(gen, 7, 9)[:, 2:6]
    check(d, "strided gate and beta")
    d["dt_bias"] = None
    check(d, "no dt_bias")


@pytest.mark.parametrize("Hk,H", [(1, 4), (2, 6), (8, 8)])
@pytest.mark.parametrize("token", [False, True])
def test_la_shared_heads(Hk, H, token):
    check(make("la", 9, H, 64, 64, seed=H, Hk=Hk, f32=token, fused=token), f"Hk{Hk} H{H}")


@pytest.mark.parametrize("bound,scale", [(0.0, 1.0), (-5.0, -0.5), (-1e-3, 0.0)])
def test_kda_bounds_and_scales(bound, scale):
    check(make("kda", 3, 2, 128, 128, seed=4), f"bound {bound} scale {scale}", lower_bound=bound, scale=scale)


def test_kda_extreme_gates_and_zero_vectors():
    """Logits and gates where the sigmoids saturate, and q or k of zeros (their normalised forms are 0)."""
    d = make("kda", 4, 2, 64, 64, seed=6)
    d["beta"][0], d["beta"][1] = 60.0, -60.0
    d["g"][0], d["g"][1] = 200.0, -200.0
    d["k"][2] = 0
    d["q"][3] = 0
    check(d, "extremes")


@pytest.mark.parametrize("op", ["kda", "la"])
def test_la_decay_extremes_and_default_rows(op):
    d = make(op, 4, 2, 64, 64, seed=13, rows=4)
    if op == "la":
        d["decay"] = torch.tensor([0.0, float("-inf")]).cuda()
    d["idx"] = torch.arange(4, dtype=torch.int32, device="cuda")
    twin = {**d, "state": d["state"].clone()}
    o = check(d, "identity rows")
    assert torch.equal(run(twin, idx=None), o) and torch.equal(twin["state"], d["state"])


@pytest.mark.parametrize("op", ["kda", "la"])
@pytest.mark.parametrize("layout", ["vk", "kv"])
def test_padding_and_rows_outside_the_pool(op, layout):
    """Negative rows are padding; rows past the pool are reported. Both give o = 0 and touch nothing."""
    d = make(op, 6, 3, 128, 128, seed=15, layout=layout)
    good, bad_rows = [0, 2, 5], d["state"].shape[0]
    ref_o, ref_pool = reference({**d, **{n: d[n][good] for n in ("q", "k", "v") + (("g", "beta") if op == "kda" else ())}},
                                d["idx"].cpu().numpy()[good])
    idx = d["idx"].clone()
    idx[1], idx[3], idx[4] = -1, -2147483648, -7
    state = d["state"].clone()
    o = run(d, idx=idx)
    assert kda.device_status() == 0
    close(o[good], ref_o, TOL_O_STEP, "o beside padding")
    close(as_kv(d["state"], layout), ref_pool, state_tol(torch.float32), "pool beside padding")
    assert not o[[1, 3, 4]].any()
    d["state"] = state
    idx[3], idx[4] = bad_rows, 2147483647
    o2 = run(d, idx=idx)
    assert kda.device_status() == BAD_STATE_INDEX and kda.device_status() == 0
    assert torch.equal(o2, o)


@pytest.mark.parametrize("op", ["kda", "la"])
def test_rows_past_32_bit_offsets(op):
    """A pool of more than 2^32 values: the last row lies past 32-bit offsets."""
    H, K, V = 32, 128, 128
    rows = (1 << 32) // (H * K * V) + 3
    d = make(op, 2, H, K, V, seed=17, rows=4, dtype=torch.bfloat16)
    pool = torch.zeros(rows, H, V, K, dtype=torch.bfloat16, device="cuda")
    small = d["state"]
    pool[rows - 1], pool[rows - 2] = small[1], small[3]
    d["idx"] = torch.tensor([1, 3], dtype=torch.int32, device="cuda")
    ref_o, ref_pool = reference(d, [1, 3])
    d["state"] = pool
    o = run(d, idx=torch.tensor([rows - 1, rows - 2], dtype=torch.int32, device="cuda"))
    close(o, ref_o, TOL_O_STEP, "far rows o")
    close(pool[[rows - 1, rows - 2]].transpose(-1, -2).float(), ref_pool[[1, 3]], state_tol(torch.bfloat16), "far rows")
    assert not pool[:rows - 2].any()


@pytest.mark.parametrize("op", ["kda", "la"])
def test_graph_stream_and_buffers(op):
    d = make(op, 5, 4, 128, 128, seed=19)
    start = d["state"].clone()
    ref = run(d)
    after = d["state"].clone()
    out = torch.empty_like(ref)
    side = torch.cuda.Stream()
    d["state"].copy_(start)
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run(d, out=out)
    side.synchronize()
    assert torch.equal(out, ref) and torch.equal(d["state"], after)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run(d, out=out)
    d["state"].copy_(start)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, ref) and torch.equal(d["state"], after)


@pytest.mark.parametrize("op", ["kda", "la"])
def test_no_requests(op):
    d = make(op, 1, 2, 64, 64)
    state = d["state"].clone()
    d = {**d, **{n: d[n][:0] for n in ("q", "k", "v") + (("g", "beta") if op == "kda" else ())}}
    assert run(d, idx=d["idx"][:0]).shape == (0, 2, 64) and torch.equal(d["state"], state)


@pytest.mark.parametrize("per_head", [False, True])
def test_kda_step_continues_the_forward(per_head):
    """fwd over a prompt and a step per token after it, against fwd over all tokens."""
    T, more, H, K, V = 150, 5, 3, 128, 128
    inp = make_inputs(custom(B=2, T=T + more, H=H, K=K, V=V, lower_bound=-1.0), seed=23)
    if per_head:
        inp["g"] = inp["g"][..., 0].contiguous()
        inp["dt_bias"] = inp["dt_bias"][:, 0].contiguous()
    d = to_dev(inp)
    part = lambda t, a, b: t[:, a:b].contiguous()  # noqa: E731

    def fwd(a, b, state):
        return kda.fwd(*(part(d[n], a, b) for n in ("q", "k", "v", "g", "beta")), d["A_log"], d["dt_bias"],
                       d["lower_bound"], d["scale"], state, True)

    ref_o, ref_s = fwd(0, T + more, d["initial_state"])
    _, pool = fwd(0, T, d["initial_state"])
    for t in range(T, T + more):
        o = kda.step(d["q"][:, t], d["k"][:, t], d["v"][:, t], d["g"][:, t], d["beta"][:, t], d["A_log"], pool,
                     dt_bias=d["dt_bias"], lower_bound=d["lower_bound"], scale=d["scale"])
        close(o, f64(ref_o[:, t]), 2 * 5e-3, f"o of token {t}")
    close(pool, f64(ref_s), 2 * TOL_S_REL, "state after the steps")
