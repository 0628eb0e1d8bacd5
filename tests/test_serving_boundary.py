"""Refusals of the serving operators: by the C ABI before anything is launched, and by the Python
binding before the library is called. No GPU is needed."""
from __future__ import annotations

import ctypes
import os

import pytest
import torch

import chunked_gated_delta_02_gb300 as kda

FAKE = 0x10000   # a 256-byte aligned address that is never dereferenced
OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3


@pytest.fixture(scope="module")
def lib():
    from chunked_gated_delta_02_gb300 import build
    if not (os.path.exists(build.LIB) and os.path.exists(build.BINDING)):
        build.build()
    from chunked_gated_delta_02_gb300._lib import lib as load
    return load()


def i64(*x):
    return (ctypes.c_int64 * len(x))(*x)


def step(lib, **kw):
    a = dict(q=FAKE, k=FAKE, v=FAKE, g=FAKE, beta=FAKE, A=FAKE, dt=None, lb=-5.0, scale=1.0, state=FAKE, idx=FAKE, N=2,
             H=2, K=64, V=64, rows=4, st=None, flags=0, o=FAKE)
    a.update(kw)
    return lib.kda_step(a["q"], a["k"], a["v"], a["g"], a["beta"], a["A"], a["dt"], a["lb"], a["scale"], a["state"],
                        a["idx"], a["N"], a["H"], a["K"], a["V"], a["rows"], a["st"], a["flags"], a["o"], None)


def la_step(lib, **kw):
    a = dict(q=FAKE, k=FAKE, v=FAKE, d=FAKE, scale=1.0, state=FAKE, idx=FAKE, N=2, Hk=1, H=2, K=64, V=64, rows=4,
             st=None, flags=0, o=FAKE)
    a.update(kw)
    return lib.kda_la_step(a["q"], a["k"], a["v"], a["d"], a["scale"], a["state"], a["idx"], a["N"], a["Hk"], a["H"],
                           a["K"], a["V"], a["rows"], a["st"], a["flags"], a["o"], None)


def la_fwd(lib, **kw):
    a = dict(q=FAKE, k=FAKE, v=FAKE, d=FAKE, scale=1.0, init=None, final=None, cu=None, B=1, T=64, Hk=1, H=2, K=64, V=64,
             N=1, st=None, flags=0, o=FAKE, ws=FAKE, bytes=0)
    a.update(kw)
    return lib.kda_la_fwd(a["q"], a["k"], a["v"], a["d"], a["scale"], a["init"], a["final"], a["cu"], a["B"], a["T"],
                          a["Hk"], a["H"], a["K"], a["V"], a["N"], a["st"], a["flags"], a["o"], a["ws"], a["bytes"], None)


def norm_gate(lib, **kw):
    a = dict(x=FAKE, g=FAKE, w=None, eps=1e-6, outer=4, inner=1, D=64, st=None, flags=0, y=FAKE)
    a.update(kw)
    return lib.kda_norm_gate(a["x"], a["g"], a["w"], a["eps"], a["outer"], a["inner"], a["D"], a["st"], a["flags"],
                             a["y"], None)


def add_norm(lib, **kw):
    a = dict(x=FAKE, r=FAKE, g=None, post=None, w=None, vec=None, scale=1.0, eps=1e-6, rows=4, D=64, st=None, flags=0,
             y=FAKE, h=FAKE)
    a.update(kw)
    return lib.kda_add_norm(a["x"], a["r"], a["g"], a["post"], a["w"], a["vec"], a["scale"], a["eps"], a["rows"], a["D"],
                            a["st"], a["flags"], a["y"], a["h"], None)


NAN, INF = float("nan"), float("inf")


@pytest.mark.parametrize("kw,code", [
    *[({n: None}, INVALID) for n in ("q", "k", "v", "g", "beta", "A", "state", "o")],
    (dict(K=96), UNSUPPORTED), (dict(V=32), UNSUPPORTED), (dict(H=0), INVALID), (dict(N=-1), INVALID),
    (dict(rows=-1), INVALID), (dict(rows=1, idx=None), INVALID), (dict(flags=0x10), INVALID),
    (dict(flags=0x10000), INVALID), (dict(lb=0.5), INVALID), (dict(lb=-5.5), INVALID), (dict(lb=NAN), INVALID),
    (dict(scale=INF), INVALID), (dict(state=FAKE + 8), INVALID), (dict(q=FAKE + 1), INVALID), (dict(idx=FAKE + 2), INVALID),
    (dict(beta=FAKE + 2, flags=2), INVALID), (dict(dt=FAKE + 2), INVALID), (dict(N=1 << 30, H=64), UNSUPPORTED),
])
def test_step_refusals(lib, kw, code):
    assert step(lib, **kw) == code


@pytest.mark.parametrize("kw,code", [
    *[({n: None}, INVALID) for n in ("q", "k", "v", "d", "state", "o")],
    (dict(Hk=3, H=4), INVALID), (dict(Hk=0), INVALID), (dict(K=32), UNSUPPORTED), (dict(flags=1), INVALID),
    (dict(flags=2), INVALID), (dict(d=FAKE + 2), INVALID), (dict(scale=NAN), INVALID), (dict(rows=1, idx=None), INVALID),
])
def test_la_step_refusals(lib, kw, code):
    assert la_step(lib, **kw) == code


def strides(q=(128, 64, 64), k=(128, 64, 64), v=(256, 128, 64), d=(2, 2, 1)):
    return i64(*q, *k, *v, *d)


@pytest.mark.parametrize("kw,code", [
    *[({n: None}, INVALID) for n in ("q", "k", "v", "d", "o")],
    (dict(B=0), INVALID), (dict(T=-1), INVALID), (dict(Hk=3), INVALID), (dict(N=2), INVALID), (dict(K=96), UNSUPPORTED),
    (dict(V=256), UNSUPPORTED), (dict(cu=FAKE, B=2, N=2), INVALID), (dict(cu=FAKE + 2), INVALID), (dict(flags=1), INVALID),
    (dict(q=FAKE + 8), INVALID), (dict(v=FAKE + 2), INVALID), (dict(o=FAKE + 8), INVALID), (dict(init=FAKE + 8), INVALID),
    (dict(final=FAKE + 4), INVALID), (dict(scale=INF), INVALID),
    (dict(st=strides(q=(128, 60, 64))), INVALID), (dict(st=strides(k=(128, -64, 64))), INVALID),
    (dict(st=strides(v=(256, 128, 4))), INVALID), (dict(st=strides(q=(128, 0, 64))), INVALID),
    (dict(cu=FAKE, N=3, bytes=16), WORKSPACE), (dict(cu=FAKE, N=3, bytes=1 << 30, ws=FAKE + 16), WORKSPACE),
    (dict(B=1 << 30, N=1 << 30, H=64), UNSUPPORTED),
])
def test_la_fwd_refusals(lib, kw, code):
    assert la_fwd(lib, **kw) == code


@pytest.mark.parametrize("kw,code", [
    *[({n: None}, INVALID) for n in ("x", "g", "y")],
    (dict(D=0), INVALID), (dict(D=40000), UNSUPPORTED), (dict(outer=-1), INVALID), (dict(inner=0), INVALID),
    (dict(eps=-1.0), INVALID), (dict(eps=NAN), INVALID), (dict(flags=2), INVALID), (dict(w=FAKE + 2), INVALID),
    (dict(x=FAKE + 1), INVALID), (dict(outer=1 << 31), UNSUPPORTED),
])
def test_norm_gate_refusals(lib, kw, code):
    assert norm_gate(lib, **kw) == code


@pytest.mark.parametrize("kw,code", [
    *[({n: None}, INVALID) for n in ("x", "r", "y", "h")],
    (dict(D=0), INVALID), (dict(D=40000), UNSUPPORTED), (dict(rows=-1), INVALID), (dict(eps=INF), INVALID),
    (dict(scale=NAN), INVALID), (dict(flags=2), INVALID), (dict(r=FAKE + 2, flags=1), INVALID), (dict(post=FAKE + 1), INVALID),
    (dict(rows=1 << 31), UNSUPPORTED),
])
def test_add_norm_refusals(lib, kw, code):
    assert add_norm(lib, **kw) == code


@pytest.mark.parametrize("kw", [
    dict(B=1 << 30, N=1 << 30, H=64), dict(T=2147483647), dict(T=2147480001),
    dict(cu=FAKE, N=500_000_001, H=2), dict(cu=FAKE, N=1_000_000_001, H=1),
])
def test_la_fwd_refuses_more_than_it_counts_in_32_bits(lib, kw):
    assert la_fwd(lib, **kw) == UNSUPPORTED


def test_empty_calls_are_no_ops(lib):
    assert step(lib, N=0, q=None, k=None, v=None, beta=None, o=None) == OK
    assert la_step(lib, N=0, q=None, k=None, v=None, o=None) == OK
    assert la_fwd(lib, cu=FAKE, N=0, T=0) == OK
    assert norm_gate(lib, outer=0, x=None, g=None, y=None) == OK
    assert add_norm(lib, rows=0, x=None, r=None, y=None, h=None) == OK


def test_la_workspace(lib):
    """Nothing for equal lengths without segments; a schedule when packed; segment states of few long sequences."""
    assert kda.la_workspace_size(64, 512, 64, 128, 128, 64) == 0
    packed = kda.la_workspace_size(1, 512 * 64, 64, 128, 128, 64, True)
    assert 0 < packed and packed % 256 == 0
    one = kda.la_workspace_size(1, 65536, 2, 128, 128, 1)
    assert one >= 2 * 2 * 128 * 128 * 4
    assert kda.la_workspace_size(0, 512, 64, 128, 128, 64) == 0


META = dict(device="meta")


def bf(*shape):
    return torch.empty(*shape, dtype=torch.bfloat16, **META)


def f32(*shape, **kw):
    return torch.empty(*shape, **{**META, **kw})


def step_args(**over):
    a = dict(q=bf(2, 4, 64), k=bf(2, 4, 64), v=bf(2, 4, 128), g=bf(2, 4, 64), beta=bf(2, 4), A_log=f32(4),
             state=f32(3, 4, 128, 64))
    a.update(over)
    return a


@pytest.mark.parametrize("over,error,text", [
    (dict(q=bf(2, 4, 1, 64)), ValueError, "q must be a 3-D"), (dict(k=bf(2, 4, 128)), ValueError, "k must have shape"),
    (dict(v=f32(2, 4, 128)), TypeError, "v must be torch.bfloat16"), (dict(v=bf(3, 4, 128)), ValueError, "v must have shape"),
    (dict(g=bf(2, 5)), ValueError, "g must have shape"), (dict(g=None), TypeError, "g must be a torch.Tensor"),
    (dict(beta=f32(2, 4, dtype=torch.float16)), TypeError, "beta must be"), (dict(beta=bf(2, 5)), ValueError, "beta must have"),
    (dict(A_log=f32(3)), ValueError, "A_log must have shape"), (dict(dt_bias=f32(5)), ValueError, "dt_bias must hold 256"),
    (dict(g=bf(2, 4), dt_bias=f32(256)), ValueError, "dt_bias must hold 4"),
    (dict(state=f32(3, 4, 64, 128)), ValueError, "state must have shape"),
    (dict(state=f32(3, 4, 128, 64, dtype=torch.float16)), TypeError, "float32 or bfloat16"),
    (dict(state=f32(3, 4, 64, 128).transpose(2, 3)), ValueError, "state must be contiguous"),
    (dict(state=f32(1, 4, 128, 64)), ValueError, "state must hold 2 rows"),
    (dict(state=torch.empty(3, 4, 128, 64)), ValueError, "state must be on meta"),
    (dict(state_indices=f32(2)), TypeError, "state_indices must be torch.int32"),
    (dict(state_indices=f32(3, dtype=torch.int32)), ValueError, "state_indices must have shape"),
    (dict(q=bf(2, 64, 4).transpose(1, 2), k=bf(2, 64, 4).transpose(1, 2)), ValueError, "contiguous in its last dimension"),
    (dict(out=bf(2, 4, 64)), ValueError, "out must have shape"), (dict(state_layout="kk"), ValueError, "state_layout"),
    (dict(lower_bound="x"), TypeError, "must be real number"), (dict(), ValueError, "CUDA tensor"),
])
def test_step_binding_refuses(lib, over, error, text):
    with pytest.raises(error, match=text):
        kda.step(**step_args(**over))


def la_step_args(**over):
    a = dict(q=bf(2, 2, 64), k=bf(2, 2, 64), v=bf(2, 4, 128), log_decay=f32(4), state=f32(3, 4, 128, 64))
    a.update(over)
    return a


@pytest.mark.parametrize("over,error,text", [
    (dict(q=bf(2, 3, 64), k=bf(2, 3, 64)), ValueError, "must be a multiple"), (dict(k=bf(2, 1, 64)), ValueError, "k must have"),
    (dict(log_decay=f32(3)), ValueError, "log_decay must have"), (dict(log_decay=bf(4)), TypeError, "log_decay must be"),
    (dict(log_decay=f32(3, 4)), ValueError, "log_decay must have shape"), (dict(v=bf(2, 4)), ValueError, "v must be a 3-D"),
    (dict(state=f32(3, 4, 64, 64)), ValueError, "state must have shape"), (dict(), ValueError, "CUDA tensor"),
])
def test_la_step_binding_refuses(lib, over, error, text):
    with pytest.raises(error, match=text):
        kda.la_step(**la_step_args(**over))


def la_fwd_args(**over):
    a = dict(q=bf(1, 9, 2, 64), k=bf(1, 9, 2, 64), v=bf(1, 9, 4, 128), log_decay=f32(4))
    a.update(over)
    return a


@pytest.mark.parametrize("over,error,text", [
    (dict(q=bf(9, 2, 64)), ValueError, "q must be a 4-D"), (dict(k=bf(1, 8, 2, 64)), ValueError, "k must have shape"),
    (dict(v=bf(1, 9, 3, 128)), ValueError, "must be a multiple"), (dict(log_decay=f32(1, 9, 3)), ValueError, "log_decay"),
    (dict(initial_state=f32(1, 4, 64, 128)), ValueError, "initial_state must have shape"),
    (dict(initial_state=torch.empty(1, 4, 128, 64)), ValueError, "initial_state must be on"),
    (dict(output_final_state=True, final_state=bf(1, 4, 128, 64)), TypeError, "final_state must be torch.float32"),
    (dict(cu_seqlens=f32(2, dtype=torch.int64)), TypeError, "cu_seqlens must be"),
    (dict(cu_seqlens=f32(2, 2, dtype=torch.int32)), ValueError, "1-D tensor"),
    (dict(out=torch.empty(1, 9, 4, 128, dtype=torch.bfloat16)), ValueError, "out must be on"),
    (dict(workspace=torch.empty(100)), ValueError, "workspace must be on"),
    (dict(state_dtype=torch.float16), TypeError, "float32 or bfloat16"), (dict(state_layout=0), ValueError, "state_layout"),
    (dict(), ValueError, "CUDA tensor"),
])
def test_la_fwd_binding_refuses(lib, over, error, text):
    with pytest.raises(error, match=text):
        kda.la_fwd(**la_fwd_args(**over))


def test_la_fwd_binding_refuses_packed_batches(lib):
    with pytest.raises(ValueError, match="need B = 1"):
        kda.la_fwd(**la_fwd_args(q=bf(2, 9, 2, 64), k=bf(2, 9, 2, 64), v=bf(2, 9, 4, 128),
                                 cu_seqlens=f32(3, dtype=torch.int32)))


@pytest.mark.parametrize("args,kw,error,text", [
    ((3, bf(2, 8)), {}, ValueError, "x must be a torch.Tensor"), ((bf(2, 0), bf(2, 0)), {}, ValueError, "x must be"),
    ((bf(2, 8), bf(2, 9)), {}, ValueError, "gate must have shape"), ((bf(2, 8), f32(2, 8)), {}, TypeError, "gate must be"),
    ((bf(2, 8), bf(2, 8), f32(9)), {}, ValueError, "weight must have shape"),
    ((bf(2, 8), bf(2, 8), bf(8)), {}, TypeError, "weight must be torch.float32"),
    ((bf(2, 8), bf(2, 8)), dict(activation="relu"), ValueError, "activation"),
    ((bf(8, 2).t(), bf(2, 8)), {}, ValueError, "last dimension"),
    ((bf(2, 3, 4, 5, 8)[:, :, ::2], bf(2, 3, 2, 5, 8)), {}, ValueError, "x must be contiguous, or a strided"),
    ((bf(4, 3, 2, 8).transpose(0, 1), bf(3, 4, 2, 8)), {}, ValueError, "one dimension"),
    ((bf(2, 8), bf(2, 8)), dict(out=bf(8, 2).t()), ValueError, "out must be contiguous"),
    ((bf(2, 8), bf(2, 8)), {}, ValueError, "CUDA tensor"),
])
def test_norm_gate_binding_refuses(lib, args, kw, error, text):
    with pytest.raises(error, match=text):
        kda.norm_gate(*args, **kw)


@pytest.mark.parametrize("args,kw,error,text", [
    ((bf(2, 8), bf(2, 9)), {}, ValueError, "residual must have shape"),
    ((bf(2, 8), f32(2, 8, dtype=torch.float16)), {}, TypeError, "residual must be"),
    ((bf(2, 8), bf(2, 8), f32(7)), {}, ValueError, "weight must have shape"),
    ((bf(2, 8), bf(2, 8)), dict(post_weight=f32(2, 8)), ValueError, "post_weight must have"),
    ((bf(2, 8), bf(2, 8)), dict(gate=bf(2, 4)), ValueError, "gate must have"),
    ((bf(2, 8), bf(2, 8)), dict(residual_scale=f32(4)), ValueError, "residual_scale must have"),
    ((bf(2, 8), bf(2, 8)), dict(residual_scale="big"), TypeError, "must be real number"),
    ((bf(2, 8), f32(2, 8)), dict(residual_out=bf(2, 8)), TypeError, "residual_out must be torch.float32"),
    ((bf(2, 3, 16)[..., :8], bf(2, 3, 8)), {}, ValueError, "x must be contiguous, or"),
    ((bf(2, 8), bf(2, 8)), {}, ValueError, "CUDA tensor"),
])
def test_add_norm_binding_refuses(lib, args, kw, error, text):
    with pytest.raises(error, match=text):
        kda.add_norm(*args, **kw)
