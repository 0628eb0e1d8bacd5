"""la_fwd with log decays of both signs in a chunk, against the fp64 definition.

Tolerances: o as a whole as elsewhere; for each token, whose rounded terms err independently, the same relative to
its own norm, twice in RMS for the tokens whose terms cancel. The fp32 state as elsewhere, and for running sums of
G (log2) the rounding of the exponents: 8 additions, each 2^-24 of |G|, times ln 2.
"""
from __future__ import annotations

import numpy as np
import pytest
import torch

import chunked_gated_delta_02_gb300 as kda
from oracle.serving_ref import f64, la_ref
from serving_testlib import TOL_O_FWD, TOL_S32, close, randn

pytestmark = pytest.mark.gpu

LN2 = float(np.log(2.0))


def check(log2_decay, K=128, V=128, init=True, lens=None, seed=1):
    """log2_decay [T, H], taken for two batch rows, or for the packed sequences of `lens`."""
    a = np.asarray(log2_decay, np.float64)
    T, H = a.shape
    B, N = (2, 2) if lens is None else (1, len(lens))
    gen = torch.Generator().manual_seed(seed)
    q, k, v = randn(gen, B, T, 1, K), randn(gen, B, T, 1, K), randn(gen, B, T, H, V)
    d = torch.tensor(a * LN2, dtype=torch.float32).expand(B, T, H).contiguous().cuda()
    cu = None if lens is None else torch.tensor([0] + lens).cumsum(0).to(torch.int32).cuda()
    st = randn(gen, N, H, V, K, dtype=torch.float32, scale=0.5) if init else None
    o, fs = kda.la_fwd(q, k, v, d, initial_state=st, output_final_state=True, cu_seqlens=cu)
    ref_o, ref_s = la_ref(q, k, v, d, K ** -0.5, None if st is None else st.transpose(-1, -2),
                          None if cu is None else cu.tolist())
    close(o, ref_o, TOL_O_FWD, "o")
    each = np.linalg.norm(f64(o) - ref_o, axis=-1) / np.linalg.norm(ref_o, axis=-1)
    rms = float(np.sqrt((each ** 2).mean()))
    assert rms <= 2 * TOL_O_FWD, f"each token's o: {rms:.3e} in RMS"
    chunks = [a[s + t:min(s + t + 128, e)] for s, e in zip(np.cumsum([0] + (lens or [T]))[:-1], np.cumsum(lens or [T]))
              for t in range(0, e - s, 128)]
    span = max(float(np.abs(c.cumsum(0)).max()) for c in chunks)
    close(fs.transpose(-1, -2), ref_s, TOL_S32 + 8 * 2.0 ** -24 * span * LN2, "state")
    assert kda.device_status() == 0


def fall_and_rise(T, down, up, steps_down, steps_up):
    """Runs of `steps_down` tokens that sum to -down, each followed by one of `steps_up` tokens that sums to up."""
    one = [-down / steps_down] * steps_down + [up / steps_up] * steps_up
    return np.resize(one, T)


CASES = {
    "fall by 160, rise by 60": fall_and_rise(128, 160, 60, 64, 64),
    "fall by 160, rise by 30": fall_and_rise(128, 160, 30, 64, 64),
    "fall by 100 at once, rise by 64": fall_and_rise(128, 100, 64, 1, 127),
    "fall by 1000 at once, rise by 40": fall_and_rise(300, 1000, 40, 9, 40),
    "rise by 64 first": np.r_[np.full(64, 1.0), np.full(64, -2.6)],
    "rise by 64 alone": np.full(128, 0.5),
    "ends above, dips below 2^-64": fall_and_rise(128, 70, 64, 8, 120),
    "rises of one token": fall_and_rise(500, 7, 5, 2, 1),
    "short": np.array([-80.0, 3.0, 3.0, 57.0, -1.0]),
}


@pytest.mark.parametrize("name", CASES)
@pytest.mark.parametrize("init", [False, True])
@pytest.mark.parametrize("K,V", [(64, 64), (128, 128)])
def test_falls_and_rises(name, init, K, V):
    a = CASES[name]
    check(np.stack([a, np.full_like(a, -0.05)], 1), K, V, init)


@pytest.mark.parametrize("lens", [None, [200, 1, 0, 129, 300]])
def test_random_signs(lens):
    """Runs of all kinds; no run of 128 tokens rises by more than 2^64."""
    rng = np.random.default_rng(3)
    T = 630
    a = rng.normal(size=(T, 4)) * np.array([0.3, 2.0, 4.0, 20.0]) - np.array([0.0, 1.0, 6.0, 40.0])
    for h in range(4):
        g = np.r_[0.0, a[:, h].cumsum()]
        assert max(float((g[n:] - g[:-n]).max()) for n in range(1, 129)) < 64
    check(a, lens=lens)


@pytest.mark.parametrize("a", [np.r_[np.full(64, -2.5), np.full(64, 1.9)],
                               np.r_[-60 / LN2, -60 / LN2, 80 / LN2, np.full(125, -0.01)]])
def test_growths_past_the_documented_ones_stay_finite(a):
    """By 2^121.6 and 2^115: still what the definition gives, on tokens of which none is zero."""
    check(a[:, None])


def test_nan_among_rising_decays_is_not_hidden():
    gen = torch.Generator().manual_seed(4)
    q, k, v = (randn(gen, 1, 128, 1, 64) for _ in range(3))
    d = torch.full((1, 128, 1), 0.1, device="cuda")
    for first in (0.1, -60.0):
        d[0, :3] = first
        d[0, 50] = float("nan")
        o, fs = kda.la_fwd(q, k, v, d, output_final_state=True)
        assert bool(torch.isnan(o[0, 50:]).all()) and bool(torch.isnan(fs).all())
        assert bool(torch.isfinite(o[0, :50]).all())
