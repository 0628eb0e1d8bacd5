"""The example's stack of layers: tokens decoded after prompts equal the longer prompts' outputs.

Bound: both ways round every block's output to bf16 (2^-8 relative at most) at the same places and
differ in the KDA forward's fp16 operands and the order of sums, a few bf16 roundings per layer; four
layers of at most two such roundings each, added up, stay below 8 * 2^-8 = 3.1e-2."""
from __future__ import annotations

import os
import sys

import pytest

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kw", [dict(), dict(lens=(5, 200), tokens=3, D=512, H=4, Hk=4, K=64, V=64),
                                dict(lens=(130,), tokens=2, D=256, H=2, Hk=1, K=64, V=128, layers=2)])
def test_decoding_continues_prompts(kw):
    from hybrid_layers import check
    worst = check(**kw)
    assert worst <= 8 * 2.0 ** -8, worst


def test_decoding_from_a_graph():
    from hybrid_layers import Model, decode_time
    assert decode_time(Model(D=256, H=2, Hk=1, layers=2), 4, steps=3) > 0
