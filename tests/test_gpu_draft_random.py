"""The draft-model calls on drawn sizes, and beam selection on further inputs of
fixed sizes, against the plain forms of perf/operators.py: listed ids and values,
choices and moved bytes exactly, losses, normalisers and scores against the 64-bit
definitions there.  SPECVERIFY_RANDOM_DRAFT_CASES sets the number of cases,
SPECVERIFY_RANDOM_OFFSET other seeds."""
import math
import os
import random
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                                "perf"))
import operators  # noqa: E402

CASES = int(os.environ.get("SPECVERIFY_RANDOM_DRAFT_CASES", "24"))
OFFSET = int(os.environ.get("SPECVERIFY_RANDOM_OFFSET", "0"))
H = 2.0 ** -24


def sum_error(V):
    """Float sums of a row: exponents off by three half steps of |d| (log2(e), its
    division by T, the fused product), |d| at most log2 V + 1 in the mean; exp2 by
    one step, five additions within a chunk by half a step each."""
    return (math.log(2) * 3 * (math.log2(max(V, 2)) + 1) + 7) * H


def both(case, seed):
    state = operators.prepare(case, seed)
    outs = []
    for own in (False, True):
        operators.own = own
        try:
            out = operators.run(state)
        finally:
            operators.own = False
        outs.append([t.clone() for t in (out if isinstance(out, (list, tuple)) else [out])])
    return outs


def compare(case, seed):
    print(case, seed, flush=True)
    plain, got = both(case, seed)
    want = operators.exact(case, seed)
    op = case["op"]
    if op == "reorder":
        assert all(torch.equal(a, b) for a, b in zip(plain, got))
        return
    e = sum_error(case["vocab"])
    if op == "topk":
        assert torch.equal(plain[0], got[0]) and torch.equal(plain[1], got[1])
        assert ((got[2] - want[2]).abs() <= e + want[2].abs() * H).all()
    elif op == "beam":
        assert all(torch.equal(a, b) for a, b in zip(plain[1:], got[1:]))
        there = torch.isfinite(want[0])
        off = (got[0] - want[0])[there].abs()
        assert (off <= e + want[0][there].abs() * H).all()
    else:
        # two logarithms of sums for a mass of one; the listed masses add up to at most
        # 1 + 2^-18 where the teacher's float32 normaliser (below 2^6) rounds them up
        loss = want if op == "loss" else want[0]
        assert ((got[0] - loss).abs() <= 2.001 * e + loss.abs() * H).all()
        assert op == "loss" or torch.isfinite(got[1].float()).all()


@pytest.mark.parametrize("first", range(0, CASES, 8))
def test_drawn_cases(first):
    for seed in range(OFFSET + first, OFFSET + min(first + 8, CASES)):
        compare(operators.draw(random.Random(1000003 * seed + 1)), seed)


@pytest.mark.parametrize("name", ["beam_b1_w4_v32000_f32", "beam_b64_w4_v128256_bf16",
                                  "beam_b128_w8_v152064_bf16"])
def test_beam_choices_on_further_inputs(name):
    (case,) = [c for c in operators.listed() if c["name"] == name]
    for seed in range(max(CASES // 8, 1)):
        compare(case, 5000 + OFFSET + seed)
