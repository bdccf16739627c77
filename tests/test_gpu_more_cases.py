"""The measured cases of perf/more_operators.py: the library's calls, the plain form
and the definition in 64 bits on the same inputs, and a pass repeated."""

import random

import pytest
import torch

import perf.more_operators as cases

pytestmark = pytest.mark.gpu

# large ones stand in smaller for their kind
SMALLER = {"sample-large": {"batch": 3, "lo": 20, "hi": 33}, "filter-ragged": {"batch": 7, "lo": 2, "hi": 9},
           "sample-trees": {"batch": 12, "lo": 9, "hi": 9}, "slots-prompts": {"batch": 20}}


def compared():
    some = [dict(c, **SMALLER.get(c["name"], {})) for c in cases.listed()]
    rng = random.Random(17)
    while len(some) < 28:
        c = cases.draw(rng)
        if cases.work(c)["bytes"] < 6e7:
            some.append(dict(c, name=f"drawn {len(some)}"))
    return some


def outputs(case, own):
    cases.own = own
    try:
        state = cases.prepare(case, 4)
        first = {k: v.clone() for k, v in cases.run(state).items()}
        again = cases.run(state)
        torch.cuda.synchronize()
        for k in first:
            assert torch.equal(first[k].float().nan_to_num(), again[k].float().nan_to_num()), (k, "a second pass")
        return first
    finally:
        cases.own = False


@pytest.mark.parametrize("case", compared(), ids=lambda c: c["name"])
def test_case(case):
    plain, own, exact = outputs(case, False), outputs(case, True), cases.exact(case, 4)
    for name, got in own.items():
        got = got.cpu().double()
        for other in (plain[name], exact[name]):
            want = other.cpu().double().reshape(got.shape)
            if name == "logp":
                # ln of a share: float32's rounding of two terms of at most 120 and of their difference
                assert bool(((got - want).abs() <= 2.0 ** -20 + 2.0 ** -22 * want.abs()).all()), name
            else:
                assert torch.equal(got, want), name
