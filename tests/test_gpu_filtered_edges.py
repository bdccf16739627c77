"""Filtered sampling and masks at the ends of float32."""

import math

import numpy as np
import pytest
import torch

import speculative_decoding_tree_build_gb300 as tv

pytestmark = pytest.mark.gpu

BF16, F32, I32 = torch.bfloat16, torch.float32, torch.int32
INF = math.inf


def i32(x):
    return torch.tensor(x, dtype=I32, device="cuda")


def f32(x):
    return torch.tensor(x, dtype=F32, device="cuda")


def both(x, t, k, p, m, noise=None):
    """Row r of x is request r's only node: tokens, logp, masked rows and kept counts."""
    rows, v = x.shape
    ld = -(-v // 8) * 8
    lg = torch.zeros(rows, ld, dtype=x.dtype, device="cuda")[:, :v]
    lg.copy_(x)
    gumbel = torch.zeros(rows, ld, device="cuda")[:, :v]
    if noise is not None:
        gumbel.copy_(noise)
    opt = lambda a, make: None if a is None else make([a] * rows)
    args = (i32(list(range(rows + 1))), f32([t] * rows), opt(k, i32), opt(p, f32), opt(m, f32), 1)
    tok, lp, st = i32([-5] * rows), f32([9.0] * rows), i32([0] * rows)
    tv.sample_filtered(lg, gumbel, *args, tok, lp, st)
    out = torch.zeros(rows, ld, dtype=x.dtype, device="cuda")[:, :v]
    kept = i32([-5] * rows)
    tv.filter_logits(lg, *args, out, kept, st)
    assert not st.any()
    return tok.tolist(), lp.tolist(), out, kept.tolist()


# ----------------------------------------------------- logits that are masked and others that overflow


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("v", [10, 3000, 9000, 40001])
@pytest.mark.parametrize("k,p,m", [(None, None, None), (None, 0.5, None), (0, 0.75, 0.5), (7, 0.5, None), (None, None, 0.3)])
def test_masked_logits_beside_the_lowest_value(v, dtype, k, p, m):
    """The type's lowest value divided by 0.5 is -inf: these tokens weigh 1 each, logits
    of -inf are no tokens. logp = -ln of a whole number: two roundings."""
    rng = np.random.default_rng(v)
    counts = [1, 4, v // 2, v - 1]
    x = torch.full((len(counts), v), -INF, dtype=dtype)
    lowest = torch.finfo(dtype).min
    places = []
    for r, n in enumerate(counts):
        at = np.sort(rng.permutation(v)[:n])
        x[r, torch.from_numpy(at)] = lowest
        places.append(at)
    tok, lp, out, kept = both(x, 0.5, k, p, m)
    for r, n in enumerate(counts):
        left = n if not k else min(n, k)
        want = left if p is None else math.ceil(p * left)            # the first whose weights reach p of them
        assert kept[r] == want
        assert torch.equal((out[r] > -INF).nonzero().flatten().cpu(), torch.from_numpy(places[r][:want]))
        assert tok[r] == places[r][0]
        assert abs(lp[r] + math.log(want)) <= 2.0 ** -23 * math.log(want)
