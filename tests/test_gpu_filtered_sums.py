"""Log-probabilities beside one heavy token, and calls on both sides of the rules that
choose a form of the kernel."""

import math

import numpy as np
import pytest
import torch

import speculative_decoding_tree_build_gb300 as tv
from oracle import draw_ref, filter_ref

pytestmark = pytest.mark.gpu

F32, I32 = torch.float32, torch.int32


def i32(x):
    return torch.tensor(x, dtype=I32, device="cuda")


def f32(x):
    return torch.tensor(x, dtype=F32, device="cuda")


@pytest.mark.parametrize("rows", [1, 40, 700])
def test_unfiltered_logp_beside_a_heavy_token(rows):
    """One token of weight 1, all others exp(-12): 51.6 units in the last place of 1, so
    a thread that adds hundreds of them to 1 one by one loses a part of a unit each time.
    Bound: a light weight's exponent, 17.3 with two roundings (2^-25 and 2^-24), and its
    2^-22: 1.3e-6 of a share of 0.48; the total's logarithm of 0.66 and its subtraction,
    1.2e-7 together: below 2^-20."""
    v = 151936
    x = torch.full((rows, v), -12.0, device="cuda")
    at = (torch.arange(rows, device="cuda") * 977 + 3) % v
    x[torch.arange(rows, device="cuda"), at] = 0.0
    noise = torch.zeros_like(x)
    tok, lp, st = torch.zeros(rows, dtype=I32, device="cuda"), torch.zeros(rows, device="cuda"), i32([0])
    per = min(rows, 1000)
    tv.sample_filtered(x, noise, i32([0, rows]), f32([1.0]), None, None, None, per, tok, lp, st)
    assert st.tolist() == [0] and torch.equal(tok, at.to(I32))
    want = -math.log(1.0 + (v - 1) * math.exp(-12.0))
    assert float((lp.double() - want).abs().max()) <= 2.0 ** -20


# (vocabulary, rows): rows below and above what is resident at once, vocabularies below
# and above 2^16
@pytest.mark.parametrize("dtype", [torch.bfloat16, F32])
@pytest.mark.parametrize("v,rows", [(5000, 620), (65536, 620), (65544, 620), (65536, 600), (65544, 9)])
@pytest.mark.parametrize("k", [None, 40])
def test_forms_of_the_kernel(dtype, v, rows, k):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(v + rows)
    x = (torch.randn(rows, v, generator=gen, device="cuda") * 2).to(dtype)
    noise = -torch.log(-torch.log(torch.rand(rows, v, generator=gen, device="cuda").clamp(1e-7, 1 - 1e-7)))
    half = rows // 2
    cu, t, p = i32([0, half, rows]), f32([0.9, 1.2]), f32([0.9, 0.6])
    kk = None if k is None else i32([k, 0])
    tok, lp, st = torch.zeros(rows, dtype=I32, device="cuda"), torch.zeros(rows, device="cuda"), i32([0, 0])
    out, kept = torch.empty_like(x), torch.zeros(rows, dtype=I32, device="cuda")
    tv.sample_filtered(x, noise, cu, t, kk, p, None, rows - half, tok, lp, st)
    tv.filter_logits(x, cu, t, kk, p, None, rows - half, out, kept, st)
    assert st.tolist() == [0, 0]
    again, kept2 = x.clone(), torch.zeros_like(kept)
    tv.filter_logits(again, cu, t, kk, p, None, rows - half, again, kept2, st)          # in place
    assert torch.equal(again, out) and torch.equal(kept, kept2)
    for r in {0, 1, half - 1, half, rows - 1}:
        b = int(r >= half)
        keep, s, w, margin = filter_ref(x[r].float().cpu().numpy(), (0.9, 1.2)[b], 0 if k is None else (k, 0)[b], (0.9, 0.6)[b], 0.0)
        assert margin > 2.0 ** -33
        token, logp = draw_ref(keep, s, w, noise[r].cpu().numpy())
        assert np.array_equal(out[r].float().cpu().numpy() > -np.inf, keep) and int(kept[r]) == int(keep.sum())
        assert int(tok[r]) == token and abs(float(lp[r]) - logp) <= 2.0 ** -18   # five roundings of up to 16
