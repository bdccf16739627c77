"""Filtered sampling and masks at the ends of float32."""

import math

import numpy as np
import pytest
import torch

import speculative_decoding_tree_build_gb300 as tv
from oracle import draw_ref, filter_ref

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


# ------------------------------------------------------------------- the smallest temperatures


@pytest.mark.parametrize("t", [3e-39, 4e-39, 5e-39])
@pytest.mark.parametrize("v", [300, 9000, 40001])
@pytest.mark.parametrize("value", [0.0, 1e-37, -1e-37])
def test_equal_logits_at_the_smallest_temperatures(v, t, value):
    """1 / T is finite from 2.94e-39 on, times log2 e it is not below 4.24e-39."""
    x = torch.full((2, v), value)
    for p in (0.5, 0.25):
        _, lp, out, kept = both(x, t, None, p, None)
        want = math.ceil(p * v)
        assert kept == [want] * 2
        assert bool((out[:, :want] == x[0, 0].item()).all()) and bool((out[:, want:] == -INF).all())
        assert max(abs(a + math.log(want)) for a in lp) <= 2.0 ** -22 * math.log(want)


@pytest.mark.parametrize("t", [3e-39, 4e-39])
@pytest.mark.parametrize("v", [300, 9000])
@pytest.mark.parametrize("k,p,m", [(None, 0.9, None), (50, 0.9, None), (None, None, 0.1), (0, 0.5, 0.01)])
def test_small_logits_at_the_smallest_temperatures(v, t, k, p, m):
    """Logits of 1e-38: scaled, they are a row like any other."""
    rng = np.random.default_rng(v)
    x = (rng.normal(0, 1, (3, v)) * 1e-38).astype(np.float32)
    g = (-np.log(-np.log(rng.uniform(1e-7, 1 - 1e-7, (3, v))))).astype(np.float32)
    tok, lp, out, kept = both(torch.from_numpy(x), t, k, p, m, torch.from_numpy(g))
    for r in range(3):
        keep, s, w, margin = filter_ref(x[r], t, k or 0, 1.0 if p is None else p, m or 0.0)
        assert margin > 2.0 ** -33
        token, logp = draw_ref(keep, s, w, g[r])
        assert kept[r] == int(keep.sum()) and tok[r] == token
        assert np.array_equal(out[r].cpu().numpy() > -np.inf, keep)
        assert abs(lp[r] - logp) <= 2.0 ** -24 * (8 * abs(logp) + 8 * math.log(v) + 8)


# ------------------------------------------------------- log-probabilities of unfiltered rows


def unfiltered_bound(scaled, logp, entries):
    """Of the log-probability of a row without a filter, `entries` of it a thread. A
    term: the difference from the reference and its product with log2 e are rounded
    (a (2^-24 + 2^-24 + 2^-26) for an exponent of a, 1 for the reference's place), ex2 is
    good to 2^-22. Moves of the reference: ln n + 2 of them count, each expf's 2^-23 and
    the difference's 2^-24. A thread's sum brought to the CTA's reference, a CTA's to the
    cluster's: ex2 and the exponent again. Additions of a warp's lanes, a CTA's warps and a
    cluster's CTAs: 5 + 8 + 8. ln of the sum: 2^-23 of it; the difference and the last
    subtraction 2^-24 each."""
    s = scaled.astype(np.float64)
    top = s.max()
    w = np.exp(s - top)
    far = float((w * (top - s)).sum() / w.sum()) + 1
    total = float(np.log(w.sum())) + 1
    return (far * 2.25 * 2.0 ** -24 + 2.0 ** -22 + (math.log(entries) + 2) * 1.5 * 2.0 ** -23 +
            2 * (2.0 ** -22 + 2.0 ** -23) + 21 * 2.0 ** -24 + total * 2.0 ** -23 + (abs(logp) + 1) * 2.0 ** -24)


@pytest.mark.parametrize("v,rows", [(32000, 3), (151936, 5), (1 << 20, 2), (32000, 400), (151936, 320), (1 << 20, 310)])
@pytest.mark.parametrize("order", ["up", "down", "stairs", "any"])
def test_unfiltered_logp_of_ordered_rows(v, rows, order):
    """Rows that rise, fall or rise in steps from end to end, by 0.01 to 60; few rows have a
    cluster each, many a CTA."""
    at = torch.linspace(0, 1, v, device="cuda", dtype=torch.float64)
    if order == "down":
        at = at.flip(0)
    elif order == "stairs":
        at = (at * 40).floor() / 40
    elif order == "any":
        g = torch.Generator(device="cuda")
        g.manual_seed(v)
        at = at[torch.randperm(v, generator=g, device="cuda")]
    x = torch.empty(rows, v, device="cuda")
    for r, rise in enumerate(np.logspace(-2, 1.778, rows)):
        x[r] = (at * rise).float()
    noise = torch.zeros(rows, v, device="cuda")
    tok, lp, st = i32([0] * rows), f32([0.0] * rows), i32([0])
    tv.sample_filtered(x, noise, i32([0, rows]), f32([1.0]), None, None, None, rows, tok, lp, st)
    assert not st.any()
    assert torch.equal(tok.long(), x.argmax(-1))
    for r in range(0, rows, max(1, rows // 12)):
        logp = float(x[r, tok[r]].double() - torch.logsumexp(x[r].double(), 0))
        host = x[r].cpu().numpy()
        assert abs(float(lp[r]) - logp) <= unfiltered_bound(host, logp, v // (8 * 256) if rows < 10 else v // 256), r


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("t", [0.3, 1.0, 1.7])
@pytest.mark.parametrize("v,rows", [(7, 3), (1000, 5), (32000, 7), (151936, 6), (50000, 400)])
def test_unfiltered_logp_of_drawn_tokens(v, rows, t, dtype):
    rng = np.random.default_rng(v)
    x = torch.from_numpy((rng.normal(0, 2, (rows, v))).astype(np.float32)).to(dtype)
    g = torch.from_numpy((-np.log(-np.log(rng.uniform(1e-7, 1 - 1e-7, (rows, v))))).astype(np.float32))
    ld = -(-v // 8) * 8
    lg, gumbel = torch.zeros(rows, ld, dtype=dtype, device="cuda")[:, :v], torch.zeros(rows, ld, device="cuda")[:, :v]
    lg.copy_(x)
    gumbel.copy_(g)
    tok, lp, st = i32([0] * rows), f32([0.0] * rows), i32([0])
    tv.sample_filtered(lg, gumbel, i32([0, rows]), f32([t]), None, None, None, rows, tok, lp, st)
    assert not st.any()
    for r in range(0, rows, max(1, rows // 12)):
        keep, s, w, _ = filter_ref(x[r].float().numpy(), t)
        token, logp = draw_ref(keep, s, w, g[r].numpy())
        assert int(tok[r]) == token
        assert abs(float(lp[r]) - logp) <= unfiltered_bound(s, logp, max(1, v // 256)), r


# ------------------------------------------------------------------------ calls that overlap


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("rows,nodes,v", [(24, 1, 50000), (64, 1, 50000), (330, 66, 20000)])
def test_two_streams_at_once(rows, nodes, v, dtype):
    """Calls issued in turn to two streams with no wait between them, other logits on each:
    few rows leave SMs to the other stream's call. Every output equals the one of a call
    alone."""
    batch = rows // nodes
    settings = [(0.9, 0, 0.95, 0.0), (0.7, 100, 0.9, 0.01), (1.0, 0, 1.0, 0.02), (1.1, 15000, 0.99, 0.0), (1.0, 0, 1.0, 0.0)]
    t, k, p, m = zip(*[settings[b % 5] for b in range(batch)])
    args = (i32([b * nodes for b in range(batch + 1)]), f32(list(t)), i32(list(k)), f32(list(p)), f32(list(m)), nodes)
    sides = []
    for seed in (1, 2):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        x = (torch.randn(rows, v, generator=g, device="cuda") * 3).to(dtype)
        u = torch.rand(rows, v, generator=g, device="cuda").clamp(1e-7, 1 - 1e-7)
        turns = [{"tok": i32([-5] * rows), "lp": f32([9.0] * rows), "out": torch.zeros_like(x), "kept": i32([-5] * rows),
                  "st": i32([0] * batch)} for _ in range(6)]
        sides.append({"x": x, "g": -torch.log(-torch.log(u)), "turns": turns, "stream": torch.cuda.Stream()})

    def make(side, o, stream=None):
        tv.sample_filtered(side["x"], side["g"], *args, o["tok"], o["lp"], o["st"], stream)
        tv.filter_logits(side["x"], *args, o["out"], o["kept"], o["st"], stream)

    for side in sides:                       # the first turn alone, and over before the others begin
        make(side, side["turns"][0])
    torch.cuda.synchronize()
    for turn in range(1, 6):
        for side in sides:
            make(side, side["turns"][turn], side["stream"])
    torch.cuda.synchronize()
    for side in sides:
        first = side["turns"][0]
        assert not first["st"].any() and bool((first["tok"] >= 0).all())
        for o in side["turns"][1:]:
            assert all(torch.equal(o[n], first[n]) for n in first)
    assert not torch.equal(sides[0]["turns"][0]["tok"], sides[1]["turns"][0]["tok"])
