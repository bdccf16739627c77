"""Filtered sampling and filtered logits on the GPU against their restatement
(oracle/filter_ref.py): kept sets and tokens are compared exactly, except where a
top-p border lies within rounding of its target (weights are good to 2^-35, a
margin of 2^-33 of the whole is counted as decided)."""

import math

import numpy as np
import pytest
import torch

import speculative_decoding_tree_build_gb300 as tv
from oracle import draw_ref, filter_ref, greedy_accept_ref, rejection_walk_ref, sampled_walk_ref
from gen import workloads as wl

pytestmark = pytest.mark.gpu

BF16, F32, I32 = torch.bfloat16, torch.float32, torch.int32
DECIDED = 2.0 ** -33
INF, NAN, LOWEST = math.inf, math.nan, -3.3895e38          # LOWEST: bf16's lowest value


def i32(x):
    return torch.tensor(x, dtype=I32, device="cuda")


def f32(x):
    return torch.tensor(x, dtype=F32, device="cuda")


def padded(rows, dtype, pad=NAN):
    """A [rows][vocab] view of rows that start on 16 bytes, `pad` behind them."""
    n, v = rows.shape
    ld = -(-v // 8) * 8 + 8
    full = torch.full((n, ld), pad, dtype=dtype, device="cuda")
    full[:, :v] = torch.from_numpy(np.ascontiguousarray(rows)).cuda().to(dtype)
    return full[:, :v]


def noise(rng, shape):
    return (-np.log(-np.log(rng.uniform(1e-7, 1 - 1e-7, shape)))).astype(np.float32)


def logp_bound(keep, s, w, token, v, filtered):
    """Of the float32 logarithm. A share above 1/2 is log1p(-a), a the quotient of two
    rounded sums: 3 roundings of a, one unit of log1p, a / (1 - a) <= 2 |logp|. Else
    ln 2 * (difference) - ln(total): four roundings of the difference, the sum's and
    the logarithm's own, one subtraction. Without a filter the total is a float32 sum
    of v / 512 terms a thread, each term's exponent rounded (2^-20 of it)."""
    top = float(np.max(s[keep]))
    a, b = abs(float(s[token]) - top), abs(float(np.log(w[keep].sum())))
    tol = 2.0 ** -24 * (8 * a + 8 * b + 8)
    if not filtered:
        tol += 2.0 ** -24 * (v / 512 + 64)
    return tol


def check(x, temps, ks, ps, ms, nodes=1, dtype=F32, seed=0, gumbel=None, exact_logp=True, skip=None):
    """Rows x [batch * nodes][v] of requests with settings of their own through both
    calls; returns the kept counts."""
    rng = np.random.default_rng(seed)
    rows, v = x.shape
    batch = rows // nodes
    lg = padded(x, dtype)
    x = lg.float().cpu().numpy()
    g = noise(rng, (rows, v)) if gumbel is None else gumbel
    gt = padded(g, F32)
    cu = i32([b * nodes for b in range(batch + 1)])
    tokens, logp = torch.full((rows,), -5, dtype=I32, device="cuda"), torch.full((rows,), 9.0, device="cuda")
    st = torch.zeros(batch, dtype=I32, device="cuda")
    opt = lambda a, make: None if a is None else make(a)
    args = (cu, f32(temps), opt(ks, i32), opt(ps, f32), opt(ms, f32), nodes)
    tv.sample_filtered(lg, gt, *args, tokens, logp, st)
    out = torch.empty(rows, lg.stride(0), dtype=dtype, device="cuda")
    out.fill_(123.0)
    kept = torch.full((rows,), -5, dtype=I32, device="cuda")
    tv.filter_logits(lg, *args, out[:, :v], kept, st)
    assert st.tolist() == [0] * batch
    assert bool((out[:, v:] == 123.0).all())
    out, kept, tokens, logp = out[:, :v].float().cpu().numpy(), kept.tolist(), tokens.tolist(), logp.tolist()
    undecided = 0
    for r in range(rows):
        b = r // nodes
        k, p, m = (0 if ks is None else ks[b]), (1.0 if ps is None else ps[b]), (0.0 if ms is None else ms[b])
        keep, s, w, margin = filter_ref(x[r], temps[b], k, p, m)
        if margin < DECIDED:
            undecided += 1
            continue
        assert kept[r] == int(keep.sum()), (r, kept[r], int(keep.sum()), margin)
        want = np.where(keep, x[r], -np.inf)
        assert np.array_equal(out[r], want, equal_nan=True), r
        token, lp = draw_ref(keep, s, w, g[r])
        if temps[b] == 0:
            token, lp = (int(np.nonzero(keep)[0][0]), 0.0) if keep.any() else (0, -INF)
        assert tokens[r] == token, (r, tokens[r], token)
        if not np.isfinite(lp) or not exact_logp or not np.isfinite(s[token]):
            assert logp[r] == pytest.approx(lp, abs=1e-5), r
        else:
            filtered = 0 < k < v or p < 1 or m > 0
            assert abs(logp[r] - lp) <= logp_bound(keep, s, w, token, v, filtered), (r, logp[r], lp)
    assert undecided <= (max(1, rows // 50) if skip is None else skip)
    return kept


def bulk(rng, rows, v, sigma=2.0, likely=40):
    x = rng.normal(0, sigma, (rows, v)).astype(np.float32)
    for r in range(rows):
        at = rng.integers(0, v, min(likely, v))
        x[r, at] += (14 * rng.random(len(at)) ** 2 + 2).astype(np.float32)
    return x


SETTINGS = [(0.8, 50, 1.0, 0.0), (1.0, 0, 0.95, 0.0), (1.2, 0, 1.0, 0.05), (0.0, 0, 1.0, 0.0), (0.7, 200, 0.9, 0.02),
            (1.0, 0, 1.0, 0.0), (1.0, 1, 1.0, 0.0), (1.5, 0, 0.5, 0.0), (0.9, 5, 0.3, 0.3), (1.0, 0, 0.0, 0.0),
            (2.0, 0, 0.999, 0.0), (1.0, 0, 1.0, 1.0)]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("v", [1, 2, 3, 7, 8, 33, 511, 1000, 4099, 8191, 8192, 8193, 8300, 32000, 151936])
def test_every_setting(v, dtype):
    rng = np.random.default_rng(v)
    n = len(SETTINGS)
    x = bulk(rng, 2 * n, v)
    t, k, p, m = zip(*SETTINGS)
    check(x, list(t), list(k), list(p), list(m), nodes=2, dtype=dtype, seed=v)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("sigma", [0.01, 1.0, 3.0])
@pytest.mark.parametrize("v", [9000, 60000, 151936])
def test_flat_rows(v, sigma, dtype):
    """Sets of a tenth of the vocabulary and more: borders that no list of the largest
    logits reaches."""
    rng = np.random.default_rng(v)
    settings = [(1.0, 0, 0.9, 0.0), (1.0, 0, 0.5, 0.0), (0.7, 0, 0.99, 0.0), (1.0, v // 3, 1.0, 0.0), (1.0, v // 2, 0.9, 0.0),
                (1.0, v - 1, 1.0, 0.0), (1.0, 8000, 0.99, 0.001), (1.0, 0, 1.0, 0.001), (1.0, 20, 0.9999, 0.0), (1.3, 0, 0.999999, 0.0)]
    t, k, p, m = zip(*settings)
    check(rng.normal(0, sigma, (len(settings), v)).astype(np.float32), list(t), list(k), list(p), list(m), dtype=dtype, seed=1)


@pytest.mark.parametrize("v", [100, 9001, 151936])
def test_ties(v):
    """Rows of one value, of two, of few: the kept tokens of equal logits are the first."""
    rng = np.random.default_rng(v)
    rows = [np.full(v, 2.5), np.full(v, -0.0), np.where(np.arange(v) % 2, 0.0, -0.0), np.where(np.arange(v) % 3, 1.0, 2.0),
            rng.integers(0, 4, v) * 1.0, rng.integers(0, 50, v) * 0.25, np.where(np.arange(v) == v - 1, 9.0, 0.0)]
    for setting in [(1.0, 0, 0.5, 0.0), (0.6, v // 2 + 1, 1.0, 0.0), (1.0, 7, 0.9, 0.0), (1.0, v - 1, 0.37, 0.0), (1.0, 0, 1.0, 0.3),
                    (1.0, 40, 1.0, 0.0)]:
        t, k, p, m = ([s] * len(rows) for s in setting)
        check(np.stack(rows).astype(np.float32), t, k, p, m, seed=2)


def test_equal_logits_split_exactly():
    """A half of equal tokens is a half of them, also where the sum is 2^17 weights."""
    for v in (2, 64, 1000, 9000, 131072):
        kept = check(np.full((1, v), 3.7, np.float32), [0.8], [0], [0.5], [0.0])
        assert kept == [v // 2]


@pytest.mark.parametrize("v", [64, 9000, 151936])
@pytest.mark.parametrize("mask", [-INF, LOWEST, -3.4028234663852886e38])
def test_masked_rows(v, mask):
    """A grammar that allows few tokens, one, or none; fewer allowed than top-k asks for."""
    rng = np.random.default_rng(v)
    rows = []
    for allowed in (0, 1, 3, 30, v // 2, v):
        x = np.full(v, mask, np.float32)
        at = rng.permutation(v)[:allowed]
        x[at] = rng.normal(0, 2, allowed)
        rows.append(x)
    x = np.stack(rows).astype(np.float32)
    for setting in SETTINGS:
        t, k, p, m = ([s] * len(rows) for s in setting)
        kept = check(x, t, k, p, m, seed=3)
        if mask == -INF:
            assert kept[0] == 0 and kept[1] == 1
    check(x[:5], [1.0] * 5, [v - 1] * 5, [0.9] * 5, [0.0] * 5, dtype=BF16 if mask != -3.4028234663852886e38 else F32)


@pytest.mark.parametrize("v", [40, 9000, 40001])
def test_infinities_and_nan(v):
    rng = np.random.default_rng(v)
    x = rng.normal(0, 2, (8, v)).astype(np.float32)
    x[0, 5] = INF
    x[1, [7, 3, 30]] = INF
    x[2, [9, 2]] = NAN
    x[3, 11], x[3, 12] = NAN, INF
    x[4, :] = INF
    x[5, :] = NAN
    x[6, ::2] = -INF
    x[7, 1:] = -INF
    for setting in SETTINGS:
        t, k, p, m = ([s] * 8 for s in setting)
        if setting[0] > 0 and setting[1:] == (0, 1.0, 0.0):
            continue                                 # without a filter: below
        check(x, t, k, p, m, seed=4)


def test_infinities_and_nan_without_a_filter():
    rng = np.random.default_rng(9)
    x = rng.normal(0, 2, (6, 3000)).astype(np.float32)
    x[0, 5] = INF
    x[1, [7, 3, 30]] = INF
    x[2, [9, 2]] = NAN
    x[3, ::2] = -INF
    x[4, :] = -INF
    x[5, 1:] = -INF
    check(x, [0.9] * 6, None, None, None, seed=5)
    got = check(x, [0.0] * 6, None, None, None, seed=5)
    assert got == [1, 1, 1, 1, 0, 1]


@pytest.mark.parametrize("v", [500, 20000])
@pytest.mark.parametrize("t", [1e-38, 1e-30, 1e-6, 1e-3, 0.01, 50.0, 1e6, 1e38])
def test_temperatures(v, t):
    """Scaled logits that overflow, underflow, and far from zero."""
    rng = np.random.default_rng(6)
    x = np.concatenate([bulk(rng, 3, v), bulk(rng, 2, v) * 1e-30, bulk(rng, 1, v) * 1e30, bulk(rng, 2, v) + 3000.0,
                        bulk(rng, 2, v) - 700.0]).astype(np.float32)
    for k, p, m in ((0, 0.9, 0.0), (30, 1.0, 0.0), (0, 1.0, 0.1), (100, 0.5, 0.01)):
        # of the two rows of 1e-30 every weight is 1 within 2^-70: where p of k is a whole
        # number (50 of 100), the border is the rounding's
        check(x, [t] * 10, [k] * 10, [p] * 10, [m] * 10, seed=7, exact_logp=False, skip=2 if k * p == 50 else 1)


def test_far_from_zero_at_the_bound():
    """Rows whose largest scaled logit lies about 512, where weights change their reference."""
    rng = np.random.default_rng(8)
    for v in (300, 30000):
        x = bulk(rng, 9, v, sigma=3.0)
        x += (np.array([490, 505, 510, 512, 520, 600, -500, -512, -530], np.float32) - x.max(1))[:, None]
        check(x, [1.0] * 9, [0] * 9, [0.95] * 9, [0.0] * 9, seed=1, exact_logp=False)
        check(x, [1.0] * 9, [200] * 9, [0.9] * 9, [0.0] * 9, seed=1, exact_logp=False)


def test_sorted_rows():
    """Rows in ascending and descending order, the largest logits in one place."""
    rng = np.random.default_rng(10)
    x = np.sort(bulk(rng, 4, 151936), axis=1)
    x = np.concatenate([x, x[:, ::-1]])
    for setting in ((1.0, 50, 1.0, 0.0), (1.0, 0, 0.9, 0.0), (1.0, 30000, 0.95, 0.0), (1.0, 0, 1.0, 1e-4)):
        t, k, p, m = ([s] * 8 for s in setting)
        check(x, t, k, p, m, seed=2)


def test_tokens_equal_the_sampler_s_without_filters():
    rng = np.random.default_rng(11)
    x, g = rng.normal(0, 2, (40, 32000)).astype(np.float32), noise(rng, (40, 32000))
    lg, gt = torch.from_numpy(x).cuda(), torch.from_numpy(g).cuda()
    cu, t = i32(list(range(0, 41, 4))), f32([0.0, 0.5, 1.0, 1.3, 0.8] * 2)
    st = torch.zeros(10, dtype=I32, device="cuda")
    a, b, c = (torch.empty(40, dtype=I32, device="cuda") for _ in range(3))
    tv.sample_tokens(lg, gt, cu, t, 4, a, st)
    tv.sample_filtered(lg, gt, cu, t, None, None, None, 4, b, None, st)
    # filters that keep all: the same through the filtering path
    tv.sample_filtered(lg, gt, cu, t, None, None, f32([1e-30] * 10), 4, c, None, st)
    assert torch.equal(a, b) and torch.equal(a, c) and not st.any()


def test_flags():
    rng = np.random.default_rng(12)
    v = 300
    settings = [(-1.0, 0, 1.0, 0.0, 64), (NAN, 0, 1.0, 0.0, 64), (INF, 0, 1.0, 0.0, 64), (1e-39, 0, 1.0, 0.0, 64),
                (1.0, -1, 1.0, 0.0, 256), (1.0, 0, 1.5, 0.0, 256), (1.0, 0, -0.1, 0.0, 256), (1.0, 0, NAN, 0.0, 256),
                (1.0, 0, 1.0, 1.1, 256), (1.0, 0, 1.0, -0.1, 256), (1.0, 0, 1.0, NAN, 256), (-1.0, -1, 1.0, 0.0, 320),
                (1.0, 5, 1.0, 0.0, 0), (0.0, 0, 1.0, 0.0, 0)]
    n = len(settings)
    t, k, p, m, want = zip(*settings)
    lg, gt = padded(rng.normal(0, 1, (2 * n, v)), F32), padded(noise(rng, (2 * n, v)), F32)
    cu = i32([2 * b for b in range(n + 1)])
    args = (cu, f32(t), i32(list(k)), f32(p), f32(m))
    tokens, logp = torch.full((2 * n,), -5, dtype=I32, device="cuda"), torch.full((2 * n,), 9.0, device="cuda")
    st = torch.zeros(n, dtype=I32, device="cuda")
    tv.sample_filtered(lg, gt, *args, 2, tokens, logp, st)
    assert st.tolist() == list(want)
    flagged = [r for b in range(n) if want[b] for r in (2 * b, 2 * b + 1)]
    assert tokens[flagged].tolist() == [-5] * len(flagged) and logp[flagged].tolist() == [9.0] * len(flagged)
    assert (tokens[-4:] >= 0).all()
    # the flagged are skipped afterwards, in the filter too
    kept = torch.full((2 * n,), -5, dtype=I32, device="cuda")
    out = padded(np.full((2 * n, v), 3.0), F32)
    tv.filter_logits(lg, *args, 2, out, kept, st)
    assert st.tolist() == list(want) and bool((out[flagged] == 3.0).all()) and (kept[flagged] == -5).all()
    assert kept[-4:].tolist() == [5, 5, 1, 1]
    # more nodes than allowed; no noise
    st = torch.zeros(2, dtype=I32, device="cuda")
    tokens.fill_(-5)
    tv.sample_filtered(lg, None, i32([0, 3, 4]), f32([0.0, 0.5]), None, None, None, 2, tokens, logp, st)
    assert st.tolist() == [1, 64] and (tokens == -5).all()
    st.zero_()
    tv.sample_filtered(lg, None, i32([0, 0, 2]), f32([0.5, 0.0]), None, None, None, 2, tokens, None, st)
    assert st.tolist() == [0, 0] and (tokens[:2] >= 0).all() and (tokens[2:] == -5).all()


def test_refusals_of_tensors():
    lg, gt = torch.zeros(4, 64, device="cuda"), torch.zeros(4, 64, device="cuda")
    cu, t, st = i32([0, 2, 4]), f32([1.0, 1.0]), torch.zeros(2, dtype=I32, device="cuda")
    tok, lp = torch.zeros(4, dtype=I32, device="cuda"), torch.zeros(4, device="cuda")
    k, p = i32([1, 1]), f32([0.5, 0.5])
    for bad in (lambda: tv.sample_filtered(lg.half(), gt, cu, t, k, p, p, 2, tok, lp, st),
                lambda: tv.sample_filtered(lg.t(), gt, cu, t, k, p, p, 2, tok, lp, st),
                lambda: tv.sample_filtered(lg, gt[:3], cu, t, k, p, p, 2, tok, lp, st),
                lambda: tv.sample_filtered(lg, gt[:, :60], cu, t, k, p, p, 2, tok, lp, st),
                lambda: tv.sample_filtered(lg, gt, cu, t, p, p, p, 2, tok, lp, st),
                lambda: tv.sample_filtered(lg, gt, cu, t, k, k, p, 2, tok, lp, st),
                lambda: tv.sample_filtered(lg, gt, cu, t[:1], k, p, p, 2, tok, lp, st),
                lambda: tv.sample_filtered(lg, gt, cu, t, k, p, p, 2, tok[:3], lp, st),
                lambda: tv.sample_filtered(lg, gt, cu, t, k, p, p, "2", tok, lp, st),
                lambda: tv.sample_filtered(lg.cpu(), gt, cu, t, k, p, p, 2, tok, lp, st),
                lambda: tv.filter_logits(lg, cu, t, k, p, p, 2, lg.bfloat16(), tok, st),
                lambda: tv.filter_logits(lg, cu, t, k, p, p, 2, lg[:3], tok, st),
                lambda: tv.filter_logits(lg, cu, t, k, p, p, 2, lg, tok.long(), st)):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(tv.TvError):
        tv.filter_logits(lg[:, 1:], cu, t, k, p, p, 2, lg[:, 1:], tok, st)     # not on 16 bytes
    with pytest.raises(tv.TvError):
        tv.sample_filtered(lg, gt, cu, t, k, p, p, 0, tok, lp, st)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_in_place_ragged_and_captured(dtype):
    """Requests of 0 to 5 nodes, filtered in place, captured and replayed on new logits."""
    rng = np.random.default_rng(13)
    lens, v = [3, 0, 5, 1, 2], 20011
    rows = sum(lens)
    cu = i32([0] + np.cumsum(lens).tolist())
    t, k, p, m = [0.7, 1.0, 1.0, 0.0, 1.1], [0, 3, 50, 0, 0], [0.9, 1.0, 0.8, 1.0, 1.0], [0.0, 0.0, 0.0, 0.0, 0.1]
    spread = np.repeat(np.arange(5), lens)
    x = padded(bulk(rng, rows + 2, v), dtype)
    buf = torch.empty_strided(x.shape, x.stride(), dtype=dtype, device="cuda")
    st, kept = torch.zeros(5, dtype=I32, device="cuda"), torch.full((rows + 2,), -5, dtype=I32, device="cuda")
    args = (cu, f32(t), i32(k), f32(p), f32(m), 5)
    buf.copy_(x)
    tv.filter_logits(buf, *args, buf, kept, st)                # (first call outside the capture)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        tv.filter_logits(buf, *args, buf, kept, st)
    for turn in range(2):
        x = padded(bulk(rng, rows + 2, v), dtype)
        buf.copy_(x)
        graph.replay()
        assert not st.any() and kept[rows:].tolist() == [-5, -5]
        assert torch.equal(buf[rows:], x[rows:])               # rows of no request
        host = x.float().cpu().numpy()
        for r in range(rows):
            b = spread[r]
            keep, _, _, margin = filter_ref(host[r], t[b], k[b], p[b], m[b])
            if margin >= DECIDED:
                assert np.array_equal(buf[r].float().cpu().numpy(), np.where(keep, host[r], -np.inf)), (turn, r)


def test_the_same_twice_and_on_two_streams():
    rng = np.random.default_rng(14)
    x, g = bulk(rng, 64, 50000, sigma=3.0), noise(rng, (64, 50000))
    lg, gt = torch.from_numpy(x).cuda(), torch.from_numpy(g).cuda()
    cu, t = i32(list(range(65))), f32([0.9] * 64)
    k, p, m = i32([0, 100, 0, 20000] * 16), f32([0.95, 0.9, 1.0, 0.99] * 16), f32([0.0, 0.01, 0.02, 0.0] * 16)
    torch.cuda.synchronize()
    outs = []
    streams = [torch.cuda.Stream() for _ in range(2)]
    for turn in range(4):
        tok, lp, st = torch.empty(64, dtype=I32, device="cuda"), torch.empty(64, device="cuda"), torch.zeros(64, dtype=I32, device="cuda")
        torch.cuda.synchronize()
        tv.sample_filtered(lg, gt, cu, t, k, p, m, 1, tok, lp, st, streams[turn % 2])
        outs.append((tok, lp))
    torch.cuda.synchronize()
    for tok, lp in outs[1:]:
        assert torch.equal(tok, outs[0][0]) and torch.equal(lp, outs[0][1])


def test_sampled_and_rejection_walks_on_filtered_logits():
    """A tree step's acceptance under top-k and top-p: tokens drawn at every node and
    walked greedily, the walk on masked logits, and rejection against them."""
    w = wl.make_config(2, batch=4)
    rng = np.random.default_rng(15)
    v = w["vocab"]
    logits, gumbel = wl.sampling_inputs(rng, w)
    dev = lambda a: torch.from_numpy(a).cuda()
    lg, gt = dev(logits), dev(gumbel)
    T, batch, mn, md = lg.shape[0], w["batch"], int(w["max_nodes"]), int(w["max_depth"])
    t, k, p = [0.8, 1.0, 0.0, 1.2], [40, 0, 0, 300], [1.0, 0.9, 1.0, 0.95]
    args = (dev(w["cu_nodes"].astype(np.int32)), f32(t), i32(k), f32(p), None, mn)
    cu, parents, draft = args[0], dev(w["parents"].astype(np.int32)), dev(w["draft_tokens"].astype(np.int32))
    st, tok = torch.zeros(batch, dtype=I32, device="cuda"), torch.empty(T, dtype=I32, device="cuda")
    tv.sample_filtered(lg, gt, *args, tok, None, st)
    masked, kept = torch.empty_like(lg), torch.empty(T, dtype=I32, device="cuda")
    tv.filter_logits(lg, *args, masked, kept, st)
    path, alen, bonus = torch.full((batch, md + 1), -9, dtype=I32, device="cuda"), torch.zeros(batch, dtype=I32, device="cuda"), torch.zeros(batch, dtype=I32, device="cuda")
    tv.sampled_accept(masked, gt, cu, args[1], parents, draft, mn, path, alen, bonus, st)
    assert not st.any()
    host, tok = masked.cpu().numpy(), tok.cpu().numpy()
    for b in range(batch):
        sl = slice(int(w["cu_nodes"][b]), int(w["cu_nodes"][b + 1]))
        par, dr = w["parents"][sl], w["draft_tokens"][sl]
        _, a, bo = sampled_walk_ref(par, dr, host[sl], gumbel[sl], t[b], md)
        _, a2, bo2 = greedy_accept_ref(par, dr, tok[sl], md)
        assert (list(a), bo) == (list(a2), bo2)
        assert int(alen[b]) == len(a) - 1 and int(bonus[b]) == bo and path[b, :len(a)].tolist() == list(a)
    # rejection: the drafter's logits filtered by top-k at temperature 1
    lgr, dr_l, gb, un, lp = wl.rejection_inputs(rng, w)
    one, top = f32([1.0] * batch), i32([60] * batch)
    target, drafter = torch.empty_like(lg), torch.empty_like(lg)
    tv.filter_logits(dev(lgr), cu, f32([0.9] * batch), top, None, None, mn, target, None, st)
    tv.filter_logits(dev(dr_l), cu, one, top, None, None, mn, drafter, None, st)
    path.fill_(-9)
    tv.rejection_accept(target, drafter, dev(gb), dev(un), cu, f32([0.9] * batch), parents, draft, dev(lp), mn, path, alen, bonus, st)
    assert not st.any()
    th, dh = target.cpu().numpy(), drafter.cpu().numpy()
    for b in range(batch):
        sl = slice(int(w["cu_nodes"][b]), int(w["cu_nodes"][b + 1]))
        rs, acc, bo, det = rejection_walk_ref(w["parents"][sl], w["draft_tokens"][sl], lp[sl], th[sl], dh[sl], un[sl], gb[sl], 0.9, md)
        key = np.sort(det["stop"][1])
        if all(abs(u - x) > 1e-5 for u, x in det["ratios"]) and key[-1] - key[-2] > 1e-5:      # no near ties
            assert rs == 0 and int(alen[b]) == len(acc) - 1 and int(bonus[b]) == bo
        last = sl.start + int(path[b, int(alen[b])])
        assert th[last, int(bonus[b])] > -np.inf     # the draw is of a token that the target keeps


def test_large_vocabulary_and_many_rows():
    """Offsets past 2^31 elements: the last rows of 5 GB of logits."""
    v, rows = 1 << 20, 2304
    free, _ = torch.cuda.mem_get_info()
    assert free > 16 << 30
    lg = torch.full((rows, v), -5.0, dtype=BF16, device="cuda")
    lg[-3:, 1000:1010] = torch.arange(10, device="cuda", dtype=F32).to(BF16)
    batch = 3
    cu = i32([0, 1000, 2000, rows])
    st, kept = torch.zeros(batch, dtype=I32, device="cuda"), torch.zeros(rows, dtype=I32, device="cuda")
    tv.filter_logits(lg, cu, f32([1.0] * 3), i32([4] * 3), None, None, 1000, lg, kept, st)
    assert not st.any() and kept.unique().tolist() == [4]
    assert (lg[-1] > -INF).nonzero().flatten().tolist() == [1006, 1007, 1008, 1009]
    assert (lg[1500] > -INF).nonzero().flatten().tolist() == [0, 1, 2, 3]
