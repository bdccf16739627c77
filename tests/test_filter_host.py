"""The restatement of top-k, top-p and min-p against brute force and closed forms,
and the host-side refusals of the calls."""

import itertools
import math

import numpy as np
import pytest

import speculative_decoding_tree_build_gb300 as tv
from oracle import draw_ref, filter_ref, sample_tokens_ref
from speculative_decoding_tree_build_gb300.build import build

P = 0x10000  # a non-null, 256-byte aligned value; never dereferenced
OK, NULL, GEOM, SIZE, MIS = 0, -1, -2, -3, -5


@pytest.fixture(scope="module")
def lib():
    build()
    return tv.load()


def swap(args, **at):
    out = list(args)
    for i, v in at.items():
        out[int(i[1:])] = v
    return out


def test_sample_filtered_refusals(lib):
    # dtype, logits, ld, gumbel, ld, cu, temperature, top_k, top_p, min_p, batch, max_nodes, vocab,
    # tokens, logp, status, stream
    args = [1, P, 1000, P, 1000, P, P, P, P, P, 2, 8, 1000, P, P, P, None]

    def call(a):
        return lib.tv_sample_filtered(*a)

    assert call(swap(args, _10=0)) == OK
    assert call(swap(args, _0=2)) == GEOM and call(swap(args, _0=-1)) == GEOM
    for i, v in ((2, 999), (4, 999), (10, -1), (10, 65536), (11, 0), (11, 1025), (12, 0), (12, (1 << 30) + 1)):
        assert call(swap(args, **{f"_{i}": v})) == SIZE
    for i in (1, 5, 6, 13, 15):
        assert call(swap(args, **{f"_{i}": None})) == NULL
    for i, v in ((1, P + 8), (2, 1002), (3, P + 4), (4, 1002)):
        assert call(swap(args, **{f"_{i}": v})) == MIS
    assert call(swap(args, _0=0, _2=1004)) == MIS                 # bf16 rows lie 8 elements apart


def test_filter_logits_refusals(lib):
    # dtype, logits, ld, cu, temperature, top_k, top_p, min_p, batch, max_nodes, vocab, out, ld, kept,
    # status, stream
    args = [0, P, 1000, P, P, P, P, P, 2, 8, 1000, P, 1000, P, P, None]

    def call(a):
        return lib.tv_filter_logits(*a)

    assert call(swap(args, _8=0)) == OK
    assert call(swap(args, _0=2)) == GEOM
    for i, v in ((2, 999), (12, 999), (8, -1), (8, 65536), (9, 0), (9, 1025), (10, 0)):
        assert call(swap(args, **{f"_{i}": v})) == SIZE
    for i in (1, 3, 4, 11, 14):
        assert call(swap(args, **{f"_{i}": None})) == NULL
    for i, v in ((1, P + 8), (2, 1004), (11, P + 2), (12, 1004)):
        assert call(swap(args, **{f"_{i}": v})) == MIS


def test_small_rows_by_brute_force():
    """Every subset of 5 tokens: the kept set is the smallest one that holds the most
    probable tokens and reaches p."""
    rng = np.random.default_rng(1)
    for _ in range(200):
        x = rng.normal(0, 2, 5).astype(np.float32)
        k, p = int(rng.integers(0, 7)), float(np.float32(rng.uniform(0.05, 1)))
        keep, s, w, _ = filter_ref(x, 1.0, k, p)
        prob = np.exp(x.astype(np.float64))
        inside = np.argsort(-prob)[:k if 0 < k < 5 else 5]
        prob /= prob[inside].sum()
        best = None
        for n in range(1, len(inside) + 1):
            for c in itertools.combinations(inside.tolist(), n):
                if best is None and sum(prob[list(c)]) >= p - 1e-12 and all(prob[i] >= prob[j] for i in c for j in inside if j not in c):
                    best = set(c)
            if best:
                break
        assert set(np.nonzero(keep)[0].tolist()) == best


def test_closed_forms():
    u = np.zeros(8, np.float32)                      # equal logits: the first ceil(8 p) tokens
    for p, n in ((0.5, 4), (0.500001, 5), (0.125, 1), (0.01, 1), (0.0, 1), (1.0, 8)):
        assert np.nonzero(filter_ref(u, 0.7, 0, p)[0])[0].tolist() == list(range(n))
    assert np.nonzero(filter_ref(u, 1.0, 3)[0])[0].tolist() == [0, 1, 2]
    g = -np.arange(20, dtype=np.float32)             # geometric with ratio 1/e: 1 - e^-n of the mass in n tokens
    for n in range(1, 12):
        assert filter_ref(g, 1.0, 0, float(1 - math.exp(-n)) - 1e-6)[0].sum() == n
        assert filter_ref(g, 1.0, 0, 1.0, float(math.exp(-n) * (1 - 1e-6)))[0].sum() == n + 1
        assert filter_ref(g, 0.5, 0, 1.0, float(math.exp(-2 * n) * (1 - 1e-6)))[0].sum() == n + 1


def test_masks_infinities_and_nan():
    i, n = np.inf, np.nan
    keep = lambda x, **kw: np.nonzero(filter_ref(np.array(x, np.float32), 1.0, **kw)[0])[0].tolist()
    assert keep([-i, -i]) == [] and keep([-i, 3, -i], top_k=2) == [1]
    assert keep([0, i, -i, i, 5], top_p=0.5) == [1] and keep([0, i, -i, i, 5], top_p=0.6) == [1, 3]
    assert keep([0, i, -i, i, 5], top_k=3) == [1, 3, 4] and keep([0, i, 5], min_p=0.5) == [1]
    assert keep([0, n, i], top_k=1) == [1] and keep([0, n, i, n], min_p=0.1) == [1, 3]
    assert draw_ref(*filter_ref(np.full(3, -i, np.float32), 1.0)[:3], np.zeros(3, np.float32)) == (0, -math.inf)


def test_without_filters_tokens_are_the_sampler_s():
    rng = np.random.default_rng(2)
    for t in (0.0, 0.6, 1.3):
        for _ in range(20):
            x = rng.normal(0, 3, 500).astype(np.float32)
            g = -np.log(-np.log(rng.uniform(1e-7, 1, 500))).astype(np.float32)
            keep, s, w, _ = filter_ref(x, t)
            assert draw_ref(keep, s, w, g)[0] == sample_tokens_ref(x[None], g[None], t)[0]


def test_draws_follow_the_kept_distribution():
    rng = np.random.default_rng(3)
    x = np.array([1.0, 0.5, 0.2, -1.0, 2.0], np.float32)
    keep, s, w, _ = filter_ref(x, 1.0, 3)
    p = np.where(keep, w, 0) / w[keep].sum()
    n = 20000
    got = np.bincount([draw_ref(keep, s, w, -np.log(-np.log(rng.random(5))))[0] for _ in range(n)], minlength=5) / n
    # five standard deviations of a share of n draws
    assert np.all(np.abs(got - p.astype(float)) <= 5 * np.sqrt(0.25 / n)) and got[~keep].sum() == 0
