"""The plain-decoding and 8-bit-cache calls at the edges of what they allow:
counts past 32 bits, offsets that overlap, values that are not finite, more
units than thread blocks, and the measured cases' own plain forms."""

import importlib.util
import os
import random
import subprocess
import sys

import numpy as np
import pytest
import torch

import speculative_decoding_tree_build_gb300 as tv
import test_gpu_decode_ops as base

pytestmark = pytest.mark.gpu

ROOT = base.ROOT
BF16, F32, I32 = torch.bfloat16, torch.float32, torch.int32


def in_a_process(code):
    """A refusal must not end the interpreter, so it is looked at from outside."""
    out = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300, cwd=ROOT,
                         env={**os.environ, "PYTHONPATH": ROOT})
    assert out.returncode == 0, (out.returncode, out.stderr[-2000:])
    return out.stdout


@pytest.mark.parametrize("call", ["rope", "read"])
def test_more_rows_than_32_bits_are_refused(call):
    """2^31 rows (8.6 GB) or requests: ValueError, and the process lives on and calls again."""
    said = in_a_process("""
import torch
import speculative_decoding_tree_build_gb300 as tv
n = 2 ** 31
big = torch.empty(n, dtype=torch.int32, device="cuda")
try:
    if %r == "rope":
        q = big.view(torch.bfloat16).view(n, 1, 2)
        tv.rope_axes(tv.rope_axes_geom(1, 0, 2, [1]), q, None, big[None], torch.ones(1, device="cuda"), q, None)
    else:
        pool = torch.zeros(1, 1, 16, 64, dtype=torch.int8, device="cuda")
        scale, out = torch.zeros(1, 1, 16, device="cuda"), torch.zeros(1, 1, 16, 64, dtype=torch.bfloat16, device="cuda")
        tv.kv_quant_read(tv.geom(1, 1, 64), None, big, big[:, None], big, pool, pool, scale, scale, big[:, None], big,
                         out, out, big)
    print("no error")
except ValueError as e:
    print("refused:", e)
q = torch.ones(1, 1, 2, device="cuda")
tv.rope_axes(tv.rope_axes_geom(1, 0, 2, [1]), q, None, torch.zeros(1, 1, dtype=torch.int32, device="cuda"),
             torch.ones(1, device="cuda"), q, None)
print("and again", q.flatten().tolist())
""" % call)
    assert "refused:" in said and "out of range" in said and "and again [1.0, 1.0]" in said


# ---------------------------------------------------------------- one-token attention: values that are not finite


def widened(c, width):
    """The same cache behind a block table of `width` pages (many take the form of two launches)."""
    if width > c.table.shape[1]:
        wide = torch.full((c.table.shape[0], width), -1, dtype=I32, device="cuda")
        wide[:, :c.table.shape[1]] = c.table
        c.table = wide
    return c


def put_values(c, b, row, pool, values):
    """values: {column: value} of one cached row, all heads, of a bf16 pool."""
    page, at = c.at(b, [row])
    for col, x in values.items():
        pool[page, :, at, col] = x


def check_special(c, q, lens, out, lse):
    """As base.check_decode, but infinities and NaN have to be where the definition has them."""
    with np.errstate(invalid="ignore"):
        for b, n in enumerate(lens):
            k, v = c.rows(b, n)
            want, wl, tol, ltol = base.decode_tolerance(base.f64(q[b]), k, v, q.shape[2] ** -0.5, c.held,
                                                        c.value_scales(b, n))
            got, gl = base.f64(out[b]), base.f64(lse[b])
            fin = np.isfinite(want)
            assert np.array_equal(np.isnan(got), np.isnan(want)), b
            assert np.array_equal(np.isposinf(got), np.isposinf(want)) and np.array_equal(np.isneginf(got), np.isneginf(want)), b
            assert np.all(np.abs(got - want)[fin] <= tol[fin]), b
            fin = np.isfinite(wl)
            assert np.array_equal(np.isnan(gl), np.isnan(wl)) and np.all(np.abs(gl - wl)[fin] <= ltol[fin]), b


INF, NAN = float("inf"), float("nan")


@pytest.mark.parametrize("width", [1, 2400])
@pytest.mark.parametrize("hq,hkv,d", [(4, 1, 64), (8, 2, 128), (24, 2, 128), (9, 1, 64)])
def test_infinite_values_reach_the_output(hq, hkv, d, width):
    """Infinities and NaN of a bf16 value pool, beside weights of every kind: exactly 1 (one key),
    rounded up and rounded down; in the last, a middle and the first row."""
    lens = [1, 2, 16, 17, 40, 300, 1200]
    c = widened(base.filled(201, lens, hkv, d, "bf16"), width)
    q = torch.randn(len(lens), hq, d, generator=base.gen(202), device="cuda").to(BF16)
    for b, n in enumerate(lens):
        put_values(c, b, n - 1, c.v, {3: INF, 7: -INF, 11: INF, 13: NAN})
        put_values(c, b, n // 2, c.v, {5: INF, d - 1: -INF, 11: -INF if n > 1 else INF})
        put_values(c, b, 0, c.v, {20: INF, 21: 3e38, 22: -INF})
    out, lse, status = base.run_decode(c, q, lens)
    assert status == [0] * len(lens)
    assert bool(torch.isposinf(out[:, :, [3, 5, 20]]).all()) and bool(torch.isneginf(out[:, :, [7, 22, d - 1]]).all())
    check_special(c, q, lens, out, lse)


@pytest.mark.parametrize("width", [1, 2400])
def test_scores_that_are_not_finite(width):
    """bf16 keys: a score of -inf has no weight, one of +inf or NaN makes the query's output NaN, and
    no other query's, head's or request's. A query that is not finite spoils itself alone."""
    lens, hkv, d = [1, 33, 700, 50], 2, 64
    c = widened(base.filled(203, lens, hkv, d, "bf16"), width)
    q = torch.randn(4, 8, d, generator=base.gen(204), device="cuda").to(BF16)
    q[:, :, 9] = torch.tensor([1.0, 0.5, -1.0, 2.0, 1.0, 1.0, 1.0, 3.0], device="cuda").to(BF16)
    for b in (1, 2):
        put_values(c, b, lens[b] // 2, c.k, {9: -INF})    # queries 0, 1, 3..7: -inf; query 2: +inf
    q[0, 1, 4], q[0, 6, 4], q[3, 5, 0] = NAN, INF, -INF
    out, lse, status = base.run_decode(c, q, lens)
    assert status == [0] * 4
    nan = torch.isnan(out).all(-1).tolist()
    assert torch.isnan(out).any(-1).tolist() == nan
    assert nan[1] == nan[2] == [i == 2 for i in range(8)]
    assert nan[0] == [i in (1, 6) for i in range(8)] and nan[3] == [i == 5 for i in range(8)]
    good = ~torch.tensor(nan, device="cuda")
    for b in range(4):
        k, v = c.rows(b, lens[b])
        keep = np.isfinite(k).all((1, 2))                  # the key with a score of -inf left out
        want, wl, tol, ltol = base.decode_tolerance(base.f64(torch.nan_to_num(q[b], 0, 0, 0)), k[keep], v[keep], d ** -0.5, "bf16")
        ok = good[b].cpu().numpy()
        assert np.all(np.abs(base.f64(out[b]) - want)[ok] <= tol[ok])
        assert np.all(np.abs(base.f64(lse[b]) - wl)[ok] <= ltol[ok])


@pytest.mark.parametrize("width", [1, 2400])
@pytest.mark.parametrize("held", ["e4m3", "int8"])
def test_marked_rows_of_an_8_bit_cache(held, width):
    """A row that was not finite reads as NaN: a value row makes its head's outputs NaN and leaves the
    log-sum-exp, a key row makes both NaN."""
    lens, hkv, d = [20, 1, 600, 33], 2, 128
    c = widened(base.filled(205, lens, hkv, d, held), width)
    q = torch.randn(4, 8, d, generator=base.gen(206), device="cuda").to(BF16)
    page, at = c.at(0, [7])
    c.vs[page, 0, at] = NAN                               # a value row of request 0, head 0
    page, at = c.at(2, [599])
    c.ks[page, 1, at] = NAN                               # a key row of request 2, head 1
    out, lse, status = base.run_decode(c, q, lens)
    assert status == [0] * 4
    bad = torch.zeros(4, 8, dtype=torch.bool, device="cuda")
    bad[0, :4] = bad[2, 4:] = True
    assert torch.equal(torch.isnan(out).all(-1), bad) and torch.equal(torch.isnan(out).any(-1), bad)
    bad[0] = False
    assert torch.equal(torch.isnan(lse), bad)
    base.check_decode(c, q, lens, out, lse, which=[1, 3])


@pytest.mark.parametrize("width", [1, 2400])
def test_an_infinite_value_of_little_weight(width):
    """Down to float32's smallest normal number (2^-126 of the largest weight) an infinity reaches the
    output, whether the heavier keys come after it or before; large finite values keep their size."""
    far = [20.0, 60.0, 100.0, 104.0, 112.0, 120.0, 125.0]                # log2 of the weight, negated
    lens, d = [200] * len(far), 64
    c = widened(base.filled(207, lens, 1, d, "bf16"), width)
    q = torch.zeros(len(far), 2, d, device="cuda")
    q[:, :, 0] = 1.0
    rows = (3, 190)
    for b, x in enumerate(far):
        page, at = c.at(b, range(200))
        c.k[page, :, at] = 0.0
        for row in rows:
            put_values(c, b, row, c.k, {0: -round(x * np.log(2) * 4) / 4})
        put_values(c, b, rows[0], c.v, {1: INF, 2: 2.0 ** 100})
        put_values(c, b, rows[1], c.v, {1: INF, 3: -INF, 4: 2.0 ** 100})
    out, lse, status = base.run_decode(c, q.to(BF16), lens, scale=1.0)
    assert status == [0] * len(far)
    assert bool(torch.isposinf(out[:, :, 1]).all()) and bool(torch.isneginf(out[:, :, 3]).all())
    for b, x in enumerate(far):
        k, v = c.rows(b, 200)
        v = np.where(np.isfinite(v), v, 0.0)
        want, wl, tol, ltol = base.decode_tolerance(base.f64(q[b].to(BF16)), k, v, 1.0, "bf16")
        cols = [i for i in range(d) if i not in (1, 3)]
        if x > 100:                                       # the smallest bf16 number, 2^-133, beside 2^100
            tol = tol + 2.0 ** -33
        assert np.all(np.abs(base.f64(out[b]) - want)[:, cols] <= tol[:, cols])
        assert np.all(np.abs(base.f64(lse[b]) - wl) <= ltol)


# ---------------------------------------------------------------- one-token attention: weights over 8-bit values


def weight_bound(c, q, b, n, scale, part):
    """Bound of the output's error from the kernel's roundings, `part` being that of a weight: the
    weights p_j vs_j are f16 numbers over a reference that keeps the largest at 2^7 or above, so that
    half of f16's smallest step, 2^-25, is 2^-32 of it."""
    k, v = c.rows(b, n)
    vs = c.value_scales(b, n)
    want, lse, absv, big = base.decode_attention_ref(base.f64(q[b]), k, v, scale)
    d, group = q.shape[2], q.shape[1] // k.shape[1]
    # score and exponent as in base.decode_tolerance; log2 of the value's scale: 2^-22 of an exponent, of which
    # the sums with it keep 2^-24 of their size (at most 2^7)
    rel = part + 2 * ((d + 4) * 2.0 ** -24 * big + 2.0 ** -21) + 2 * n * 2.0 ** -24 + 2.0 ** -16
    tol = absv * rel[:, None] + base.HALF[BF16] * np.abs(want) + 1e-30
    for h in range(q.shape[1]):
        g = h // group
        p = np.exp(scale * (k[:, g] @ base.f64(q[b])[h]) - lse[h])
        tol[h] += 2.0 ** -32 * (p * vs[:, g]).max() * (np.abs(v[:, g]) / vs[:, g][:, None]).sum(0)
    return want, tol


@pytest.mark.parametrize("width", [1, 2400])
@pytest.mark.parametrize("group", [1, 4, 8, 12])
@pytest.mark.parametrize("held", ["e4m3", "int8"])
def test_many_light_rows_beside_a_heavy_one(held, group, width):
    """A column in which the heaviest row is 0 consists of rows of 2^-26 of its weight: they are not
    lost, before it or behind it."""
    n, d = 2500, 64
    for at in (5, 2400):
        c = widened(base.Cache(211, [n], 1, d, held), width)
        k = torch.zeros(n, 1, d, device="cuda")
        k[at, 0, 0] = 18.0                                # exp(18) = 2^25.97; exact in both formats
        v = torch.ones(n, 1, d, device="cuda")
        v[:, 0, ::2] = -0.5
        v[at, 0, 1:9] = 0.0
        c.put(0, k.to(BF16), v.to(BF16))
        q = torch.zeros(1, group, d, device="cuda", dtype=BF16)
        q[:, :, 0] = 1.0
        out, lse, status = base.run_decode(c, q, [n], scale=1.0)
        assert status == [0]
        want, tol = weight_bound(c, q, 0, n, 1.0, 2.0 ** -11)
        assert np.all(np.abs(base.f64(out[0]) - want) <= tol)
        assert np.all(tol[:, 1] < np.abs(want[:, 1]) / 8)           # the bound tells lost from kept
        assert np.abs(base.f64(out[0]))[:, 1:9].min() > 0


@pytest.mark.parametrize("width", [1, 2400])
@pytest.mark.parametrize("hq,hkv,d", [(4, 4, 64), (8, 2, 128), (6, 2, 128), (4, 1, 64)])
@pytest.mark.parametrize("held", ["e4m3", "int8"])
def test_weights_of_up_to_four_queries_keep_22_bits(held, hq, hkv, d, width):
    """Two keys whose values nearly cancel: the weights' own roundings are what is left. Keys 0 and 1
    have the values 1 and -1 times 1.75, weights p and 1 - p around a half."""
    cases = 64
    c = widened(base.Cache(213, [2] * cases, hkv, d, held), width)
    q = torch.zeros(cases, hq, d, device="cuda")
    k = torch.zeros(2, hkv, d, device="cuda")
    k[0, :, 0] = 1.0
    v = torch.full((2, hkv, d), 1.75, device="cuda")
    v[1] = -1.75
    for b in range(cases):
        c.put(b, k.to(BF16), v.to(BF16))
        q[b, :, 0] = (b - 32) * 2.0 ** -12 + 2.0 ** -13 * torch.arange(hq, device="cuda")
    q = q.to(BF16)
    out, lse, status = base.run_decode(c, q, [2] * cases, scale=1.0)
    assert status == [0] * cases
    for b in range(cases):
        kk, vv = c.rows(b, 2)
        want, _, absv, _ = base.decode_attention_ref(base.f64(q[b]), kk, vv, 1.0)
        # scores below 2^-6: products and factors of 2^-24 of that, exponents and the base-2 logarithm 2^-22 each,
        # sums 2^-24, the two parts 2^-22
        tol = absv * (8 * 2.0 ** -22) + base.HALF[BF16] * np.abs(want)
        assert np.all(np.abs(base.f64(out[b]) - want) <= tol), b


# ---------------------------------------------------------------- append: offsets that run backwards


def claims(cu, rows, start):
    """Which requests' offsets are refused, by the header's words."""
    bad = []
    for b in range(len(cu) - 1):
        n = cu[b + 1] - cu[b]
        over = n < 0 or (n > 0 and b > 0 and cu[b] < max(cu[:b]))
        bad.append(over or (n > 0 and (cu[b] < 0 or cu[b + 1] > rows or start[b] < 0)))
    return bad


@pytest.mark.parametrize("held", ["e4m3", "int8"])
@pytest.mark.parametrize("cu,rows", [
    ([0, 5, 3, 8], 8),                      # the second ends before it begins, the third begins inside the first
    ([0, 8, 4, 12], 12),
    ([0, 4, 0, 4], 4),                      # two begin at the same row
    ([4, 0, 4, 8], 8),
    ([0, 6, 2, 2, 6, 9], 9),                # an empty one among those that overlap has nothing to object to
    ([2, 5, 9, 7], 12),                     # the last alone; rows before the first offset are nobody's
    ([0, 3, 2 ** 31 - 1, 3, 6], 6),
    ([0, 3, -2 ** 31, 3, 6], 6),
    ([0, 700, 350, 1000], 1000),            # over many thread blocks
])
def test_append_offsets_that_run_backwards(cu, rows, held):
    n = len(cu) - 1
    start = [3 + 5 * b for b in range(n)]
    # room for what is written, and for the most that an overlapping request could ask for
    c = base.Cache(221, [start[b] + min(max(cu[b + 1] - cu[b], 1), rows) for b in range(n)], 2, 64, held)
    k, v = base.fresh(222, rows, 2, 64)
    before = [t.clone() for t in (c.k, c.v, c.ks, c.vs)]
    bad = claims(cu, rows, start)
    assert base.run_append(c, k, v, cu, start) == [int(x) for x in bad]
    base.check_append(c, before, k, v, cu, start, [b for b in range(n) if not bad[b] and cu[b + 1] > cu[b]])


def test_append_many_offsets_some_of_which_run_backwards():
    """More requests than a thread block has threads; flagged ones keep their status."""
    rng = np.random.default_rng(223)
    lens = rng.integers(0, 5, 700)
    cu = [0] + np.cumsum(lens).tolist()
    rows = cu[-1]
    for b in (40, 41, 300, 555):
        cu[b] = max(0, cu[b] - int(rng.integers(5, 200)))
    start = rng.integers(0, 40, 700).tolist()
    c = base.Cache(224, [s + max(cu[b + 1] - cu[b], 1) for b, s in enumerate(start)], 1, 64, "int8")
    k, v = base.fresh(225, rows, 1, 64)
    before = [t.clone() for t in (c.k, c.v, c.ks, c.vs)]
    bad = claims(cu, rows, start)
    assert 4 <= sum(bad) < 200          # each lowered offset spoils the request before it, or its own
    status = [0] * 700
    status[bad.index(True)], status[0] = 4, 2
    want = [int(x) if s == 0 else s for x, s in zip(bad, status)]
    assert base.run_append(c, k, v, cu, start, base.i32(status)) == want
    base.check_append(c, before, k, v, cu, start, [b for b in range(700) if want[b] == 0 and cu[b + 1] > cu[b]])


# ---------------------------------------------------------------- rotary positions: angles


def two_pi_fraction(n):
    """floor(2^n / 2 pi), pi from Machin's 16 arctan(1/5) - 4 arctan(1/239) in integers."""
    def arctan_of_one_over(x):
        term = total = (1 << (n + 64)) // x
        k, sign = 1, -1
        while term:
            term //= x * x
            k += 2
            total += sign * (term // k)
            sign = -sign
        return total
    pi = (16 * arctan_of_one_over(5) - 4 * arctan_of_one_over(239)) >> 64
    return (1 << 2 * n) // (2 * pi)


def turned(positions, inv_freq):
    """cos and sin of position * inv_freq, reduced by whole turns in integers ([rows][pairs])."""
    n = 640                                               # bits behind the point: 2^-640 * 2^31 * 2^128 is far below
    unit = two_pi_fraction(n)
    cos, sin = np.empty((len(positions), len(inv_freq))), np.empty((len(positions), len(inv_freq)))
    for i, f in enumerate(inv_freq):
        num, den = float(f).as_integer_ratio()            # a power of two below, 2^149 at the most
        for r, p in enumerate(positions):
            turns = ((p * num * unit << 160) // den) % (1 << (n + 160))
            angle = (turns >> (n + 160 - 80)) / 2.0 ** 80 * 2 * np.pi
            cos[r, i], sin[r, i] = np.cos(angle), np.sin(angle)
    return cos, sin


FREQS = [1e-45, 1.2e-38, 3e-20, 1e-6, 0.00133, 0.31, 1.0, 3.99, 7.9999995, 8.0, 9.25, 100.7, 1030.3, 65537.0, 1e6, 33554430.0,
         33554432.0, 2.5e9, 2.0 ** 40 + 2.0 ** 20, 1.5e19, 1e24, 3.3e30, 1e38, 3.4028234e38]


@pytest.mark.parametrize("style", [0, 1])
@pytest.mark.parametrize("negative", [False, True])
def test_angles_of_every_size(style, negative):
    """Frequencies over all of float32 and positions over all of int32, against angles reduced in
    integers (a float64 product would itself be off by 2^-22 rad at 2^31)."""
    positions = [0, 1, 2, 3, 7, 1000, 4097, 123457, 2 ** 20 + 1, 10 ** 8 + 7, 2 ** 30, 2 ** 31 - 1, -1, -2, -77, -65536, -2 ** 31 + 1, -2 ** 31]
    freqs = np.array(FREQS, np.float32) * np.float32(-1.0 if negative else 1.0)
    rows, pairs = len(positions), len(freqs)
    q = torch.randn(rows, 2, 2 * pairs, generator=base.gen(231), device="cuda")
    x, out = base.f64(q), torch.empty_like(q)
    tv.rope_axes(tv.rope_axes_geom(2, 0, 2 * pairs, [pairs], style), q, None, base.i32([positions]),
                 torch.from_numpy(freqs).cuda(), out, None)
    cos, sin = turned(positions, freqs)
    a, b = (x[..., :pairs], x[..., pairs:]) if style else (x[..., 0::2], x[..., 1::2])
    ra, rb = a * cos[:, None] - b * sin[:, None], b * cos[:, None] + a * sin[:, None]
    # The angle: 2^31 * 2^-63 + 2 * 2^-32 turns = 3 * 2^-32 turns, 2 pi times that in rad. The remainder as a
    # float and times 2 pi 2^-32 (a constant of 24 bits): 3 roundings, 3 * 2^-24 of at most pi / 4. The series:
    # 2^-29 left out, the last sum's rounding 2^-25, those inside it 2^-24 of z / 2 < 0.31 or less each, three that
    # matter. A product each and the sum: 3 * 2^-24 of |a| + |b| at the most.
    angle = 2 * np.pi * 3 * 2.0 ** -32 + 3 * 2.0 ** -24 * np.pi / 4
    tol = (np.abs(a) + np.abs(b)) * (angle + 2.0 ** -29 + 2.0 ** -25 + 3 * 0.31 * 2.0 ** -24 + 3 * 2.0 ** -24)
    got = base.f64(out)
    ga, gb = (got[..., :pairs], got[..., pairs:]) if style else (got[..., 0::2], got[..., 1::2])
    worst = max((np.abs(ga - ra) / tol).max(), (np.abs(gb - rb) / tol).max())
    assert worst <= 1, (worst, [FREQS[i] for i in np.unique(np.nonzero(np.abs(ga - ra) > tol)[2])])


@pytest.mark.parametrize("rows", [2 ** 31 - 1, 2 ** 31 - 2049])
def test_the_most_rows(rows):
    """Row counts up to int32's largest (8.6 GB of queries and of positions)."""
    pos = torch.arange(rows, dtype=I32, device="cuda")
    q = torch.ones(rows, 1, 2, dtype=BF16, device="cuda")
    q[..., 1] = 0.5
    inv = torch.tensor([0.25], device="cuda")
    tv.rope_axes(tv.rope_axes_geom(1, 0, 2, [1], 0), q, None, pos[None], inv, q, None)
    at = torch.cat([torch.arange(5000), torch.arange(rows - 5000, rows), torch.randint(0, rows, (200000,))]).cuda()
    angle = at.double() * 0.25
    want = torch.stack([angle.cos() - 0.5 * angle.sin(), 0.5 * angle.cos() + angle.sin()], 1)
    # the float64 angle is exact (a power of two times an integer); bf16's rounding and float32's, as above
    assert bool(((q[at, 0].double() - want).abs() <= base.HALF[BF16] * want.abs() + 1.5 * 8 * 2.0 ** -24).all())


# ---------------------------------------------------------------- one-token attention: more units than thread blocks


def ragged_batch(seed, batch, longest, rng):
    lens = np.exp(rng.uniform(0, np.log(longest), batch)).astype(int).tolist()
    lens[0], lens[1], lens[2], lens[-1] = 0, 1, longest, 0
    return lens


@pytest.mark.parametrize("held", ["bf16", "e4m3", "int8"])
@pytest.mark.parametrize("batch,hkv,group,d,longest", [
    (1500, 1, 3, 64, 40),
    (100, 8, 4, 128, 700),
    (100, 8, 8, 64, 400),
    (90, 8, 5, 128, 300),
    (60, 12, 11, 128, 250),
    (700, 1, 16, 64, 90),
])
def test_more_units_than_blocks_in_two_launches(batch, hkv, group, d, longest, held):
    """Tables wide enough for two launches, and more (request, head) units than thread blocks, whose
    records then go by block: empty, tiny and longer requests, a flagged one and one with a missing
    page, in a unit that two blocks share."""
    rng = np.random.default_rng(241)
    lens = ragged_batch(242, batch, longest, rng)
    c = widened(base.filled(243, lens, hkv, d, held), 2400)
    q = torch.randn(batch, group * hkv, d, generator=base.gen(244), device="cuda").to(BF16)
    assert batch * hkv > 4 * torch.cuda.get_device_properties(0).multi_processor_count
    status = [0] * batch
    missing, flagged = 2, batch // 2                      # the longest one lacks its last page but one
    lens[flagged] = max(lens[flagged], 1)
    status[flagged] = 16
    page = max((lens[missing] - 1) // 16 - 1, 0)
    good = int(c.table[missing, page])
    some = sorted(set(rng.choice(batch, 20).tolist() + [0, 1, batch - 1]) - {missing, flagged})
    for bad in (good, -1, c.pool):
        c.table[missing, page] = bad
        out, lse, got = base.run_decode(c, q, lens, base.i32(status))
        want = list(status)
        if bad != good:
            want[missing] = 8
        assert got == want
        for b in range(batch):
            if want[b]:
                assert bool((out[b] == 9.0).all()) and bool((lse[b] == 9.0).all())
        base.check_decode(c, q, lens, out, lse, which=some + ([missing] if bad == good else []))
    again = base.run_decode(c, q, lens, base.i32(status))
    assert np.array_equal(base.bits(out), base.bits(again[0])) and np.array_equal(base.bits(lse), base.bits(again[1]))


def test_every_request_of_a_batch_in_two_launches():
    """All of 1500 requests checked against float32 arithmetic on the same GPU, not a sample of them."""
    rng = np.random.default_rng(245)
    lens = ragged_batch(246, 1500, 300, rng)
    c = widened(base.filled(247, lens, 1, 64, "bf16"), 2400)
    q = torch.randn(1500, 2, 64, generator=base.gen(248), device="cuda").to(BF16)
    out, lse, status = base.run_decode(c, q, lens)
    assert status == [0] * 1500
    page = c.table.long()[:, :19].clamp(min=0)
    seen = torch.arange(19 * 16, device="cuda") < torch.tensor(lens, device="cuda")[:, None]
    k = c.k[page].double().permute(0, 2, 1, 3, 4).reshape(1500, 304, 64)
    v = torch.where(seen[..., None], c.v[page].double().permute(0, 2, 1, 3, 4).reshape(1500, 304, 64), 0.0)
    score = torch.where(seen[:, None], torch.einsum("bhd,bnd->bhn", q.double(), torch.where(seen[..., None], k, 0.0)) / 8, -INF)
    want_lse = torch.logsumexp(score, -1)
    p = torch.where(seen[:, None], torch.exp(score - torch.where(want_lse > -INF, want_lse, 0.0)[..., None]), 0.0)
    want = p @ v
    # as base.decode_tolerance
    big = torch.einsum("bhd,bnd->bhn", q.double().abs(), torch.where(seen[..., None], k, 0.0).abs()).amax(-1, keepdim=True) / 8
    rel = 2.0 ** -16 + 2 * (68 * 2.0 ** -24 * big + 2.0 ** -21) + 2 * 300 * 2.0 ** -24
    tol = rel * (p @ v.abs()) + base.HALF[BF16] * want.abs() + 1e-30
    assert bool(((out.double() - want).abs() <= tol).all())
    fin = want_lse > -INF
    assert bool(((lse.double() - want_lse).abs() <= rel[..., 0] + 2.0 ** -22 * want_lse.abs())[fin].all()) and bool(torch.isneginf(lse[~fin]).all())


# ---------------------------------------------------------------- the measured cases


def measured():
    spec = importlib.util.spec_from_file_location("operators", os.path.join(ROOT, "perf", "operators.py"))
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def largest(t):
    return float(t.double().nan_to_num(0.0).abs().max()) if t.numel() else 0.0


def close_to_exact(m, case, seed):
    """Both forms of a measured case against its definition in 64 bits and against each other."""
    exact = m.exact(case, seed)
    got = {}
    for own in (False, True):
        m.own = own
        state = m.prepare(case, seed)
        got[own] = {k: t.clone() for k, t in m.run(state).items()}
        for name, want in exact.items():
            if want is None:
                continue
            x = got[own][name]
            if case["op"] == "decode":
                s = state
                scale = [1.0 if t is None else largest(t) for t in (s["ks"], s["vs"])]
                v = largest(s["v"]) * scale[1]
                score = 132 * 2.0 ** -24 * (largest(s["q"]) * largest(s["k"]) * scale[0] * case["d"] ** 0.5) + 2.0 ** -21
                err = 2.0 ** -11 + 2 * score + case["hi"] * 2.0 ** -23
                tol = base.HALF[BF16] * want.abs() + err * v if name == "out" else err + 2.0 ** -22 * want.abs()
            elif case["op"] == "rope":
                tol = base.HALF[x.dtype] * want.abs() + 2 * largest(state[name]) * 7 * 2.0 ** -24
            else:                                         # one rounding, of a scale to float32 or a value to bf16
                tol = base.HALF.get(x.dtype, 0.0) * want.abs()
            same = (x.double() == want) | ((x.double() - want).abs() <= tol)
            assert bool(same.all()), (case.get("name"), own, name)
    assert torch.equal(got[False].get("status", torch.zeros(1)), got[True].get("status", torch.zeros(1)))
    if case["op"] in ("append", "read"):
        for name in got[True]:
            assert torch.equal(got[False][name].view(torch.uint8), got[True][name].view(torch.uint8)), name


@pytest.mark.parametrize("name", ["rope-step", "rope-image", "append-step", "append-ragged", "read-step", "decode-short",
                                  "decode-wide"])
def test_measured_cases(name):
    m = measured()
    close_to_exact(m, next(c for c in m.listed() if c["name"] == name), 3)


def test_measured_cases_drawn():
    m = measured()
    rng, seen = random.Random(7), 0
    while seen < 8:
        case = m.draw(rng)
        work = m.work(case)
        if work["bytes"] < 3e7 and work["flops"] < 1e9:
            close_to_exact(m, case, seen)
            seen += 1


# ---------------------------------------------------------------- together with the tree step


@pytest.mark.parametrize("held", ["e4m3", "int8"])
def test_a_tree_step_over_an_8_bit_cache_and_back(held):
    """The cache read back, the tree step on the bf16 pools, its accepted rows gathered from them and
    appended, and the next token's attention over the 8-bit cache."""
    from gen import workloads as wl
    from speculative_decoding_tree_build_gb300.step import DeviceBatch
    w = wl.make_config(2, batch=3, prompt_scale=0.1)
    z = DeviceBatch(w)
    hq, hkv, d = w["num_q_heads"], w["num_kv_heads"], w["head_dim"]
    plen = [int(x) for x in w["prompt_len"]]
    depth = int(w["max_depth"])
    c = base.Cache(251, [n + depth + 1 for n in plen], hkv, d, held)
    cu = [0] + np.cumsum(plen).tolist()

    def gathered(first, counts):
        """Rows first[b].. of each request from the bf16 pools, [rows][Hkv][D]."""
        req = torch.repeat_interleave(torch.arange(len(counts), device="cuda"), torch.tensor(counts, device="cuda"))
        slot = torch.cat([torch.arange(f, f + n, device="cuda") for f, n in zip(first, counts)])
        page = z.block_table[req, slot // 16].long()
        return z.k_cache[page, :, slot % 16], z.v_cache[page, :, slot % 16]

    k, v = gathered([0] * 3, plen)
    assert base.run_append(c, k, v, cu, [0] * 3) == [0] * 3
    status = base.i32([0] * 3)
    tv.kv_quant_read(c.geom, None, base.i32(plen), c.table, c.n_blocks, c.k, c.v, c.ks, c.vs, z.block_table, z.n_blocks,
                     z.k_cache, z.v_cache, status)
    z.step()
    assert status.tolist() == z.status.tolist() == [0] * 3
    new = z.new_len.tolist()
    count = [b - a for a, b in zip(plen, new)]
    assert min(count) >= 1 and max(count) <= depth + 1
    k, v = gathered(plen, count)
    cu = [0] + np.cumsum(count).tolist()
    before = [t.clone() for t in (c.k, c.v, c.ks, c.vs)]
    assert base.run_append(c, k, v, cu, plen) == [0] * 3
    base.check_append(c, before, k, v, cu, plen, range(3))
    q = torch.randn(3, hq, d, generator=base.gen(252), device="cuda").to(BF16)
    out, lse, got = base.run_decode(c, q, new)
    assert got == [0] * 3
    base.check_decode(c, q, new, out, lse)
