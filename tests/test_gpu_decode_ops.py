"""The plain-decoding and 8-bit-cache calls on the GPU against their float64
restatement (oracle/decode_ref.py)."""

import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import speculative_decoding_tree_build_gb300 as tv
from oracle import decode_attention_ref, kv_quant_ref, rope_axes_ref

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
BF16, F32, I32 = torch.bfloat16, torch.float32, torch.int32
HALF = {BF16: 2.0 ** -8, F32: 2.0 ** -24}        # largest relative error of one rounding
HELD = {"bf16": BF16, "e4m3": torch.float8_e4m3fn, "int8": torch.int8}


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def f64(t):
    return t.double().cpu().numpy()


def i32(x):
    return torch.tensor(x, dtype=I32, device="cuda")


def bits(t):
    return t.view({1: torch.int8, 2: torch.int16, 4: torch.int32}[t.element_size()]).cpu().numpy()


# ---------------------------------------------------------------- rotary positions


def rope_case(seed, rows, hq, hkv, d, sections, style, order, dtype, far, pad=0, shift=0, negative=False):
    g = gen(seed)
    n = (hq + hkv) * d + pad
    flat = torch.randn(rows * n + shift, generator=g, device="cuda").to(dtype)[shift:]
    both = flat.view(rows, n)
    q = both[:, :hq * d].unflatten(1, (hq, d))
    k = both[:, hq * d:(hq + hkv) * d].unflatten(1, (hkv, d)) if hkv else None
    lo = -far if negative else 0
    pos = torch.randint(lo, far + 1, (len(sections), rows), generator=g, device="cuda").to(I32)
    pairs = sum(sections)
    inv = (10000.0 ** (-torch.arange(pairs, device="cuda", dtype=torch.float64) / pairs)).float()
    geom = tv.rope_axes_geom(hq, hkv, d, sections, style, order)
    return geom, q, k, pos, inv


def test_rope_axes_leaves_the_other_columns_alone():
    """Infinities and NaN behind the rotated columns pass through and touch nothing else."""
    for style in (0, 1):
        for pairs in (1, 3, 5, 13, 16):
            g, q, k, pos, inv = rope_case(17, 6, 2, 1, 40, [pairs], style, 0, BF16, 50)
            q = q.clone()
            q[:, :, 2 * pairs] = float("nan")
            q[:, :, -1] = float("inf")
            qo, ko = torch.empty_like(q), torch.empty(6, 1, 40, dtype=BF16, device="cuda")
            tv.rope_axes(g, q, k, pos, inv, qo, ko)
            assert np.array_equal(bits(qo[..., 2 * pairs:].contiguous()), bits(q[..., 2 * pairs:].contiguous()))
            assert bool(torch.isfinite(qo[..., :2 * pairs]).all())


def check_rope(x, out, pos, inv, sections, style, order):
    want = rope_axes_ref(f64(x), pos.cpu().numpy(), f64(inv), sections, style, order)
    got = f64(out)
    n = sum(sections)
    mag = np.zeros_like(want)
    xa = np.abs(f64(x))
    ia, ib = (np.arange(n), np.arange(n) + n) if style else (2 * np.arange(n), 2 * np.arange(n) + 1)
    mag[..., ia] = mag[..., ib] = xa[..., ia] + xa[..., ib]
    # angle: 2^-27 turns = 2 pi 2^-27 rad from the fraction's rounding; sincospif 2 units of 2^-24;
    # two products and a sum: 3 roundings; then the output's rounding
    tol = mag * (2 * np.pi * 2.0 ** -27 + 5 * 2.0 ** -24)
    if x.dtype == BF16:
        tol = tol + HALF[BF16] * np.abs(want)
    assert np.all(np.abs(got - want) <= tol)
    assert np.array_equal(got[..., 2 * n:], f64(x)[..., 2 * n:])


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("style", [0, 1])
@pytest.mark.parametrize("rows,hq,hkv,d,sections,order,pad,shift", [
    (1, 1, 1, 2, [1], 0, 0, 0),
    (5, 4, 2, 128, [16, 24, 24], 0, 0, 0),
    (67, 32, 8, 128, [24, 20, 20], 1, 1024, 0),
    (33, 3, 1, 80, [20, 20], 1, 0, 0),
    (7, 5, 5, 72, [18, 18], 0, 8, 0),
    (9, 2, 1, 64, [4, 3, 2, 1], 1, 0, 0),           # 44 columns pass through
    (6, 3, 1, 50, [9, 8, 8], 0, 3, 1),              # nothing aligned beyond an element
    (11, 4, 4, 512, [256], 0, 0, 0),
    (3, 130, 0, 96, [0, 40, 8], 0, 0, 0),           # no keys
    (4, 2, 2, 33, [7, 9], 1, 0, 0),                 # an odd head dimension
    (2500, 2, 1, 64, [16, 16], 0, 0, 0),            # many rows of few heads
    (2000, 10, 2, 72, [36], 0, 0, 0),
    (40, 19, 1, 80, [20, 7, 10], 1, 0, 0),          # 74 columns turn: a vector on both sides of their end
    (300, 3, 3, 32, [1], 0, 4, 2),                  # one pair, rows aligned to 4 bytes in bf16
    (5, 2, 2, 48, [11], 0, 2, 0),
])
def test_rope_axes(rows, hq, hkv, d, sections, order, pad, shift, style, dtype):
    g, q, k, pos, inv = rope_case(11, rows, hq, hkv, d, sections, style, order, dtype, 5000, pad, shift)
    qo = torch.full((rows, hq, d), 7.0, dtype=dtype, device="cuda")
    ko = torch.full((rows, hkv, d), 7.0, dtype=dtype, device="cuda") if hkv else None
    tv.rope_axes(g, q, k, pos, inv, qo, ko)
    check_rope(q, qo, pos, inv, sections, style, order)
    if hkv:
        check_rope(k, ko, pos, inv, sections, style, order)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("place", ["apart", "in place"])
@pytest.mark.parametrize("rows,d,pairs", [
    (3, 128, 1), (700, 64, 2), (5, 72, 4), (9, 128, 6), (600, 32, 9), (17, 80, 12), (40, 128, 46),
    (3, 256, 63), (9, 72, 36), (200, 96, 47), (4, 512, 254), (6, 512, 3),
])
def test_rope_axes_halves_of_any_length(rows, d, pairs, place, dtype):
    """The second half starts inside a vector, and the columns left alone may too."""
    g, q, k, pos, inv = rope_case(14, rows, 5, 2, d, [pairs], 1, 0, dtype, 5000, 64, 0, True)
    q0, k0 = q.clone(), k.clone()
    qo, ko = (q, k) if place == "in place" else (torch.full_like(q0, 7.0), torch.full_like(k0, 7.0))
    tv.rope_axes(g, q, k, pos, inv, qo, ko)
    check_rope(q0, qo, pos, inv, [pairs], 1, 0)
    check_rope(k0, ko, pos, inv, [pairs], 1, 0)


@pytest.mark.parametrize("style", [0, 1])
def test_rope_axes_far_negative_and_in_place(style):
    g, q, k, pos, inv = rope_case(12, 40, 4, 2, 64, [12, 10, 10], style, 1, F32, 2 ** 31 - 1, 64, 0, True)
    q0, k0 = q.clone(), k.clone()
    tv.rope_axes(g, q, k, pos, inv, q, k)           # each output is its own input
    # inv_freq / 2 pi in float64 and F's rounding: |position| * (2^-54 + 2^-65) turns at the most,
    # 2^31 * 2^-53 * 2 pi = 1.5e-6 rad on top of the usual bound
    for x, out in ((q0, q), (k0, k)):
        want = rope_axes_ref(f64(x), pos.cpu().numpy(), f64(inv), [12, 10, 10], style, 1)
        pair = np.abs(f64(x)).max() * 2
        assert np.abs(f64(out) - want).max() <= pair * (1.5e-6 + 1e-6)


def test_rope_axes_no_rows_and_other_stream():
    g, q, k, pos, inv = rope_case(13, 8, 4, 2, 64, [32], 1, 0, BF16, 100)
    tv.rope_axes(g, q[:0], k[:0], pos[:, :0], inv, torch.empty_like(q[:0]), torch.empty_like(k[:0]))
    qo, ko = torch.empty(8, 4, 64, dtype=BF16, device="cuda"), torch.empty(8, 2, 64, dtype=BF16, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    tv.rope_axes(g, q, k, pos, inv, qo, ko, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    check_rope(q, qo, pos, inv, [32], 1, 0)
    # one row of positions stands for all axes
    g3 = tv.rope_axes_geom(4, 2, 64, [10, 12, 10], 1, 1)
    tv.rope_axes(g3, q, k, pos.expand(3, -1), inv, qo, ko)
    check_rope(q, qo, pos.expand(3, -1), inv, [10, 12, 10], 1, 1)
    with pytest.raises(ValueError):
        tv.rope_axes(g, q, k, pos, inv[:-1], qo, ko)
    with pytest.raises(ValueError):
        tv.rope_axes(g, q.transpose(1, 2), k, pos, inv, qo, ko)
    with pytest.raises(ValueError):
        tv.rope_axes(g, q, k, pos.long(), inv, qo, ko)


# ---------------------------------------------------------------- the 8-bit cache


def table_for(seed, slots, spare=3, width=0):
    need = [-(-n // 16) for n in slots]
    pool = sum(need) + spare
    order = torch.randperm(pool, generator=gen(seed), device="cuda").to(I32)
    t = torch.full((len(slots), max(max(need), width, 1)), -1, dtype=I32, device="cuda")
    at = 0
    for b, n in enumerate(need):
        t[b, :n] = order[at:at + n]
        at += n
    return t, i32(need), pool


class Cache:
    """An 8-bit (or bf16) paged cache for sequences of up to `slots` rows."""

    def __init__(self, seed, slots, hkv, d, held, fill=0x5a):
        self.table, self.n_blocks, self.pool = table_for(seed, slots)
        self.hkv, self.d, self.held = hkv, d, held
        shape = (self.pool, hkv, 16, d)
        size = 2 if held == "bf16" else 1
        raw = torch.full((self.pool, hkv, 16, d * size), fill, dtype=torch.uint8, device="cuda")
        self.k = raw.view(HELD[held]).view(shape)
        self.v = raw.clone().view(HELD[held]).view(shape)
        self.ks = None if held == "bf16" else torch.full(shape[:3], -3.0, device="cuda")
        self.vs = None if held == "bf16" else torch.full(shape[:3], -3.0, device="cuda")
        self.geom = tv.geom(hkv, hkv, d)

    def at(self, b, slots):
        slots = torch.as_tensor(slots, device="cuda", dtype=torch.long)
        return self.table[b].long()[slots // 16], slots % 16

    def put(self, b, k, v):
        """Rows 0.. of request b, from bf16 [n][hkv][d] (quantised by the restatement)."""
        page, at = self.at(b, range(k.shape[0]))
        for x, pool, scales in ((k, self.k, self.ks), (v, self.v, self.vs)):
            if self.held == "bf16":
                pool[page, :, at] = x
                continue
            code, sc = kv_quant_ref(f64(x), self.held)
            code = torch.from_numpy(code).to("cuda")
            pool.view(torch.int8)[page, :, at] = code.to(HELD[self.held]).view(torch.int8)
            scales[page, :, at] = torch.from_numpy(sc).to("cuda")

    def rows(self, b, n):
        """(k, v) of slots [0, n) as float64 values."""
        page, at = self.at(b, range(n))
        out = []
        for pool, scales in ((self.k, self.ks), (self.v, self.vs)):
            x = pool.view(torch.int16 if self.held == "bf16" else torch.int8)[page, :, at]
            x = x.view(pool.dtype).double()
            if scales is not None:
                x = x * scales[page, :, at].double()[..., None]
            out.append(x.cpu().numpy())
        return out

    def value_scales(self, b, n):
        if self.vs is None:
            return None
        page, at = self.at(b, range(n))
        return f64(self.vs[page, :, at])


def fresh(seed, rows, hkv, d, pad=0):
    """Two bf16 row sets, slices of one matrix; a few rows are made difficult."""
    g = gen(seed)
    both = torch.randn(rows, 2 * hkv * d + pad, generator=g, device="cuda")
    both *= torch.exp2(torch.randint(-20, 20, (rows, 1), generator=g, device="cuda").float())
    both = both.to(BF16)
    return (both[:, :hkv * d].unflatten(1, (hkv, d)), both[:, hkv * d:2 * hkv * d].unflatten(1, (hkv, d)))


def run_append(c, k, v, cu, start, status=None):
    status = torch.zeros(len(start), dtype=I32, device="cuda") if status is None else status
    tv.kv_quant_append(c.geom, k, v, i32(cu), i32(start), c.table, c.n_blocks, c.k, c.v, c.ks, c.vs, status)
    return status.cpu().tolist()


def check_append(c, before, k, v, cu, start, wrote):
    want = [bits(t).copy() for t in before]
    for b in wrote:
        n = cu[b + 1] - cu[b]
        page, at = (t.cpu().numpy() for t in c.at(b, range(start[b], start[b] + n)))
        for x, codes, scales in ((k, want[0], want[2]), (v, want[1], want[3])):
            code, sc = kv_quant_ref(f64(x[cu[b]:cu[b + 1]]), c.held)
            code = torch.from_numpy(code).to(HELD[c.held]).view(torch.int8).numpy()
            codes[page, :, at] = code
            scales[page, :, at] = sc.view(np.int32)
    got = [bits(t) for t in (c.k, c.v, c.ks, c.vs)]
    for g, w, name in zip(got, want, ("k", "v", "k_scale", "v_scale")):
        assert np.array_equal(g, w), (name, int((g != w).sum()))


@pytest.mark.parametrize("held", ["e4m3", "int8"])
@pytest.mark.parametrize("hkv,d,lens,start,pad,tail", [
    (1, 64, [1], [0], 0, 0),
    (8, 128, [1] * 9, [0, 15, 16, 17, 31, 100, 7, 8, 160], 1024, 0),
    (2, 128, [0, 5, 0, 0, 33, 1, 0], [3, 14, 0, 9, 16, 0, 2], 0, 4),     # rows behind the last request
    (3, 64, [70, 1, 129], [5, 0, 250], 8, 0),
    (16, 128, [37, 2], [0, 11], 0, 1),
])
def test_append_matches_restatement_bit_for_bit(hkv, d, lens, start, pad, tail, held):
    cu = [0] + np.cumsum(lens).tolist()
    c = Cache(21, [s + n for s, n in zip(start, lens)], hkv, d, held)
    k, v = fresh(22, cu[-1] + tail, hkv, d, pad)
    before = [t.clone() for t in (c.k, c.v, c.ks, c.vs)]
    assert run_append(c, k, v, cu, start) == [0] * len(lens)
    check_append(c, before, k, v, cu, start, range(len(lens)))


@pytest.mark.parametrize("held", ["e4m3", "int8"])
def test_append_special_rows(held):
    d = 64
    rows = torch.zeros(14, 1, d)
    rows[1, 0, 3] = 2.0 ** -130                      # subnormal bf16 alone
    rows[2, 0] = 2.0 ** -101
    rows[3, 0, :] = 3.3e38                           # near the largest bf16
    rows[3, 0, 1] = 1e38
    rows[4, 0, 5] = float("nan")
    rows[5, 0, 6] = float("inf")
    rows[6, 0, 7] = -float("inf")
    rows[7, 0] = torch.linspace(-448, 448, d)
    rows[8, 0, 0], rows[8, 0, 1] = 1.5, 1.125        # 9 against 3 halves: an exact e4m3 tie
    rows[9, 0, 0], rows[9, 0, 1:] = 254.0, torch.arange(1, d).float()    # exact int8 ties at odd values
    rows[10, 0, 0], rows[10, 0, 1:] = 1.75, torch.arange(1, d) * 2.0 ** -9
    rows[11, 0, 0] = -1.7578125                      # just above 1.75
    rows[12, 0] = -0.0
    rows[13, 0, 2], rows[13, 0, 3] = float("nan"), float("inf")
    x = rows.to(BF16).cuda()
    c = Cache(23, [14], 1, d, held)
    before = [t.clone() for t in (c.k, c.v, c.ks, c.vs)]
    assert run_append(c, x, x.flip(0), [0, 14], [0]) == [0]
    # -0 keeps its sign in e4m3 and has none in int8; the values are equal
    got, want = [], []
    for codes, scales, src in ((c.k, c.ks, x), (c.v, c.vs, x.flip(0))):
        page, at = c.at(0, range(14))
        got.append((f64(codes.view(torch.int8)[page, :, at].view(codes.dtype)), scales[page, :, at].cpu().numpy()))
        want.append(kv_quant_ref(f64(src), held))
    for (gc, gs), (wc, wsc) in zip(got, want):
        assert np.array_equal(gc, wc)
        assert np.array_equal(np.isnan(gs), np.isnan(wsc))
        assert np.array_equal(gs[~np.isnan(gs)], wsc[~np.isnan(wsc)])
    assert before[0].shape == c.k.shape


@pytest.mark.parametrize("held", ["e4m3", "int8"])
def test_append_skips_and_flags(held):
    lens, start = [20, 3, 40, 2, 17, 6], [0, 14, 8, 5, 0, 2]
    cu = [0] + np.cumsum(lens).tolist()
    c = Cache(24, [s + n for s, n in zip(start, lens)], 2, 128, held)
    k, v = fresh(25, cu[-1], 2, 128)
    c.table[1, 1] = c.pool                           # past the pool, second block of the span
    c.table[2, 2] = -1                               # missing, third block
    c.n_blocks[4] = 1                                # the second block is not held
    bad_start = list(start)
    bad_start[3] = -1
    status = i32([0, 0, 0, 0, 0, 64])
    before = [t.clone() for t in (c.k, c.v, c.ks, c.vs)]
    assert run_append(c, k, v, cu, bad_start, status) == [0, 8, 8, 1, 8, 64]
    check_append(c, before, k, v, cu, start, [0])


def test_append_offsets_past_the_rows_are_flagged():
    c = Cache(26, [32, 32], 1, 64, "e4m3")
    k, v = fresh(27, 6, 1, 64)
    before = [t.clone() for t in (c.k, c.v, c.ks, c.vs)]
    assert run_append(c, k, v, [0, 4, 9], [0, 0]) == [0, 1]    # rows 4..8 of 6
    check_append(c, before, k, v, [0, 4, 9], [0, 0], [0])
    assert run_append(c, k, v, [0, 4, 4], [0, -1]) == [0, 0]   # no rows, nothing to object to
    c = Cache(26, [32, 32, 32], 1, 64, "e4m3")
    assert run_append(c, k, v, [0, 6, 6, 9], [0, 0, 0]) == [0, 0, 1]    # rows 6..8 of 6


@pytest.mark.parametrize("held,hkv,d", [("e4m3", 8, 128), ("int8", 3, 64), ("e4m3", 40, 64)])
def test_append_many_rows_with_bad_requests_among_them(held, hkv, d):
    """Requests that reach over many thread blocks, one of them with a missing block far from most
    of its rows; empty requests between; more requests than a thread block has threads."""
    rng = np.random.default_rng(29)
    lens = [700, 0, 1, 900] + rng.integers(0, 4, 300).tolist() + [0, 650]
    start = [5, 0, 30, 11] + rng.integers(0, 50, 300).tolist() + [3, 16]
    cu = [0] + np.cumsum(lens).tolist()
    c = Cache(30, [s + n for s, n in zip(start, lens)], hkv, d, held)
    c.table[3, 2] = -1                                # the second long request's rows 21 to 36
    k, v = fresh(31, cu[-1] + 3, hkv, d, 16)
    before = [t.clone() for t in (c.k, c.v, c.ks, c.vs)]
    want = [0] * len(lens)
    want[3] = 8
    assert run_append(c, k, v, cu, start) == want
    check_append(c, before, k, v, cu, start, [b for b in range(len(lens)) if b != 3])


@pytest.mark.parametrize("held", ["e4m3", "int8"])
def test_append_every_pair_of_significands(held):
    """Every bf16 significand under every largest one, at eight binary distances: all exact ties
    of the quotient, and the quotients nearest to one."""
    top = torch.arange(128, 256).float().repeat_interleave(8)
    x = torch.arange(128, 256).float()[None] * torch.exp2(-torch.arange(1, 9).float()).repeat(128)[:, None]
    x[:, 127] = top                                   # 255 gives way to the largest
    y = torch.arange(128, 256).float()[None] * torch.exp2(-torch.arange(1, 9).float()).repeat(128)[:, None]
    y[:, 0] = -top
    k, v = x.to(BF16).cuda()[:, None], y.to(BF16).cuda()[:, None]
    assert bool((k.float().cpu()[:, 0] == x).all())
    c = Cache(28, [1024], 1, 128, held)
    before = [t.clone() for t in (c.k, c.v, c.ks, c.vs)]
    assert run_append(c, k, v, [0, 1024], [0]) == [0]
    check_append(c, before, k, v, [0, 1024], [0], [0])


@pytest.mark.parametrize("held", ["e4m3", "int8"])
@pytest.mark.parametrize("hkv,d,first,last", [
    (1, 64, None, [1]),
    (8, 128, [0, 3, 16, 40], [40, 3, 33, 47]),       # nothing, a page's middle, a page's edge
    (2, 64, [5, 0, 0, 70], [4, 0, 16, 200]),         # an empty range, no slots
    (3, 128, None, [300, 0, 1]),
])
def test_read_back_bit_for_bit(hkv, d, first, last, held):
    c = Cache(31, [max(n, 1) for n in last], hkv, d, held)
    for b, n in enumerate(last):
        if n:
            k, v = fresh(40 + b, n, hkv, d)
            c.put(b, k, v)
    # one row that reads back as NaN
    page, at = c.at(0, [last[0] - 1])
    c.ks[page, :, at] = float("nan")
    table, nb, pool = table_for(32, [max(n, 1) for n in last], spare=2, width=40)
    ko = torch.full((pool, hkv, 16, d), 5.0, dtype=BF16, device="cuda")
    vo = ko.clone()
    status = torch.zeros(len(last), dtype=I32, device="cuda")
    tv.kv_quant_read(c.geom, None if first is None else i32(first), i32(last), c.table, c.n_blocks,
                     c.k, c.v, c.ks, c.vs, table, nb, ko, vo, status)
    assert status.cpu().tolist() == [0] * len(last)
    for out, codes, scales in ((ko, c.k, c.ks), (vo, c.v, c.vs)):
        want = torch.full_like(out, 5.0)
        for b, n in enumerate(last):
            lo = first[b] if first else 0
            if n <= lo:
                continue
            page, at = c.at(b, range(lo, n))
            slots = torch.arange(lo, n, device="cuda")
            x = codes.view(torch.int8)[page, :, at].view(codes.dtype).float() * scales[page, :, at][..., None]
            want[table[b].long()[slots // 16], :, slots % 16] = x.to(BF16)
        same = (bits(out) == bits(want)) | (torch.isnan(out) & torch.isnan(want)).cpu().numpy()
        assert same.all()


def test_read_back_skips_and_flags():
    lens = [20, 33, 5, 17, 9]
    c = Cache(33, lens, 2, 64, "int8")
    for b, n in enumerate(lens):
        c.put(b, *fresh(50 + b, n, 2, 64))
    table, nb, pool = table_for(34, lens)
    c.table[0, 1] = -1
    table[1, 2] = pool
    nb[3] = 1
    status = i32([0, 0, 2, 0, 0])
    ko = torch.full((pool, 2, 16, 64), 5.0, dtype=BF16, device="cuda")
    vo = ko.clone()
    tv.kv_quant_read(c.geom, i32([0, 0, 0, 0, -1]), i32(lens), c.table, c.n_blocks, c.k, c.v, c.ks,
                     c.vs, table, nb, ko, vo, status)
    assert status.cpu().tolist() == [8, 8, 2, 8, 1]
    assert bool((ko == 5.0).all()) and bool((vo == 5.0).all())


# ---------------------------------------------------------------- one-token attention


def decode_tolerance(q, k, v, scale, held, vs=None):
    """Element-wise bounds of the output and of lse from the kernel's roundings
    (vs: the value rows' scales [n][Hkv])."""
    out, lse, absv, big = decode_attention_ref(q, k, v, scale)
    d, n = q.shape[1], k.shape[0]
    # a score: D products and sums in float32, the scale factors, 2^-24 each; exp2: 2^-22; the
    # terms that one lane adds up, at most n, 2^-24 each
    score = (d + 4) * 2.0 ** -24 * big + 2.0 ** -21
    sums = max(n, 1) * 2.0 ** -24
    weight = 2.0 ** -16 if held == "bf16" else 2.0 ** -11           # weights as two bf16 parts, or f16
    rel = weight + 2 * score + 2 * sums
    tol = absv * rel[:, None] + HALF[BF16] * np.abs(out) + 1e-30
    if held != "bf16" and n:
        # The weights p_j vs_j are f16 numbers over a common power 2^M <= max_j p_j vs_j, and f16's
        # smallest step is 2^-24: each is off by up to 2^-25 2^M besides its relative 2^-11, and
        # multiplies the code |v_j| / vs_j. Where the heaviest row's code is 0, all that a column
        # holds can lie below that step.
        for h in range(q.shape[0]):
            g = h // (q.shape[0] // k.shape[1])
            p = np.exp(scale * (k[:, g] @ q[h]) - lse[h])
            tol[h] += 2.0 ** -25 * (p * vs[:, g]).max() * (np.abs(v[:, g]) / vs[:, g][:, None]).sum(0)
    return out, lse, tol, score + sums + 2.0 ** -22 * np.abs(np.where(np.isfinite(lse), lse, 0))


def run_decode(c, q, lens, status=None, with_lse=True, scale=0.0, stream=None):
    batch, hq, d = q.shape
    g = tv.geom(hq, c.hkv, d, softmax_scale=scale)
    out = torch.full((batch, hq, d), 9.0, dtype=BF16, device="cuda")
    lse = torch.full((batch, hq), 9.0, device="cuda") if with_lse else None
    status = torch.zeros(batch, dtype=I32, device="cuda") if status is None else status
    ws = torch.full((tv.decode_workspace_bytes(g, batch),), 0xff, dtype=torch.uint8, device="cuda")
    tv.decode_attention(g, q, i32(lens), c.table, c.n_blocks, c.k, c.v, c.ks, c.vs, out, lse, ws, status,
                        stream)
    return out, lse, status.cpu().tolist()


def check_decode(c, q, lens, out, lse, scale=0.0, which=None):
    scale = scale or q.shape[2] ** -0.5
    for b in (range(len(lens)) if which is None else which):
        k, v = c.rows(b, lens[b])
        want, wl, tol, ltol = decode_tolerance(f64(q[b]), k, v, scale, c.held, c.value_scales(b, lens[b]))
        err = np.abs(f64(out[b]) - want)
        assert np.all(err <= tol), (b, lens[b], float((err - tol).max()))
        if lse is not None:
            got = f64(lse[b])
            if lens[b] == 0:
                assert np.isneginf(got).all()
            else:
                assert np.all(np.abs(got - wl) <= ltol), (b, lens[b], np.abs(got - wl).max())


def filled(seed, lens, hkv, d, held, spread=1.0):
    c = Cache(seed, [max(n, 1) for n in lens], hkv, d, held, fill=0xff)      # what is not written is NaN
    if c.ks is not None:
        c.ks.fill_(float("nan"))
        c.vs.fill_(float("nan"))
    if held == "int8":
        c.k.fill_(-128)
        c.v.fill_(127)
    g = gen(seed + 1)
    for b, n in enumerate(lens):
        if n:
            k = torch.randn(n, hkv, d, generator=g, device="cuda") * spread
            c.put(b, k.to(BF16), torch.randn(n, hkv, d, generator=g, device="cuda").to(BF16))
    return c


@pytest.mark.parametrize("held", ["bf16", "e4m3", "int8"])
@pytest.mark.parametrize("hq,hkv,d,lens", [
    (1, 1, 64, [1]),
    (4, 4, 128, [0, 1, 2, 15, 16, 17, 31, 32, 33]),
    (32, 8, 128, [63, 64, 65, 127, 128, 129, 0, 500]),
    (16, 2, 64, [255, 256, 257, 1000, 3]),
    (6, 2, 128, [700, 1, 47]),
    (32, 2, 128, [900, 16, 0, 333]),                # sixteen query heads to a cached head
    (9, 1, 64, [5, 77, 2100]),
    (24, 2, 128, [1031]),
])
def test_decode_attention(hq, hkv, d, lens, held):
    c = filled(61, lens, hkv, d, held)
    q = torch.randn(len(lens), hq * d + 8, generator=gen(62), device="cuda").to(BF16)
    q = q[:, :hq * d].unflatten(1, (hq, d))         # rows further apart than their heads
    out, lse, status = run_decode(c, q, lens)
    assert status == [0] * len(lens)
    check_decode(c, q, lens, out, lse)
    again, lse2, _ = run_decode(c, q, lens)
    assert np.array_equal(bits(out), bits(again)) and np.array_equal(bits(lse), bits(lse2))
    alone, none, _ = run_decode(c, q, lens, with_lse=False)
    assert none is None and np.array_equal(bits(out), bits(alone))
    # a block table with room for long requests takes the other way of cutting and joining
    wide = torch.full((len(lens), 2400), -1, dtype=I32, device="cuda")
    wide[:, :c.table.shape[1]] = c.table
    c.table = wide
    out, lse, status = run_decode(c, q, lens)
    assert status == [0] * len(lens)
    check_decode(c, q, lens, out, lse)


@pytest.mark.parametrize("held", ["bf16", "e4m3", "int8"])
def test_decode_attention_split_over_one_long_cache(held):
    lens = [20011, 4]
    c = filled(63, lens, 2, 64, held)
    q = torch.randn(2, 8, 64, generator=gen(64), device="cuda").to(BF16)
    out, lse, status = run_decode(c, q, lens)
    assert status == [0, 0]
    check_decode(c, q, lens, out, lse)


@pytest.mark.parametrize("held", ["bf16", "e4m3", "int8"])
def test_decode_attention_peaked_scores_and_scale(held):
    lens = [300, 41]
    c = filled(65, lens, 2, 128, held, spread=30.0)
    q = torch.randn(2, 8, 128, generator=gen(66), device="cuda") * 100
    q = q.to(BF16)
    out, lse, _ = run_decode(c, q, lens, scale=0.25)
    check_decode(c, q, lens, out, lse, scale=0.25)


@pytest.mark.parametrize("held", ["bf16", "e4m3", "int8"])
def test_decode_attention_query_of_any_size(held):
    """Queries near bf16's largest and smallest numbers, with a scale that keeps the scores small."""
    lens = [50, 50]
    c = filled(67, lens, 1, 64, held)
    q = torch.randn(2, 4, 64, generator=gen(68), device="cuda")
    big = (q * torch.tensor([2.0 ** 100, 2.0 ** 60], device="cuda")[:, None, None]).to(BF16)
    big[1, 2] = 0.0
    out, lse, _ = run_decode(c, big, lens, scale=2.0 ** -100)
    check_decode(c, big, lens, out, lse, scale=2.0 ** -100)


@pytest.mark.parametrize("held", ["e4m3", "int8"])
def test_decode_attention_row_scales_of_every_size(held):
    lens = [120, 64]
    c = Cache(69, lens, 1, 64, held)
    g = gen(70)
    for b, n in enumerate(lens):
        k = torch.randn(n, 1, 64, generator=g, device="cuda")
        v = torch.randn(n, 1, 64, generator=g, device="cuda")
        v *= torch.exp2(torch.randint(-90, 90, (n, 1, 1), generator=g, device="cuda").float()) if b else 0.0
        c.put(b, k.to(BF16), v.to(BF16))
    q = torch.randn(2, 2, 64, generator=g, device="cuda").to(BF16)
    out, lse, _ = run_decode(c, q, lens)
    check_decode(c, q, lens, out, lse)


@pytest.mark.parametrize("hkv,lens", [(1, [1900, 33, 900]), (2, [500, 0, 1, 129]), (16, [300, 200])])
@pytest.mark.parametrize("held", ["bf16", "e4m3", "int8"])
def test_decode_attention_bad_page_in_a_short_table(hkv, lens, held):
    """One request of a short table lacks a page that one of the blocks of a cluster alone reads."""
    c = filled(99, lens, hkv, 128, held)
    q = torch.randn(len(lens), 4 * hkv, 128, generator=gen(100), device="cuda").to(BF16)
    page = (lens[0] - 1) // 16 - 1
    good = int(c.table[0, page])
    for bad in (-1, c.pool, 2 ** 31 - 1):
        c.table[0, page] = bad
        out, lse, st = run_decode(c, q, lens)
        assert st == [8] + [0] * (len(lens) - 1)
        assert bool((out[0] == 9.0).all()) and bool((lse[0] == 9.0).all())
        check_decode(c, q, lens, out, lse, which=range(1, len(lens)))
    c.table[0, page] = good
    out, lse, st = run_decode(c, q, lens)
    assert st == [0] * len(lens)
    check_decode(c, q, lens, out, lse)


@pytest.mark.parametrize("held", ["bf16", "e4m3", "int8"])
@pytest.mark.parametrize("group,d", [(3, 64), (8, 128), (13, 128)])
@pytest.mark.parametrize("pages", [4, 5, 9, 13, 25, 49, 97, 300, 400])
def test_decode_attention_warps_of_a_request(pages, group, d, held):
    """Tables of one length after the other at which a request gets more warps, blocks and launches."""
    lens = [16 * pages - 3, 1, 16 * (pages // 2) + 1]
    c = filled(103, lens, 1, d, held)
    q = torch.randn(3, group, d, generator=gen(104), device="cuda").to(BF16)
    out, lse, st = run_decode(c, q, lens)
    assert st == [0, 0, 0]
    check_decode(c, q, lens, out, lse)
    c.table[2, pages // 2] = -1
    out, lse, st = run_decode(c, q, lens, i32([0, 2, 0]))
    assert st == [0, 2, 8]
    check_decode(c, q, lens, out, lse, which=[0])
    assert bool((out[1:] == 9.0).all()) and bool((lse[1:] == 9.0).all())


@pytest.mark.parametrize("width", [3, 2400])
def test_decode_attention_shared_pages_skips_and_flags(width):
    lens = [40, 40, 33, 20, 18, 9]
    c = filled(71, lens, 2, 128, "e4m3")
    c.table = torch.cat([c.table, torch.full((6, width), -1, dtype=I32, device="cuda")], 1)[:, :max(width, 3)].contiguous()
    c.table[1] = c.table[0]                          # two requests read the same pages
    c.table[2, 1] = c.pool
    c.n_blocks[3] = 1
    q = torch.randn(6, 8, 128, generator=gen(72), device="cuda").to(BF16)
    status = i32([0, 0, 0, 0, 0, 4])
    run = [40, 40, 33, 20, -1, 9]
    out, lse, st = run_decode(c, q, run, status)
    assert st == [0, 0, 8, 8, 1, 4]
    # a flagged request is not looked at again, whatever else is wrong with it
    assert run_decode(c, q, [40, 40, 33, 20, -1, -9], i32([0, 0, 2, 2, 2, 2]))[2] == [0, 0, 2, 2, 2, 2]
    check_decode(c, q, run, out, lse, which=[0, 1])
    assert bool((out[2:] == 9.0).all()) and bool((lse[2:] == 9.0).all())


@pytest.mark.parametrize("held", ["bf16", "int8"])
def test_decode_attention_missing_page_deep_in_a_long_cache(held):
    lens = [9000, 700]
    c = filled(73, lens, 4, 64, held)
    c.table[0, 400] = -1
    q = torch.randn(2, 8, 64, generator=gen(74), device="cuda").to(BF16)
    out, lse, st = run_decode(c, q, lens)
    assert st == [8, 0]
    assert bool((out[0] == 9.0).all()) and bool((lse[0] == 9.0).all())
    check_decode(c, q, lens, out, lse, which=[1])


def test_decode_attention_many_requests():
    rng = np.random.default_rng(75)
    lens = rng.integers(0, 40, 1500).tolist()
    c = filled(76, lens, 1, 64, "bf16")
    q = torch.randn(1500, 2, 64, generator=gen(77), device="cuda").to(BF16)
    out, lse, st = run_decode(c, q, lens)
    assert st == [0] * 1500
    check_decode(c, q, lens, out, lse, which=rng.choice(1500, 60, replace=False).tolist() + [0, 1499])


def test_offsets_past_32_bits():
    """Pools of more than 2^32 bytes, used at their far end by every call."""
    d, hkv = 128, 8
    blocks = (1 << 32) // (hkv * 16 * d) + 40        # 4.3 GB of codes, 8.6 GB of bf16
    g = tv.geom(hkv, hkv, d)
    kc, vc = (torch.empty(blocks, hkv, 16, d, dtype=torch.int8, device="cuda") for _ in range(2))
    ks, vs = (torch.empty(blocks, hkv, 16, device="cuda") for _ in range(2))
    table, nb = torch.arange(blocks - 3, blocks, device="cuda").to(I32)[None], i32([3])
    k, v = fresh(78, 40, hkv, d)
    k, v = k.clamp(-4, 4).contiguous(), v.clamp(-4, 4).contiguous()
    status = i32([0])
    tv.kv_quant_append(g, k, v, i32([0, 40]), i32([0]), table, nb, kc, vc, ks, vs, status)
    ko, vo = (torch.empty(blocks, hkv, 16, d, dtype=BF16, device="cuda") for _ in range(2))
    tv.kv_quant_read(g, None, i32([40]), table, nb, kc, vc, ks, vs, table, nb, ko, vo, status)
    q = torch.randn(1, hkv, d, generator=gen(79), device="cuda").to(BF16)
    got = []
    ws = torch.empty(tv.decode_workspace_bytes(g, 1), dtype=torch.uint8, device="cuda")
    for pools in ((kc, vc, ks, vs), (ko, vo, None, None)):
        out, lse = torch.empty_like(q), torch.empty(1, hkv, device="cuda")
        tv.decode_attention(g, q, i32([40]), table, nb, *pools, out, lse, ws, status)
        got.append((out, lse))
    assert status.cpu().tolist() == [0]
    code, sc = kv_quant_ref(f64(k), "int8")
    slots = torch.arange(40, device="cuda")
    page = table[0].long()[slots // 16]
    assert np.array_equal(f64(kc[page, :, slots % 16]), code)
    assert np.array_equal(ks[page, :, slots % 16].cpu().numpy(), sc)
    vcode, vsc = kv_quant_ref(f64(v), "int8")
    rows = [code * sc.astype(np.float64)[..., None], vcode * vsc.astype(np.float64)[..., None]]
    want, wl, tol, ltol = decode_tolerance(f64(q[0]), *rows, d ** -0.5, "int8", vsc.astype(np.float64))
    assert np.all(np.abs(f64(got[0][0][0]) - want) <= tol) and np.all(np.abs(f64(got[0][1][0]) - wl) <= ltol)
    rows = [f64(x[page, :, slots % 16]) for x in (ko, vo)]
    want, wl, tol, ltol = decode_tolerance(f64(q[0]), *rows, d ** -0.5, "bf16")
    assert np.all(np.abs(f64(got[1][0][0]) - want) <= tol) and np.all(np.abs(f64(got[1][1][0]) - wl) <= ltol)


# ---------------------------------------------------------------- together


def decode_step(c, qkv, hq, pos, inv, start, bufs, stream=None):
    """One layer's decode step: rotate, write the cache, attend."""
    hkv, d, batch = c.hkv, c.d, qkv.shape[0]
    q = qkv[:, :hq * d].unflatten(1, (hq, d))
    k = qkv[:, hq * d:(hq + hkv) * d].unflatten(1, (hkv, d))
    v = qkv[:, (hq + hkv) * d:].unflatten(1, (hkv, d))
    rg, g = tv.rope_axes_geom(hq, hkv, d, [d // 8, 3 * d // 16, 3 * d // 16]), tv.geom(hq, hkv, d)
    tv.rope_axes(rg, q, k, pos, inv, q, k, stream)
    tv.kv_quant_append(g, k, v, bufs["cu"], start, c.table, c.n_blocks, c.k, c.v, c.ks, c.vs,
                       bufs["status"], stream)
    tv.decode_attention(g, q, bufs["len"], c.table, c.n_blocks, c.k, c.v, c.ks, c.vs, bufs["out"],
                        bufs["lse"], bufs["ws"], bufs["status"], stream)
    assert batch == bufs["cu"].numel() - 1


def step_setup(held, seed=81):
    hq, hkv, d, lens = 8, 2, 128, [1, 17, 700, 48]
    c = filled(seed, lens, hkv, d, held)
    g = gen(seed + 1)
    qkv = torch.randn(4, (hq + 2 * hkv) * d, generator=g, device="cuda").to(BF16)
    pos = (i32(lens) - 1)[None].repeat(3, 1) + i32([[0], [5], [9]])
    inv = (10000.0 ** (-torch.arange(d // 2, device="cuda", dtype=torch.float64) * 2 / d)).float()
    b = {"cu": i32([0, 1, 2, 3, 4]), "len": i32(lens), "status": i32([0] * 4),
         "out": torch.zeros(4, hq, d, dtype=BF16, device="cuda"), "lse": torch.zeros(4, hq, device="cuda"),
         "ws": torch.zeros(tv.decode_workspace_bytes(tv.geom(hq, hkv, d), 4), dtype=torch.uint8, device="cuda")}
    return c, qkv, hq, pos, inv, i32([n - 1 for n in lens]), b, lens


@pytest.mark.parametrize("held", ["e4m3", "int8"])
def test_decode_step_together(held):
    c, qkv, hq, pos, inv, start, b, lens = step_setup(held)
    raw = qkv.clone()
    decode_step(c, qkv, hq, pos, inv, start, b)
    assert b["status"].cpu().tolist() == [0] * 4
    d, hkv = c.d, c.hkv
    q, k = qkv[:, :hq * d].unflatten(1, (hq, d)), qkv[:, hq * d:(hq + hkv) * d].unflatten(1, (hkv, d))
    check_rope(raw[:, :hq * d].unflatten(1, (hq, d)), q, pos, inv, [16, 24, 24], 1, 0)
    check_rope(raw[:, hq * d:(hq + hkv) * d].unflatten(1, (hkv, d)), k, pos, inv, [16, 24, 24], 1, 0)
    for i, n in enumerate(lens):                     # the new rows are where and what they should be
        code, sc = kv_quant_ref(f64(k[i]), held)
        page, at = c.at(i, [n - 1])
        assert np.array_equal(f64(c.k.view(torch.int8)[page, :, at].view(c.k.dtype))[0], code)
        assert np.array_equal(c.ks[page, :, at].cpu().numpy()[0], sc)
    check_decode(c, q, lens, b["out"], b["lse"])


def test_first_calls_of_a_process_may_be_captured(tmp_path):
    """No call needs an eager one before it: a fresh process captures all four at once."""
    code = """
import sys, torch
sys.path.insert(0, %r)
sys.path.insert(0, %r)
import test_gpu_decode_ops as t
from speculative_decoding_tree_build_gb300 import kv_quant_read
c, qkv, hq, pos, inv, start, b, lens = t.step_setup("e4m3")
ko = torch.zeros(c.pool, c.hkv, 16, c.d, dtype=torch.bfloat16, device="cuda")
vo = torch.zeros_like(ko)
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    t.decode_step(c, qkv, hq, pos, inv, start, b)
    kv_quant_read(c.geom, start, b["len"], c.table, c.n_blocks, c.k, c.v, c.ks, c.vs, c.table, c.n_blocks, ko, vo, b["status"])
g.replay()
torch.cuda.synchronize()
t.check_decode(c, qkv[:, :hq * c.d].unflatten(1, (hq, c.d)), lens, b["out"], b["lse"])
assert bool(ko.any()) and b["status"].tolist() == [0] * 4
print("captured")
""" % (ROOT, os.path.join(ROOT, "tests"))
    out = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300)
    assert out.returncode == 0 and "captured" in out.stdout, out.stderr[-2000:]


def test_two_decodes_at_once_on_two_streams():
    """Two calls in flight on two streams, each with a workspace of its own."""
    sets = []
    for seed, held in ((95, "e4m3"), (97, "bf16")):
        lens = [3000, 70, 1200]
        c = filled(seed, lens, 2, 128, held)
        q = torch.randn(3, 8, 128, generator=gen(seed + 1), device="cuda").to(BF16)
        sets.append((c, q, lens, run_decode(c, q, lens), torch.cuda.Stream()))
    for _ in range(10):
        got = []
        for c, q, lens, _, s in sets:
            s.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(s):
                got.append(run_decode(c, q, lens))
        torch.cuda.synchronize()
        for (out, lse, _), (_, _, _, want, _) in zip(got, sets):
            assert np.array_equal(bits(out), bits(want[0])) and np.array_equal(bits(lse), bits(want[1]))


def test_decode_step_captured_and_replayed():
    """A graph of the three calls, replayed on new inputs, and two graphs that share a workspace."""
    c, qkv, hq, pos, inv, start, b, lens = step_setup("e4m3")
    raw, pools = qkv.clone(), [t.clone() for t in (c.k, c.v, c.ks, c.vs)]

    def reset(x):
        qkv.copy_(x)
        for t, s in zip((c.k, c.v, c.ks, c.vs), pools):
            t.copy_(s)

    decode_step(c, qkv, hq, pos, inv, start, b)
    eager = b["out"].clone(), b["lse"].clone()
    graphs = []
    for _ in range(2):
        reset(raw)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            decode_step(c, qkv, hq, pos, inv, start, b)
        graphs.append(g)
    for g in graphs + graphs:
        reset(raw)
        b["out"].zero_()
        b["ws"].fill_(0xff)
        g.replay()
        torch.cuda.synchronize()
        assert np.array_equal(bits(b["out"]), bits(eager[0])) and np.array_equal(bits(b["lse"]), bits(eager[1]))
    other = torch.randn(raw.shape, generator=gen(90), device="cuda").to(BF16)
    reset(other)
    graphs[0].replay()
    torch.cuda.synchronize()
    q = qkv[:, :hq * c.d].unflatten(1, (hq, c.d))
    check_decode(c, q, lens, b["out"], b["lse"])


def test_tree_verification_over_a_read_back_cache():
    """An 8-bit cache read back feeds the tree step: the same bits as over a
    bf16 cache that holds the values the codes stand for."""
    from gen import workloads as wl
    from speculative_decoding_tree_build_gb300.step import DeviceBatch
    w = wl.make_config(2, batch=3, prompt_scale=0.1)
    a, z = DeviceBatch(w), DeviceBatch(w)
    hkv, d = w["num_kv_heads"], w["head_dim"]
    plen = [int(x) for x in w["prompt_len"]]
    c = Cache(91, plen, hkv, d, "int8")
    cu = [0] + np.cumsum(plen).tolist()
    rows = []
    for cache in (a.k_cache, a.v_cache):
        got = []
        for b, n in enumerate(plen):
            s = torch.arange(n, device="cuda")
            got.append(cache[a.block_table[b].long()[s // 16], :, s % 16])
        rows.append(torch.cat(got).contiguous())
    assert run_append(c, rows[0], rows[1], cu, [0] * 3) == [0] * 3
    z.k_cache.zero_()
    z.v_cache.zero_()
    st = i32([0] * 3)
    tv.kv_quant_read(c.geom, None, i32(plen), c.table, c.n_blocks, c.k, c.v, c.ks, c.vs, z.block_table,
                     z.n_blocks, z.k_cache, z.v_cache, st)
    assert st.cpu().tolist() == [0] * 3
    for cache, x in ((a.k_cache, rows[0]), (a.v_cache, rows[1])):
        code, sc = kv_quant_ref(f64(x), "int8")
        val = (torch.from_numpy(code).float() * torch.from_numpy(sc)[..., None]).to(BF16).cuda()
        for b, n in enumerate(plen):
            s = torch.arange(n, device="cuda")
            cache[a.block_table[b].long()[s // 16], :, s % 16] = val[cu[b]:cu[b + 1]]
    for x in (a, z):
        x.step()
    torch.cuda.synchronize()
    assert a.status.cpu().tolist() == z.status.cpu().tolist() == [0] * 3
    assert np.array_equal(bits(a.out), bits(z.out))
    assert np.array_equal(a.accept_path.cpu().numpy(), z.accept_path.cpu().numpy())
    assert np.array_equal(a.new_len.cpu().numpy(), z.new_len.cpu().numpy())
