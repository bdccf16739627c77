"""The float64 restatement of the plain-decoding calls, held to facts that do
not come from it: torch's e4m3 cast, brute-force nearest codes, one-axis rotary
positions, the tree oracle's attention for a lone root."""

import numpy as np
import pytest
import torch

from oracle import (axis_of_pair_ref, decode_attention_ref, kv_quant_ref, packed_attention_ref,
                    rope_axes_ref, rope_ref, round_e4m3_ref)


def test_axis_orders():
    assert axis_of_pair_ref([2, 3, 1], 0) == [0, 0, 1, 1, 1, 2]
    assert axis_of_pair_ref([2, 3, 1], 1) == [0, 1, 2, 0, 1, 1]
    assert axis_of_pair_ref([0, 2, 2], 1) == [1, 2, 1, 2]


@pytest.mark.parametrize("style", [0, 1])
def test_rope_axes_with_equal_positions_is_plain_rope(style):
    rng = np.random.default_rng(3)
    d, rows = 16, 5
    x = rng.standard_normal((rows, 2, d))
    pos = np.array([0, 1, 7, 30, 100], np.int32)
    inv = np.float32(10000.0) ** (-np.arange(d // 2, dtype=np.float32) * 2 / d)
    got = rope_axes_ref(x, np.stack([pos] * 3), inv, [3, 3, 2], style, 1)
    want = rope_ref(x, pos, 10000.0, style, round_bf16=False)
    # the tree oracle rounds inv_freq and the angle to float32: 100 * 2^-22 rad at most
    assert np.abs(got - want).max() < 100 * 2.0 ** -22 * np.abs(x).max() * 2


def test_rope_axes_turns_each_pair_by_its_own_axis():
    x = np.zeros((1, 1, 8))
    x[..., 0::2] = 1.0                              # unit vectors along each pair's first column
    got = rope_axes_ref(x, [[2], [3]], [0.5, 0.25, 0.125], [1, 2], 0, 0)[0, 0]
    ang = np.array([2 * 0.5, 3 * 0.25, 3 * 0.125])
    assert np.allclose(got[0:6:2], np.cos(ang)) and np.allclose(got[1:6:2], np.sin(ang))
    assert got[6] == 1.0 and got[7] == 0.0          # past the rotated pairs


def test_e4m3_rounding_is_torchs():
    y = np.concatenate([np.linspace(-448, 448, 40001), np.ldexp(1.0, np.arange(-14, 9)),
                        np.arange(-64, 65) * 2.0 ** -10])
    y = y.astype(np.float32)
    want = torch.from_numpy(y).to(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(round_e4m3_ref(y), want)


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_codes_are_the_nearest(fmt):
    rng = np.random.default_rng(5)
    x = torch.from_numpy(rng.standard_normal((40, 32)) * 2.0 ** rng.integers(-30, 30, (40, 1)))
    x = x.to(torch.bfloat16).double().numpy()
    x[3] = 0.0
    code, scale = kv_quant_ref(x, fmt)
    if fmt == "e4m3":
        all_codes = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
        grid = np.unique(all_codes[np.isfinite(all_codes)])
        unit = scale.astype(np.float64)
        top = np.abs(x).max(-1)
        assert np.all(top <= 448 * unit) and np.all((top > 224 * unit) | (unit == 2.0 ** -100))
        assert np.array_equal(np.exp2(np.rint(np.log2(unit))), unit)
    else:
        grid = np.arange(-127.0, 128.0)
        unit = np.maximum(np.abs(x).max(-1), 2.0 ** -100) / 127
        assert np.array_equal(unit.astype(np.float32), scale)
    y = x / unit[:, None]
    best = np.abs(y[..., None] - grid).min(-1)
    assert np.allclose(np.abs(y - code), best, rtol=0, atol=1e-12)
    assert not code[3].any()


def test_rows_that_are_not_finite_are_marked():
    x = np.ones((3, 8))
    x[0, 2], x[1, 5] = np.nan, np.inf
    for fmt in ("e4m3", "int8"):
        code, scale = kv_quant_ref(x, fmt)
        assert np.isnan(scale[:2]).all() and not code[:2].any() and np.isfinite(scale[2])


def test_decode_attention_is_a_lone_root():
    rng = np.random.default_rng(7)
    hq, hkv, d, n = 4, 2, 8, 11
    q, k, v = rng.standard_normal((hq, d)), rng.standard_normal((n, hkv, d)), rng.standard_normal((n, hkv, d))
    got, lse, _, _ = decode_attention_ref(q, k, v, d ** -0.5)
    # the last row is the token itself: a tree of one node
    want = packed_attention_ref(q[None], k[:-1], v[:-1], k[-1:], v[-1:], np.ones((1, n), bool))
    assert np.abs(got - want.reshape(hq, d)).max() < 1e-12
    s = np.einsum("hd,nhd->hn", q, np.repeat(k, hq // hkv, 1)) * d ** -0.5
    assert np.allclose(lse, np.log(np.exp(s).sum(1)))
    out, lse, _, _ = decode_attention_ref(q, k[:0], v[:0], 1.0)
    assert not out.any() and np.isneginf(lse).all()
