"""Pages, slots, rows and filters where sizes pass 31 bits or weights lose steps."""

import numpy as np
import pytest
import torch

import speculative_decoding_tree_build_gb300 as tv
from oracle import draw_ref, filter_ref

pytestmark = pytest.mark.gpu

BF16, F32, I32 = torch.bfloat16, torch.float32, torch.int32


def i32(x):
    return torch.tensor(x, dtype=I32, device="cuda")


def f32(x):
    return torch.tensor(x, dtype=F32, device="cuda")


@pytest.mark.parametrize("rows", [2 ** 31 - 1, 2 ** 31 - 2047])
def test_slot_map_of_the_most_rows(rows):
    assert torch.cuda.mem_get_info()[0] > 40 << 30
    slots = torch.empty(rows, dtype=torch.int64, device="cuda")
    st = i32([0, 0])
    table, n = i32([[4, 2], [7, 1]]), i32([2, 2])
    tv.slot_map(i32([rows - 25, rows - 8, rows]), i32([3, 20]), table, n, 8, slots, st)
    assert st.tolist() == [0, 0]
    assert slots[-25:].tolist() == [4 * 16 + 3 + i for i in range(13)] + [2 * 16 + i for i in range(4)] + [16 + 4 + i for i in range(8)]
    for part in slots[:-25].split(1 << 28):
        assert int(part.max()) == int(part.min()) == -1


def test_rows_in_a_pool_past_31_bits():
    """2.3e9 elements of K and of V; the rows lie at both ends and around 2^31."""
    pool, hkv, d = 140001, 8, 128
    assert torch.cuda.mem_get_info()[0] > 16 << 30
    g = tv.geom(32, hkv, d)
    kc, vc = (torch.zeros(pool, hkv, 16, d, dtype=BF16, device="cuda") for _ in range(2))
    edge = 2 ** 31 // (hkv * d)
    where = [0, 1, edge - 1, edge, edge + 17, 16 * pool - 1, 16 * pool, -1, 2 ** 40]
    slots = torch.tensor(where, dtype=torch.int64, device="cuda")
    k, v = (torch.randn(len(where), hkv, d, device="cuda").to(BF16) for _ in range(2))
    tv.kv_rows_write(g, k, v, slots, kc, vc)
    ko, vo = torch.full_like(k, 3.0), torch.full_like(v, 3.0)
    tv.kv_rows_read(g, slots, kc, vc, ko, vo)
    assert torch.equal(ko[:6], k[:6]) and torch.equal(vo[:6], v[:6])
    assert bool((ko[6:] == 3.0).all()) and bool((vo[6:] == 3.0).all())
    for i, s in enumerate(where[:6]):
        assert torch.equal(kc[s // 16, :, s % 16], k[i]) and torch.equal(vc[s // 16, :, s % 16], v[i])
    assert int((kc != 0).any(dim=3).sum()) == 6 * hkv == int((vc != 0).any(dim=3).sum())


@pytest.mark.parametrize("v", [1 << 18, (1 << 20) - 3])
@pytest.mark.parametrize("sigma", [0.01, 2.0])
def test_top_p_of_a_vocabulary_with_coarser_steps(v, sigma):
    """Steps are 2^-(62 - log2 v) of the largest weight; v half steps move a sum by
    v 2^-(63 - log2 v) at most."""
    rng = np.random.default_rng(v % 1000)
    rows = 3
    x = (rng.standard_normal((rows, v)) * sigma).astype(np.float32)
    ld = -(-v // 4) * 4
    lg = torch.zeros(rows, ld, device="cuda")
    lg[:, :v] = torch.from_numpy(x).cuda()
    noise = torch.zeros(rows, ld, device="cuda")
    noise[:, :v] = -torch.log(-torch.log(torch.from_numpy(rng.uniform(1e-7, 1 - 1e-7, (rows, v)).astype(np.float32)).cuda()))
    cu, t, p = i32([0, 1, 2, 3]), f32([1.0, 0.7, 1.5]), f32([0.9, 0.5, 0.99])
    tok, lp, st, kept = i32([0] * 3), f32([0.0] * 3), i32([0] * 3), i32([0] * 3)
    out = torch.empty_like(lg)
    tv.sample_filtered(lg[:, :v], noise[:, :v], cu, t, None, p, None, 1, tok, lp, st)
    tv.filter_logits(lg[:, :v], cu, t, None, p, None, 1, out[:, :v], kept, st)
    assert st.tolist() == [0] * 3
    for r in range(rows):
        keep, s, w, margin = filter_ref(x[r], float(t[r]), 0, float(p[r]), 0.0)
        assert margin > 2.0 ** -33 + v * 2.0 ** (np.ceil(np.log2(v)) - 63) / float(w.sum())
        token, logp = draw_ref(keep, s, w, noise[r, :v].cpu().numpy())
        assert int(tok[r]) == token and int(kept[r]) == int(keep.sum())
        assert np.array_equal(out[r, :v].cpu().numpy() > -np.inf, keep)
        assert abs(float(lp[r]) - logp) <= 2.0 ** -18      # five roundings of up to 16
