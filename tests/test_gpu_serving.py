"""A tree step whose pages, tokens and acceptance stay on the device: pages from the
list, tokens from a filtered distribution, the commit's pages back on the list. The
same step over a table laid out by hand gives the same bits."""

import numpy as np
import pytest
import torch

import speculative_decoding_tree_build_gb300 as tv
from gen import workloads as wl
from speculative_decoding_tree_build_gb300.step import DeviceBatch

pytestmark = pytest.mark.gpu

I32 = torch.int32


def filters(batch, dev):
    f = lambda x: torch.tensor((x * batch)[:batch], device=dev)
    return f([0.8, 1.0, 0.6]).float(), f([30, 0, 0]).to(I32), f([0.9, 0.8, 1.0]).float(), f([0.0, 0.02, 0.1]).float()


@pytest.mark.parametrize("capture", [False, True])
def test_step_with_pages_and_filtered_tokens(capture):
    w = wl.make_config(2, batch=3, seed=77)
    rng = np.random.default_rng(5)
    logits, gumbel = (torch.from_numpy(a).cuda() for a in wl.sampling_inputs(rng, w))
    by_hand, db = DeviceBatch(w, device="cuda"), DeviceBatch(w, device="cuda")
    batch, dev = w["batch"], by_hand.device
    pool = by_hand.k_cache.shape[0]
    temps = filters(batch, dev)
    cu = w["cu_nodes"].astype(np.int64)
    plen, nodes = w["prompt_len"].astype(np.int64), np.diff(cu)
    # the prompts' pages are held, all others are on the list in an order of their own
    held = -(-plen // 16)
    table = np.array(w["block_table"], copy=True)
    for b in range(batch):
        table[b, held[b]:] = -1
    used = {int(i) for b in range(batch) for i in table[b, :held[b]]}
    free = rng.permutation([i for i in range(pool) if i not in used]).astype(np.int32)
    db.block_table.copy_(torch.from_numpy(table))
    db.n_blocks.copy_(torch.from_numpy(held.astype(np.int32)))
    list_ = torch.full((pool,), -1, dtype=I32, device=dev)
    list_[:len(free)] = torch.from_numpy(free).cuda()
    top = torch.tensor([len(free)], dtype=I32, device=dev)
    want = torch.from_numpy((plen + nodes).astype(np.int32)).cuda()
    kept_len = torch.zeros(batch, dtype=I32, device=dev)
    tokens = [torch.zeros(int(cu[-1]), dtype=I32, device=dev) for _ in range(2)]
    logp = torch.zeros(int(cu[-1]), device=dev)

    def step(d, tok, pages):
        d.tree_build()
        if pages:
            tv.block_tables(want, d.block_table, d.n_blocks, list_, top, d.status, d.released, d.released_count)
        d.attention()
        tv.sample_filtered(logits, gumbel, d.cu_nodes, *temps, d.max_nodes, tok, logp, d.status)
        tv.greedy_accept(tok, d.draft_tokens, d.cu_nodes, d.next_token, d.next_sibling, d.max_nodes, d.accept_path,
                         d.accept_len, d.bonus, d.status)
        d.commit()

    step(by_hand, tokens[0], False)
    if capture:
        state = [t.clone() for t in (db.k_cache, db.v_cache, db.table_state, list_, top)]
        step(db, tokens[1], True)                # (first calls outside the capture)
        for t, s in zip((db.k_cache, db.v_cache, db.table_state, list_, top), state):
            t.copy_(s)
        db.released_count.zero_()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step(db, tokens[1], True)
        graph.replay()
    else:
        step(db, tokens[1], True)
    torch.cuda.synchronize()
    assert db.status.tolist() == [0] * batch == by_hand.status.tolist()
    for name in ("out", "accept_path", "accept_len", "bonus", "new_len", "released_count"):
        assert torch.equal(getattr(db, name), getattr(by_hand, name)), name
    assert torch.equal(tokens[0], tokens[1])
    # every page is in one place: a table, the commit's list, the free list
    def everywhere():
        ids = [int(i) for b in range(batch) for i in db.block_table[b, :int(db.n_blocks[b])]]
        ids += [int(i) for b in range(batch) for i in db.released[b, :int(db.released_count[b])]]
        return sorted(ids + list_[:int(top[0])].tolist())
    assert everywhere() == list(range(pool))
    # the committed rows lie where the new lengths say, read through a slot map
    lens = db.new_len.tolist()
    rows = sum(lens)
    offsets = torch.tensor([0] + np.cumsum(lens).tolist(), dtype=I32, device=dev)
    got = []
    for d in (db, by_hand):
        slots = torch.empty(rows + 3, dtype=torch.int64, device=dev)
        st = torch.zeros(batch, dtype=I32, device=dev)
        tv.slot_map(offsets, torch.zeros(batch, dtype=I32, device=dev), d.block_table, d.n_blocks, pool, slots, st)
        assert st.tolist() == [0] * batch and slots[rows:].tolist() == [-1] * 3
        k, v = (torch.zeros(rows + 3, d.k_cache.shape[1], d.k_cache.shape[3], dtype=torch.bfloat16, device=dev) for _ in range(2))
        tv.kv_rows_read(d.g, slots, d.k_cache, d.v_cache, k, v)
        got.append((k, v))
    assert torch.equal(got[0][0].view(torch.int16), got[1][0].view(torch.int16))
    assert torch.equal(got[0][1].view(torch.int16), got[1][1].view(torch.int16))
    # the next step's pages: what the commit released comes back first
    kept_len.copy_(db.new_len)
    db.status.zero_()
    tv.block_tables(kept_len, db.block_table, db.n_blocks, list_, top, db.status, db.released, db.released_count)
    assert db.status.tolist() == [0] * batch and db.released_count.tolist() == [0] * batch
    assert db.n_blocks.tolist() == [-(-n // 16) for n in lens] and everywhere() == list(range(pool))
