"""The restatement of block tables and slot maps against facts of other origin,
and the host-side refusals of the calls."""

import ctypes
import random

import pytest

import speculative_decoding_tree_build_gb300 as tv
from oracle import block_tables_ref, kv_commit_ref, slot_map_ref
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


def test_block_tables_refusals(lib):
    # batch, want, table, n_blocks, max_blocks, num_blocks, free, count, released, released_count,
    # status, stream
    args = [2, P, P, P, 4, 9, P, P, P, P, P, None]

    def call(a):
        return lib.tv_block_tables(*a)

    assert call(swap(args, _0=0)) == OK
    for i, v in ((0, -1), (0, 4097), (4, 0), (5, 0)):
        assert call(swap(args, **{f"_{i}": v})) == SIZE
    for i in (1, 2, 3, 6, 7, 8, 9, 10):              # released and its count come together
        assert call(swap(args, **{f"_{i}": None})) == NULL


def test_slot_map_refusals(lib):
    # batch, rows, cu, start, table, n_blocks, max_blocks, num_blocks, slots, status, stream
    args = [2, 5, P, P, P, P, 4, 9, P, P, None]

    def call(a):
        return lib.tv_slot_map(*a)

    assert call(swap(args, _1=0)) == OK
    for i, v in ((0, -1), (0, 4097), (1, -1), (6, 0), (7, 0)):
        assert call(swap(args, **{f"_{i}": v})) == SIZE
    for i in (2, 3, 4, 5, 8, 9):
        assert call(swap(args, **{f"_{i}": None})) == NULL
    assert call(swap(args, _8=P + 4)) == MIS


def test_slot_map_refuses_tables_past_31_bits(lib):
    """A table of more than 2^27 pages has token positions that 32 bits do not hold."""
    args = [2, 5, P, P, P, P, (1 << 27) + 1, 9, P, P, None]
    assert lib.tv_slot_map(*args) == SIZE
    assert lib.tv_slot_map(*swap(args, _6=1 << 27, _1=0)) == OK


def test_kv_rows_refusals(lib):
    g, d96, many = tv.geom(32, 8, 128), tv.geom(32, 8, 96), tv.geom(4097, 4097, 64)
    # geom, rows, k, k_ld, v, v_ld, slots, k_cache, v_cache, num_blocks, stream
    args = [ctypes.byref(g), 5, P, 1024, P, 1024, P, P, P, 9, None]

    def write(a):
        return lib.tv_kv_rows_write(*a)

    def read(a):                                     # geom, rows, slots, kc, vc, blocks, k, ld, v, ld
        return lib.tv_kv_rows_read(a[0], a[1], a[6], a[7], a[8], a[9], a[2], a[3], a[4], a[5], a[10])

    for call in (write, read):
        assert call(swap(args, _1=0)) == OK
        assert call(swap(args, _0=None)) == NULL
        assert call(swap(args, _0=ctypes.byref(d96))) == GEOM
        assert call(swap(args, _0=ctypes.byref(many), _3=4097 * 64, _5=4097 * 64)) == GEOM
        for i, v in ((1, -1), (3, 1023), (5, 1016), (9, 0)):
            assert call(swap(args, **{f"_{i}": v})) == SIZE
        for i in (2, 4, 6, 7, 8):
            assert call(swap(args, **{f"_{i}": None})) == NULL
        for i, v in ((2, P + 8), (3, 1028), (4, P + 2), (5, 1025), (6, P + 4), (7, P + 8), (8, P + 1)):
            assert call(swap(args, **{f"_{i}": v})) == MIS


def test_a_shrink_undoes_a_growth():
    rng = random.Random(3)
    for _ in range(200):
        batch, width, pool = rng.randint(1, 6), rng.randint(1, 9), 60
        ids = rng.sample(range(pool), pool)
        n = [rng.randint(0, width) for _ in range(batch)]
        table = [[ids.pop() for _ in range(c)] + [-1] * (width - c) for c in n]
        grown = [rng.randint(c, width) for c in n]
        up = block_tables_ref([16 * g - rng.randint(0, 15) if g else 0 for g in grown], table, n, ids, pool, [0] * batch)
        assert up[1] == grown and len(up[2]) == len(ids) - (sum(grown) - sum(n)) and up[3] == [0] * batch
        down = block_tables_ref([16 * c for c in n], *up[:3], pool, [0] * batch)
        assert down[:3] == (table, n, ids)


def test_blocks_are_never_lost_or_held_twice():
    rng = random.Random(4)
    for _ in range(200):
        batch, width, pool = rng.randint(1, 8), 7, rng.randint(1, 40)
        n, free, table = [0] * batch, list(range(pool)), [[-1] * width for _ in range(batch)]
        for _ in range(6):
            want = [rng.randint(-2, 16 * width + 3) for _ in range(batch)]
            table, n, free, status, _ = block_tables_ref(want, table, n, free, pool, [0] * batch)
            held = [i for r, c in zip(table, n) for i in r[:c]]
            assert sorted(held + free) == list(range(pool))
            refused = False
            for b in range(batch):
                if want[b] < 0 or want[b] > 16 * width:
                    assert status[b] == 1
                elif status[b]:
                    assert status[b] == 128
                    refused = True
                else:
                    assert n[b] == -(-want[b] // 16)
            assert refused or 128 not in status


def test_released_blocks_come_back_once():
    # kv_commit's own release: 3 pages held, 18 slots kept
    import numpy as np
    k = np.zeros((6, 1, 16, 64), np.uint16)
    table = np.array([5, 2, 4], np.int32)
    st, new_len, held, released = kv_commit_ref(k, k.copy(), table, 3, 14, [0, 1, 2, 3])
    assert (st, new_len, held, list(released)) == (0, 18, 2, [4])
    got = block_tables_ref([18], [list(table[:2]) + [-1]], [2], [0, 1, 3], 6, [0], [list(released) + [-1, -1]], [1])
    assert got[2] == [0, 1, 3, 4] and got[4] == [0]
    again = block_tables_ref([18], *got[:3], 6, [0], [list(released) + [-1, -1]], got[4])
    assert again[2] == [0, 1, 3, 4]


def test_slot_map_by_hand():
    table = [[7, 3, -1], [0, 5, 9]]
    slots, status = slot_map_ref([1, 4, 6], [15, 31], table, [2, 3], 10, 8, [0, 0])
    assert slots.tolist() == [-1, 7 * 16 + 15, 3 * 16, 3 * 16 + 1, 5 * 16 + 15, 9 * 16, -1, -1] and status == [0, 0]
    assert slot_map_ref([0, 3], [30], table[:1], [2], 10, 3, [0])[1] == [8]        # the third page is not held
    assert slot_map_ref([0, 3, 2], [0, 0], table, [2, 3], 10, 3, [0, 0])[1] == [0, 1]
    assert slot_map_ref([0, 3, 4], [0, 0], table, [2, 3], 4, 4, [0, 0])[1] == [8, 0]   # page 7 of 4
