"""Block tables, slot maps and rows at slots on the GPU against their
restatement (oracle/pages_ref.py): every number is compared exactly."""

import random

import numpy as np
import pytest
import torch

import speculative_decoding_tree_build_gb300 as tv
from oracle import block_tables_ref, slot_map_ref

pytestmark = pytest.mark.gpu

BF16, I32 = torch.bfloat16, torch.int32


def i32(x):
    return torch.tensor(x, dtype=I32, device="cuda")


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def bits(t):
    return t.view(torch.int16).cpu().numpy()


# ---------------------------------------------------------------- block tables


class Pages:
    """Requests that hold random pages of a pool, the rest on the list."""

    def __init__(self, rng, batch, width, pool, released=0):
        ids = rng.sample(range(pool), pool)
        self.pool = pool
        self.n = [min(rng.randint(0, width), pool // batch) for _ in range(batch)]
        self.table = [[ids.pop() for _ in range(c)] + [-1] * (width - c) for c in self.n]
        self.count = [min(rng.randint(0, released), width, len(ids) // batch) for _ in range(batch)]
        self.released = [[ids.pop() for _ in range(c)] + [-7] * (width - c) for c in self.count]
        self.free = ids
        self.status = [0] * batch

    def device(self):
        free = torch.full((self.pool,), -9, dtype=I32, device="cuda")
        free[:len(self.free)] = i32(self.free)
        return {"table": i32(self.table), "n": i32(self.n), "free": free, "top": i32([len(self.free)]),
                "released": i32(self.released), "count": i32(self.count), "status": i32(self.status)}


def call(d, want, with_released=True, stream=None):
    tv.block_tables(want if torch.is_tensor(want) else i32(want), d["table"], d["n"], d["free"], d["top"], d["status"],
                    d["released"] if with_released else None, d["count"] if with_released else None, stream)


def check(d, ref):
    table, n, free, status, count = ref
    assert d["status"].tolist() == status
    assert d["n"].tolist() == n
    assert d["count"].tolist() == count
    assert d["top"].tolist() == [len(free)]
    assert d["free"][:len(free)].tolist() == free
    assert d["table"].tolist() == table


def reference(p, want):
    return block_tables_ref(want, p.table, p.n, p.free, p.pool, p.status, p.released, p.count)


@pytest.mark.parametrize("batch,width,pool", [(1, 1, 1), (1, 5, 4), (2, 3, 30), (7, 40, 120), (64, 60, 2500),
                                              (1023, 7, 5000), (1025, 5, 4000), (4096, 3, 9000), (3, 5000, 12000)])
@pytest.mark.parametrize("seed", [0, 1, 2])
def test_block_tables(batch, width, pool, seed):
    rng = random.Random(1000 * seed + batch)
    p = Pages(rng, batch, width, pool, released=2)
    want = [rng.randint(0, 16 * width) for _ in range(batch)]
    if seed == 1:
        want = [max(0, 16 * c - rng.randint(0, 40)) for c in p.n]      # nothing grows
    if seed == 2:
        want = [16 * width] * batch                                    # more than there is
    d = p.device()
    call(d, want)
    check(d, reference(p, want))


def test_block_tables_flags():
    rng = random.Random(5)
    p = Pages(rng, 12, 6, 80, released=3)
    want = [rng.randint(0, 96) for _ in range(12)]
    want[0], want[1] = -1, 97                       # sizes
    p.n[2] = 7
    p.n[3] = -1
    p.count[4], p.count[5] = -1, 7
    p.status[6] = 16                                # flagged before
    p.n[7], want[7] = 2, 0
    p.table[7][:2] = [3, 80]                        # an id of another pool goes back
    p.count[8], p.released[8][:2] = 2, [1, -1]
    d = p.device()
    call(d, want)
    ref = reference(p, want)
    assert [ref[3][b] for b in range(9)] == [1, 1, 1, 1, 1, 1, 16, 8, 8]
    check(d, ref)


def test_block_tables_long_shrink_with_one_bad_id():
    """A bad id that only another thread block meets holds its request back in all of them."""
    rng = random.Random(6)
    p = Pages(rng, 3, 9000, 30000)
    p.n = [9000, 9000, 9000]
    ids = rng.sample(range(30000), 27000)
    p.table = [ids[9000 * b:9000 * (b + 1)] for b in range(3)]
    p.free = [i for i in range(30000) if i not in set(ids)]
    p.count = [0, 0, 0]
    p.table[1][8765] = 30000
    d = p.device()
    call(d, [160, 0, 16])
    ref = reference(p, [160, 0, 16])
    assert ref[3] == [0, 8, 0]
    check(d, ref)


@pytest.mark.parametrize("top", [-1, 41, 2 ** 31 - 1])
def test_block_tables_list_out_of_range(top):
    p = Pages(random.Random(7), 4, 5, 40)
    d = p.device()
    before = {k: v.clone() for k, v in d.items()}
    d["top"].fill_(top)
    call(d, [80, 0, 16, 3])
    assert d["status"].tolist() == [1] * 4 and d["top"].tolist() == [top]
    for k in ("table", "n", "free", "count"):
        assert torch.equal(d[k], before[k])


def test_block_tables_list_too_full():
    """Pages that are on the list and in a table at once: nothing is written past the list."""
    p = Pages(random.Random(8), 4, 5, 40)
    p.free = list(range(40))
    d = p.device()
    before = {k: v.clone() for k, v in d.items()}
    want = [0] * 4
    call(d, want)
    assert sum(p.n) > 0 and d["status"].tolist() == [1] * 4
    for k in ("table", "n", "free", "top", "count"):
        assert torch.equal(d[k], before[k])


def test_block_tables_growth_and_back_restores_everything():
    rng = random.Random(9)
    p = Pages(rng, 37, 50, 4000)
    d = p.device()
    before = {k: v.clone() for k, v in d.items()}
    call(d, [16 * min(50, c + rng.randint(0, 9)) for c in p.n], with_released=False)
    assert not torch.equal(d["n"], before["n"])
    call(d, [16 * c for c in p.n], with_released=False)
    for k in ("table", "n", "top", "status", "free"):
        assert torch.equal(d[k], before[k])


def test_block_tables_captured():
    """A captured call takes blocks again at every replay."""
    p = Pages(random.Random(10), 5, 30, 400)
    p.n, p.table, p.free = [0] * 5, [[-1] * 30 for _ in range(5)], list(range(400))
    p.count = [0] * 5
    d = p.device()
    want = i32([16] * 5)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(d, want)
    ref = reference(p, [16] * 5)
    for step in range(1, 4):
        graph.replay()
        check(d, ref)
        want += 16
        ref = block_tables_ref([16 * (step + 1)] * 5, *ref[:3], 400, [0] * 5, p.released, ref[4])


# ---------------------------------------------------------------- slots


def slots_case(seed, batch, most, spare, start_most):
    rng = np.random.default_rng(seed)
    lens = rng.integers(0, most + 1, batch)
    cu = np.concatenate([[3], 3 + np.cumsum(lens)])
    start = rng.integers(0, start_most + 1, batch)
    need = -(-(start + lens) // 16)
    width, pool = max(int(need.max()), 1), int(need.sum()) + 5
    ids = rng.permutation(pool)
    table, at = np.full((batch, width), -1, np.int32), 0
    for b in range(batch):
        table[b, :need[b]] = ids[at:at + need[b]]
        at += need[b]
    return cu, start, table, need, pool, int(cu[-1]) + spare


def run_slots(cu, start, table, n_blocks, pool, rows, status):
    slots = torch.full((rows,), 77, dtype=torch.int64, device="cuda")
    st = i32(list(status))
    tv.slot_map(i32(list(map(int, cu))), i32(list(map(int, start))), i32(np.asarray(table).tolist()),
                i32(list(map(int, n_blocks))), pool, slots, st)
    return slots, st


def check_slots(cu, start, table, n_blocks, pool, rows, status):
    got, st = run_slots(cu, start, table, n_blocks, pool, rows, status)
    want, ref = slot_map_ref(cu, start, np.asarray(table).tolist(), n_blocks, pool, rows, status)
    assert st.tolist() == [int(x) for x in ref]
    assert np.array_equal(got.cpu().numpy(), want)
    return ref


@pytest.mark.parametrize("batch,most,spare,start_most", [(1, 1, 0, 0), (1, 700, 9, 40), (5, 33, 4, 3000), (64, 129, 50, 9000),
                                                         (4096, 2, 1, 50), (3, 300000, 7, 100), (40, 20000, 0, 17),
                                                         (513, 3000, 11, 33)])
def test_slot_map(batch, most, spare, start_most):
    case = slots_case(batch, batch, most, spare, start_most)
    status = [0] * batch
    if batch > 3:
        status[2] = 64
    check_slots(*case, status)


def test_slot_map_no_requests():
    slots = torch.full((6,), 5, dtype=torch.int64, device="cuda")
    e = torch.empty(0, dtype=I32, device="cuda")
    tv.slot_map(i32([0]), e, torch.empty(0, 1, dtype=I32, device="cuda"), e, 4, slots, e)
    assert slots.tolist() == [-1] * 6


def test_slot_map_missing_and_foreign_blocks():
    cu, start, table, n, pool, rows = slots_case(11, 6, 9000, 3, 50)
    n = n.copy()
    n[1] -= 1                                        # a page short
    table[2, n[2] - 1] = pool                        # ids outside the pool, at the ends of long requests
    table[3, int(start[3]) // 16] = -1
    table[4, n[4] - 1:] = 5                          # (a page of another request: no fault that the call can see)
    ref = check_slots(cu, start, table, n, pool, rows, [0] * 6)
    assert ref[:4] == [0, 8, 8, 8]
    n[0] = table.shape[1] + 9                        # more than the table has: what is needed is there
    assert check_slots(cu, start, table, n, pool, rows, [0] * 6)[0] == 0


@pytest.mark.parametrize("cu", [[0, 5, 3, 9], [0, 5, 3, 3], [4, 2, 6, 9], [-2, 3, 5, 9], [0, 3, 5, 13], [0, 9, 9, 9],
                                [7, 7, 7, 7], [0, 12, 2, 12], [12, 0, 5, 9]])
def test_slot_map_offsets(cu):
    table = [[0, 1], [2, 3], [4, 5]]
    check_slots(cu, [0, 4, 9], table, [2, 2, 2], 6, 12, [0, 0, 0])


def test_slot_map_bad_start():
    table = [[0, 1], [2, 3], [4, 5]]
    ref = check_slots([0, 3, 6, 9], [-1, 2 ** 31 - 2, 29], table, [2, 2, 2], 6, 9, [0] * 3)
    assert ref == [1, 8, 0]


# ---------------------------------------------------------------- rows


@pytest.mark.parametrize("rows,hkv,d,fused", [(1, 1, 64, False), (5, 8, 128, True), (700, 3, 64, False), (301, 8, 128, False),
                                              (33, 16, 128, True), (2000, 1, 128, False), (3, 600, 64, False),
                                              (257, 5, 64, True)])
def test_rows_written_and_read(rows, hkv, d, fused):
    g = gen(rows)
    blocks = -(-rows // 16) + 3
    geom = tv.geom(hkv, hkv, d)
    n = hkv * d
    if fused:
        kv = torch.randn(rows, 2 * n + 8, generator=g, device="cuda").to(BF16)
        k, v = kv[:, :n].unflatten(1, (hkv, d)), kv[:, n:2 * n].unflatten(1, (hkv, d))
    else:
        k, v = (torch.randn(rows, hkv, d, generator=g, device="cuda").to(BF16) for _ in range(2))
    k[0, 0, 0] = float("nan")
    slots = torch.randperm(blocks * 16, generator=g, device="cuda")[:rows]
    off = torch.rand(rows, generator=g, device="cuda") < 0.2
    slots[off] = torch.tensor([-1, blocks * 16, -2 ** 62, 2 ** 62], device="cuda")[torch.arange(rows, device="cuda") % 4][off]
    kc, vc = (torch.randn(blocks, hkv, 16, d, generator=g, device="cuda").to(BF16) for _ in range(2))
    want = []
    for pool, x in ((kc, k), (vc, v)):
        w = pool.clone()
        on = ~off
        w[slots[on] // 16, :, slots[on] % 16] = x[on]
        want.append(w)
    tv.kv_rows_write(geom, k, v, slots, kc, vc)
    assert np.array_equal(bits(kc), bits(want[0])) and np.array_equal(bits(vc), bits(want[1]))
    # and back, into rows that keep what has no slot
    ko, vo = (torch.randn(rows, hkv, d, generator=g, device="cuda").to(BF16) for _ in range(2))
    back = []
    for pool, x in ((kc, ko), (vc, vo)):
        w = x.clone()
        w[~off] = pool[slots[~off] // 16, :, slots[~off] % 16]
        back.append(w)
    tv.kv_rows_read(geom, slots, kc, vc, ko, vo)
    assert np.array_equal(bits(ko), bits(back[0])) and np.array_equal(bits(vo), bits(back[1]))


def test_rows_of_different_strides():
    """K rows of one array, V rows of another."""
    g = gen(3)
    geom = tv.geom(4, 4, 64)
    k = torch.randn(50, 296, generator=g, device="cuda").to(BF16)[:, 8:264].unflatten(1, (4, 64))
    v = torch.randn(50, 4, 64, generator=g, device="cuda").to(BF16)
    kc, vc = (torch.zeros(4, 4, 16, 64, dtype=BF16, device="cuda") for _ in range(2))
    slots = torch.randperm(64, generator=g, device="cuda")[:50]
    tv.kv_rows_write(geom, k, v, slots, kc, vc)
    ko, vo = torch.zeros(50, 4, 64, dtype=BF16, device="cuda"), torch.zeros(50, 512, dtype=BF16, device="cuda")
    tv.kv_rows_read(geom, slots, kc, vc, ko, vo[:, 256:].unflatten(1, (4, 64)))
    assert torch.equal(ko, k) and torch.equal(vo[:, 256:].unflatten(1, (4, 64)), v) and not vo[:, :256].any()


# ---------------------------------------------------------------- together


def test_refusals_of_tensors():
    p = Pages(random.Random(1), 3, 4, 20)
    d = p.device()
    want = i32([0, 0, 0])
    for bad in (lambda: tv.block_tables(want.long(), d["table"], d["n"], d["free"], d["top"], d["status"]),
                lambda: tv.block_tables(want, d["table"][:2], d["n"], d["free"], d["top"], d["status"]),
                lambda: tv.block_tables(want, d["table"], d["n"][:2], d["free"], d["top"], d["status"]),
                lambda: tv.block_tables(want, d["table"], d["n"], d["free"][::2], d["top"], d["status"]),
                lambda: tv.block_tables(want, d["table"], d["n"], d["free"], d["top"], d["status"][:1]),
                lambda: tv.block_tables(want, d["table"], d["n"], d["free"], d["top"], d["status"], d["released"]),
                lambda: tv.block_tables(want, d["table"], d["n"], d["free"], d["top"], d["status"],
                                        d["released"][:, :3].contiguous(), d["count"]),
                lambda: tv.block_tables(want.cpu(), d["table"], d["n"], d["free"], d["top"], d["status"])):
        with pytest.raises(ValueError):
            bad()
    slots = torch.zeros(4, dtype=torch.int64, device="cuda")
    for bad in (lambda: tv.slot_map(i32([0, 1, 2, 3]), want, d["table"], d["n"], 20, slots.int(), d["status"]),
                lambda: tv.slot_map(i32([0, 1, 2]), want, d["table"], d["n"], 20, slots, d["status"]),
                lambda: tv.slot_map(i32([0, 1, 2, 3]), want, d["table"], d["n"], "20", slots, d["status"]),
                lambda: tv.slot_map(i32([0, 1, 2, 3]), want, d["table"], d["n"], 2 ** 40, slots, d["status"])):
        with pytest.raises(ValueError):
            bad()
    geom = tv.geom(2, 2, 64)
    x = torch.zeros(4, 2, 64, dtype=BF16, device="cuda")
    pool = torch.zeros(2, 2, 16, 64, dtype=BF16, device="cuda")
    for bad in (lambda: tv.kv_rows_write(geom, x.float(), x, slots, pool, pool.clone()),
                lambda: tv.kv_rows_write(geom, x, x[:3], slots, pool, pool.clone()),
                lambda: tv.kv_rows_write(geom, x, x, slots[:3], pool, pool.clone()),
                lambda: tv.kv_rows_write(geom, x, x, slots, pool.to(torch.int8), pool.to(torch.int8)),
                lambda: tv.kv_rows_read(geom, slots.int(), pool, pool.clone(), x, x.clone()),
                lambda: tv.kv_rows_read(geom, slots, pool[:, :1], pool.clone(), x, x.clone())):
        with pytest.raises(ValueError):
            bad()


@pytest.mark.parametrize("capture", [False, True])
def test_pages_slots_rows_and_attention(capture):
    """Pages for new requests and their next tokens, rows written through the slot
    map, attention over them: as over a cache laid out by hand. Captured, the same
    graph serves a second round after all pages went back."""
    g = gen(12)
    hq, hkv, d = 8, 2, 64
    lens = [0, 17, 16, 100, 1]
    batch, rows = len(lens), sum(lens) + 6                # six padded rows
    geom = tv.geom(hq, hkv, d)
    k, v = (torch.randn(rows, hkv, d, generator=g, device="cuda").to(BF16) for _ in range(2))
    q = torch.randn(batch, hq, d, generator=g, device="cuda").to(BF16)
    cu = i32([0] + np.cumsum(lens).tolist())
    seq = i32(lens)
    pool, width = 20, 8
    kc, vc = (torch.full((pool, hkv, 16, d), float("nan"), dtype=BF16, device="cuda") for _ in range(2))
    table, n = torch.full((batch, width), -1, dtype=I32, device="cuda"), torch.zeros(batch, dtype=I32, device="cuda")
    free = torch.randperm(pool, generator=g, device="cuda").to(I32)
    top, status = i32([pool]), torch.zeros(batch, dtype=I32, device="cuda")
    slots = torch.empty(rows, dtype=torch.int64, device="cuda")
    zero = torch.zeros(batch, dtype=I32, device="cuda")
    out, lse = torch.empty_like(q), torch.empty(batch, hq, device="cuda")
    ws = torch.empty(tv.decode_workspace_bytes(geom, batch), dtype=torch.uint8, device="cuda")

    def step():
        tv.block_tables(seq, table, n, free, top, status)
        tv.slot_map(cu, zero, table, n, pool, slots, status)
        tv.kv_rows_write(geom, k, v, slots, kc, vc)
        tv.decode_attention(geom, q, seq, table, n, kc, vc, None, None, out, lse, ws, status)

    if capture:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step()
        run = graph.replay
    else:
        run = step
    for _ in range(2):
        out.fill_(9.0)
        run()
        assert status.tolist() == [0] * batch and n.tolist() == [-(-c // 16) for c in lens]
        assert slots[sum(lens):].tolist() == [-1] * 6
        for b, c in enumerate(lens):
            if c == 0:
                assert not out[b].any()
                continue
            a = sum(lens[:b])
            kd, vd = k[a:a + c].double(), v[a:a + c].double()
            s = torch.einsum("hgd,nhd->hgn", q[b].double().view(hkv, hq // hkv, d), kd) * d ** -0.5
            want = torch.einsum("hgn,nhd->hgd", s.softmax(-1), vd).flatten(0, 1)
            # output rounding 2^-9 of a value below 4, weights and sums far below it
            assert (out[b].double() - want).abs().max() < 2.0 ** -7
        tv.block_tables(zero, table, n, free, top, status)
        assert top.tolist() == [pool] and sorted(free.tolist()) == list(range(pool)) and not (table != -1).any()


def test_two_streams():
    """Calls on two streams work on lists of their own."""
    made = [Pages(random.Random(s), 50, 40, 3000, released=2) for s in (21, 22)]
    devices = [p.device() for p in made]
    wants = [i32([640] * 50), i32([320] * 50)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for d, w, s in zip(devices, wants, streams):
        call(d, w, stream=s)
    torch.cuda.synchronize()
    for d, p, w in zip(devices, made, wants):
        check(d, reference(p, w.tolist()))
