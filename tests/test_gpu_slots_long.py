"""Slot maps of requests with very many rows: every row against the restatement, faults
anywhere in them, and time that grows with the rows alone."""

import numpy as np
import pytest
import torch

import speculative_decoding_tree_build_gb300 as tv
from oracle import slot_map_ref

pytestmark = pytest.mark.gpu

I32 = torch.int32


def i32(x):
    return torch.tensor(x, dtype=I32, device="cuda")


def paged(lens, start, seed, spare=0):
    """Requests of `lens` new rows from slot `start` on, their pages anywhere in the pool."""
    need = [-(-(n + s) // 16) for n, s in zip(lens, start)]
    g = torch.Generator().manual_seed(seed)
    ids = torch.randperm(sum(need) + 3, generator=g).to(I32)
    table = torch.full((len(lens), max(max(need), 1)), -1, dtype=I32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = ids[at:at + n]
        at += n
    cu = np.concatenate([[0], np.cumsum(lens)]).astype(np.int64).tolist()
    return {"cu": cu, "start": list(start), "table": table, "n": need, "pool": sum(need) + 3, "rows": cu[-1] + spare}


def call(c, status, slots=None):
    st = i32(status)
    if slots is None:
        slots = torch.full((c["rows"],), -7, dtype=torch.int64, device="cuda")
    tv.slot_map(i32(c["cu"]), i32(c["start"]), c["table"].cuda(), i32(c["n"]), c["pool"], slots, st)
    return slots, st


def check(c, status):
    slots, st = call(c, status)
    want, st_ref = slot_map_ref(c["cu"], c["start"], c["table"].numpy(), c["n"], c["pool"], c["rows"], status)
    assert st.tolist() == st_ref
    assert np.array_equal(slots.cpu().numpy(), want)
    return st_ref


@pytest.mark.parametrize("lens", [[5000001], [300000, 0, 7, 400001, 1], [100] * 3000, [155648], [155649], [160000, 160000]])
@pytest.mark.parametrize("first", [0, 13])
def test_long_requests(lens, first):
    c = paged(lens, [first + b % 5 for b in range(len(lens))], len(lens), spare=3001)
    assert check(c, [0] * len(lens)) == [0] * len(lens)


@pytest.mark.parametrize("where", [0, 1, 12345, -2, -1])
@pytest.mark.parametrize("bad", [-1, "pool", 2 ** 31 - 1])
def test_a_bad_page_anywhere_in_a_long_request(where, bad):
    lens = [250000, 400000, 9, 0, 300000]
    c = paged(lens, [5, 1, 0, 3, 14], 7, spare=17)
    row = c["table"][1, :c["n"][1]]
    row[where] = c["pool"] if bad == "pool" else bad
    assert check(c, [0] * 5) == [0, 8, 0, 0, 0]
    # two at once, one of them in the requests' last one, one flagged before
    c["table"][4, 9000] = -5
    assert check(c, [4, 0, 0, 0, 0]) == [4, 8, 0, 0, 8]
    # a bad page behind the rows is none of theirs
    c = paged(lens, [5, 1, 0, 3, 14], 8)
    c["n"][1] += 1
    c["table"] = torch.cat([c["table"], torch.full((5, 1), -1, dtype=I32)], 1)
    assert check(c, [0] * 5) == [0] * 5


def test_rows_that_several_long_requests_claim():
    """Offsets that run backwards: their requests are flagged, and what a request flagged
    before claims of another one's rows stays with that one."""
    c = paged([400000] * 5, [0, 3, 5, 7, 1], 9)
    c["rows"] = 600000
    c["cu"] = [0, 400000, 100000, 300000, 500000, 600000]
    assert check(c, [0] * 5) == [0, 1, 1, 1, 0]
    assert check(c, [0, 0, 8, 8, 0]) == [0, 1, 8, 8, 0]
    c["table"][0, 20000] = -1
    assert check(c, [0, 0, 8, 8, 0]) == [8, 1, 8, 8, 0]
    c["n"][4] = 3                                   # too few pages
    assert check(c, [0, 8, 8, 0, 0]) == [8, 8, 8, 1, 8]


def test_replayed_with_and_without_a_fault():
    c = paged([200000, 300000, 100000], [3, 0, 9], 10, spare=5)
    cu, start, table, n = i32(c["cu"]), i32(c["start"]), c["table"].cuda(), i32(c["n"])
    slots, st = torch.full((c["rows"],), -7, dtype=torch.int64, device="cuda"), i32([0] * 3)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        tv.slot_map(cu, start, table, n, c["pool"], slots, st)
    for page in (None, 17000, 0, None):
        host = c["table"].clone()
        if page is not None:
            host[1, page] = -1
        table.copy_(host)
        st.zero_()
        slots.fill_(-7)
        graph.replay()
        want, st_ref = slot_map_ref(c["cu"], c["start"], host.numpy(), c["n"], c["pool"], c["rows"], [0] * 3)
        assert st.tolist() == st_ref and np.array_equal(slots.cpu().numpy(), want)


@pytest.mark.parametrize("fault", [False, True])
def test_one_request_of_the_most_rows(fault):
    rows, pages = 2 ** 31 - 1, 2 ** 27
    assert torch.cuda.mem_get_info()[0] > 40 << 30
    table = torch.arange(pages - 1, -1, -1, dtype=I32, device="cuda").view(1, pages)
    if fault:
        table[0, pages // 3] = -1
    slots = torch.empty(rows, dtype=torch.int64, device="cuda")
    st = i32([0])
    tv.slot_map(i32([0, rows]), i32([0]), table, i32([pages]), pages, slots, st)
    assert st.tolist() == [8 if fault else 0]
    for at in range(0, rows, 1 << 27):
        part = slots[at:at + (1 << 27)]
        if fault:
            assert int(part.max()) == int(part.min()) == -1
        else:
            pos = torch.arange(at, at + part.numel(), device="cuda")
            assert torch.equal(part, (pages - 1 - pos // 16) * 16 + pos % 16)


def test_time_does_not_grow_with_a_request_s_share():
    """8.4M rows of one request within four times what they take in 512 requests (every CTA
    used to check all of a request's pages: 1391 us against 31)."""
    times = []
    for lens in ([16384] * 512, [16384 * 512]):
        c = paged(lens, [0] * len(lens), 11)
        cu, start, table, n = i32(c["cu"]), i32(c["start"]), c["table"].cuda(), i32(c["n"])
        slots, st = torch.empty(c["rows"], dtype=torch.int64, device="cuda"), i32([0] * len(lens))
        best = None
        for _ in range(8):
            begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            begin.record()
            for _ in range(10):
                tv.slot_map(cu, start, table, n, c["pool"], slots, st)
            end.record()
            torch.cuda.synchronize()
            best = min(best or 1e9, begin.elapsed_time(end))
        assert not st.any()
        times.append(best)
    assert times[1] <= 4 * times[0], times
