"""Calls from several host threads at once, each on a stream and arrays of its own, whose
launches need different amounts of shared memory."""

import threading

import pytest
import torch

import speculative_decoding_tree_build_gb300 as tv

pytestmark = pytest.mark.gpu

F32, I32 = torch.float32, torch.int32


def together(jobs):
    """Start all jobs at once; the first exception of one of them, if any, is raised."""
    gate, faults = threading.Barrier(len(jobs)), []

    def body(job):
        try:
            gate.wait()
            job()
        except Exception as e:
            faults.append(e)

    threads = [threading.Thread(target=body, args=(job,)) for job in jobs]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    if faults:
        raise faults[0]
    torch.cuda.synchronize()


def i32(x):
    return torch.tensor(x, dtype=I32, device="cuda")


def test_block_tables_of_one_and_of_many_requests():
    sets = []
    for batch in (1, 4096, 37, 4096, 2):
        pool = 2 * batch
        sets.append({"want": i32([32] * batch), "none": i32([0] * batch), "table": torch.full((batch, 2), -1, dtype=I32, device="cuda"),
                     "n": i32([0] * batch), "free": torch.arange(pool, dtype=I32, device="cuda"), "top": i32([pool]),
                     "st": i32([0] * batch), "stream": torch.cuda.Stream()})
    torch.cuda.synchronize()

    def job(s):
        for turn in range(20):
            tv.block_tables(s["none"] if turn % 2 else s["want"], s["table"], s["n"], s["free"], s["top"], s["st"], stream=s["stream"])
        tv.block_tables(s["want"], s["table"], s["n"], s["free"], s["top"], s["st"], stream=s["stream"])

    together([lambda s=s: job(s) for s in sets])
    for s in sets:
        batch = s["n"].numel()
        assert not s["st"].any() and s["top"].tolist() == [0] and bool((s["n"] == 2).all())
        assert torch.equal(s["table"].flatten(), torch.arange(2 * batch - 1, -1, -1, dtype=I32, device="cuda"))


@pytest.mark.parametrize("dtype", [F32, torch.bfloat16])
def test_filters_with_and_without_clusters(dtype):
    sets = []
    for rows, v in ((1, 40000), (700, 9000), (3, 20000), (650, 9000)):
        x = torch.randn(rows, v, device="cuda").to(dtype)
        sets.append({"x": x, "outs": [torch.empty_like(x) for _ in range(3)], "cu": i32([0, rows]), "rows": rows,
                     "t": torch.ones(1, device="cuda"), "p": torch.full((1,), 0.9, device="cuda"), "k": i32([50]),
                     "st": i32([0]), "stream": torch.cuda.Stream()})
    torch.cuda.synchronize()

    def job(s):
        for out in s["outs"]:
            tv.filter_logits(s["x"], s["cu"], s["t"], s["k"], s["p"], None, s["rows"], out, None, s["st"], s["stream"])

    together([lambda s=s: job(s) for s in sets])
    for s in sets:
        want = torch.empty_like(s["x"])
        tv.filter_logits(s["x"], s["cu"], s["t"], s["k"], s["p"], None, s["rows"], want, None, s["st"])
        assert not s["st"].any() and all(torch.equal(out, want) for out in s["outs"])
        assert 1 <= int((want > -float("inf")).sum(-1).min()) and int((want > -float("inf")).sum(-1).max()) <= 50
