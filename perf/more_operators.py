"""Measured cases of the operators around a serving step: block tables grown
and shrunk on the GPU, slot maps, bf16 rows written to and read from slots of
the paged cache, sampling with temperature, top-k, top-p and min-p, and the
same filter as masked logits.

``run`` takes one pass through an operator. With ``own`` false it is the plain
form: elementary torch operations in 32 bits (the filter's weights and sums in
64, since a token is kept or not by a comparison of sums). With ``own`` true it
is the library's call. ``exact`` restates the operator's definition in 64 bits.
"""

import math

import torch

own = False

PAGE = 16                      # slots per page of the paged cache
NO_BLOCKS = 128                # status: the free list was too short for the request
TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
# (temperature, top_k, top_p, min_p) of a batch whose requests ask for different things
MIX = [(0.8, 50, 1.0, 0.0), (1.0, 0, 0.95, 0.0), (1.2, 0, 1.0, 0.05), (0.0, 0, 1.0, 0.0),
       (0.7, 200, 0.9, 0.02), (1.0, 0, 1.0, 0.0)]
PIECE = 1 << 24                # logits that the plain form works on at a time


# ------------------------------------------------------------------- cases


def listed():
    return [
        # pages for the trees of 64 ragged sequences, after those of the last step went back
        {"name": "tables-step", "op": "tables", "batch": 64, "held_lo": 4096, "held_hi": 32768,
         "new_lo": 17, "new_hi": 129, "released": 4, "short": False},
        # pages for 64 whole prompts
        {"name": "tables-prompts", "op": "tables", "batch": 64, "held_lo": 0, "held_hi": 0,
         "new_lo": 4096, "new_hi": 32768, "released": 0, "short": False},
        # slots of the nodes of 64 trees
        {"name": "slots-step", "op": "slots", "batch": 64, "held_lo": 4096, "held_hi": 32768,
         "new_lo": 17, "new_hi": 129, "empty": 0, "spare": 50},
        # slots of 64 whole prompts, two of them without new rows
        {"name": "slots-prompts", "op": "slots", "batch": 64, "held_lo": 0, "held_hi": 0,
         "new_lo": 4096, "new_hi": 32768, "empty": 2, "spare": 0},
        # the rows that 32 sequences accepted, gathered for an 8-bit cache
        {"name": "rows-accepted", "op": "rows", "to": "read", "rows": 160, "hkv": 8, "d": 128,
         "padded": 32, "fused": False},
        # four whole prompts written to the bf16 pools
        {"name": "rows-prompts", "op": "rows", "to": "write", "rows": 32381, "hkv": 8, "d": 128,
         "padded": 0, "fused": True},
        # the next token of eight sequences: call latency counts
        {"name": "sample-step", "op": "sample", "batch": 8, "lo": 1, "hi": 1, "vocab": 32000,
         "type": "fp32", "t": 0.8, "k": 50, "p": 0.95, "m": 0.0, "mix": False, "flat": 0,
         "masked": 0.0},
        # 64 sequences, bf16 logits over a large vocabulary, top-p alone
        {"name": "sample-batch", "op": "sample", "batch": 64, "lo": 1, "hi": 1, "vocab": 151936,
         "type": "bf16", "t": 0.9, "k": 0, "p": 0.9, "m": 0.0, "mix": False, "flat": 8,
         "masked": 0.0},
        # every node of 32 trees, requests with settings of their own
        {"name": "sample-trees", "op": "sample", "batch": 32, "lo": 65, "hi": 65, "vocab": 32000,
         "type": "fp32", "t": 1.0, "k": 0, "p": 1.0, "m": 0.0, "mix": True, "flat": 8,
         "masked": 0.0},
        # every node of 16 large trees over a large vocabulary
        {"name": "sample-large", "op": "sample", "batch": 16, "lo": 257, "hi": 257,
         "vocab": 151936, "type": "fp32", "t": 0.8, "k": 64, "p": 0.95, "m": 0.0, "mix": False,
         "flat": 8, "masked": 0.0},
        # the target's distribution for rejection sampling along paths of eight small trees
        {"name": "filter-trees", "op": "filter", "batch": 8, "lo": 41, "hi": 41, "vocab": 32000,
         "type": "fp32", "t": 0.8, "k": 0, "p": 0.95, "m": 0.02, "mix": False, "flat": 8,
         "masked": 0.0},
        # ragged trees over a large vocabulary in bf16, requests with settings of their own
        {"name": "filter-ragged", "op": "filter", "batch": 24, "lo": 17, "hi": 129,
         "vocab": 151936, "type": "bf16", "t": 1.0, "k": 0, "p": 1.0, "m": 0.0, "mix": True,
         "flat": 8, "masked": 0.0},
    ]


def _log(rng, lo, hi):
    """An integer spread evenly over the logarithm of [lo, hi]."""
    return min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    op = rng.choice(["tables", "slots", "rows", "sample", "sample", "sample", "filter", "filter"])
    if op in ("tables", "slots"):
        batch = _log(rng, 1, 512)
        most = 2000000 // batch                     # slots of a sequence
        held_hi = rng.choice([0, _log(rng, 1, min(most, 60000))])
        new_hi = _log(rng, 1, min(most, 60000))
        case = {"op": op, "batch": batch, "held_lo": rng.randint(0, held_hi), "held_hi": held_hi,
                "new_lo": _log(rng, 1, new_hi), "new_hi": new_hi}
        if op == "tables":
            case.update(released=rng.choice([0, 0, 1, 7]), short=rng.random() < 0.3)
        else:
            case.update(empty=rng.randint(0, 2) if batch > 2 else 0,
                        spare=rng.choice([0, 1, 77]))
        return case
    if op == "rows":
        hkv, d = rng.choice([1, 2, 3, 4, 8, 8, 16]), rng.choice([64, 128])
        return {"op": op, "to": rng.choice(["read", "write"]), "hkv": hkv, "d": d,
                "rows": _log(rng, 1, 32000000 // (hkv * d)), "padded": rng.choice([0, 1, 19]),
                "fused": rng.random() < 0.5}
    vocab = rng.choice([32000, 151936, _log(rng, 50, 200000), _log(rng, 2000, 200000)])
    rows = _log(rng, 1, min(20000, 300000000 // vocab))
    hi = min(_log(rng, 1, 257), rows)
    return {"op": op, "batch": max(1, rows // hi), "lo": _log(rng, 1, hi), "hi": hi,
            "vocab": vocab, "type": rng.choice(["fp32", "bf16"]),
            "t": round(rng.uniform(0.5, 1.5), 2),
            "k": rng.choice([0, 0, 1, 20, 50, 1000, _log(rng, 1, 2 * vocab)]),
            "p": rng.choice([1.0, 0.5, 0.9, 0.95, 0.99, round(rng.uniform(0.05, 1.0), 3)]),
            "m": rng.choice([0.0, 0.0, 0.02, 0.1, round(rng.uniform(0.001, 0.5), 3)]),
            "mix": rng.random() < 0.4, "flat": rng.choice([0, 1, 8]),
            "masked": rng.choice([0.0, 0.0, 0.0, 0.5, 0.999])}


def _ragged(batch, lo, hi, empty=0):
    """`batch` lengths from lo to hi, spread over their logarithm (the first
    `empty` of them none at all)."""
    base = max(lo, 1)
    at = [i / (batch - 1) for i in range(batch)] if batch > 1 else [1.0]
    got = [round(base * (max(hi, 1) / base) ** x) for x in at]
    got = [min(hi, max(lo, n)) for n in got]
    return [0] * min(empty, batch) + got[min(empty, batch):]


def _spans(case):
    """(slots held before, slots to come) of each sequence."""
    old = _ragged(case["batch"], case["held_lo"], case["held_hi"])[::-1]
    return old, _ragged(case["batch"], case["new_lo"], case["new_hi"], case.get("empty", 0))


def _pages_of(slots):
    return -(-slots // PAGE)


def _settings(case):
    """Each request's (temperature, top_k, top_p, min_p)."""
    if case["mix"]:
        return [MIX[b % len(MIX)] for b in range(case["batch"])]
    return [(case["t"], case["k"], case["p"], case["m"])] * case["batch"]


# ------------------------------------------------------------------- inputs


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 2654435761 % (1 << 62) + 29)
    return g


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _logits(g, rows, case):
    """Rows as a language model gives them: a broad bulk and a few dozen likely
    tokens above it, every `flat`-th row the bulk alone (no idea what comes).
    A share `masked` of the tokens is not allowed (a grammar's mask)."""
    vocab = case["vocab"]
    ld = -(-vocab // 8) * 8                        # rows start on 16 bytes
    x = torch.randn(rows, ld, generator=g, device="cuda").mul_(2.0)
    likely = min(40, vocab)
    at = torch.randint(0, vocab, (rows, likely), generator=g, device="cuda")
    up = 14.0 * torch.rand(rows, likely, generator=g, device="cuda") ** 2 + 2.0
    if case["flat"]:
        up[torch.arange(rows, device="cuda") % case["flat"] == case["flat"] - 1] = 0.0
    x.scatter_add_(1, at, up)
    if case["masked"]:
        mask = torch.rand(rows, ld, generator=g, device="cuda") < case["masked"]
        mask.scatter_(1, at[:, :1], False)
        x.masked_fill_(mask, -math.inf)
    return x.to(TYPES[case["type"]])[:, :vocab]


def prepare(case, seed):
    g = _gen(seed)
    s = {"case": case}
    if case["op"] in ("tables", "slots"):
        old, new = _spans(case)
        at = torch.randperm(case["batch"], generator=torch.Generator().manual_seed(int(seed))).tolist()
        old, new = [old[i] for i in at], [new[i] for i in at]
        ends = [a + b for a, b in zip(old, new)]
        have = [_pages_of(n) for n in (old if case["op"] == "tables" else ends)]
        grow = sum(_pages_of(e) - h for e, h in zip(ends, have))
        back = case.get("released", 0) * case["batch"]
        if case.get("short"):
            grow = max(grow // 2 - back, 0)        # half of what is asked for
        pool = sum(have) + grow + back + 5
        order = torch.randperm(pool, generator=g, device="cuda").to(torch.int32)
        width = max(_pages_of(max(ends)), case.get("released", 0), 1)
        counts = _i32(have)
        s["table"] = torch.full((case["batch"], width), -1, dtype=torch.int32, device="cuda")
        s["table"][torch.arange(width, device="cuda")[None] < counts[:, None]] = order[:sum(have)]
        s["n_blocks"], s["pool"] = counts, pool
        s["old"], s["end"] = _i32(old), _i32(ends)
        s["status"] = torch.zeros(case["batch"], dtype=torch.int32, device="cuda")
        if case["op"] == "slots":
            cu = [0]
            for n in new:
                cu.append(cu[-1] + n)
            s["cu"] = _i32(cu)
            s["slots"] = torch.empty(cu[-1] + case["spare"], dtype=torch.int64, device="cuda")
            return s
        # pages that the last commit took off the tables
        s["released"] = torch.full_like(s["table"], -1)
        s["released"][:, :case["released"]] = order[sum(have):sum(have) + back].view(case["batch"], -1)
        s["released_count"] = _i32([case["released"]] * case["batch"])
        free = order[sum(have) + back:]
        s["free"] = torch.full((pool,), -1, dtype=torch.int32, device="cuda")
        s["free"][:free.numel()] = free
        s["free_count"] = _i32([free.numel()])
        return s
    if case["op"] == "rows":
        rows, hkv, d = case["rows"], case["hkv"], case["d"]
        blocks = _pages_of(rows) + 40
        # slots of whole pages in order, the pages anywhere; some rows without a slot
        page = torch.randperm(blocks, generator=g, device="cuda")[:_pages_of(rows)]
        slots = (page[:, None] * PAGE + torch.arange(PAGE, device="cuda")).flatten()[:rows]
        if case["padded"]:
            slots[torch.randint(0, rows, (min(case["padded"], rows // 2),), generator=g, device="cuda")] = -1
        s["slots"] = slots
        if case["to"] == "write":
            n = hkv * d
            if case["fused"]:                      # slices of one fused projection's output
                kv = torch.randn(rows, 2 * n, generator=g, device="cuda").bfloat16()
                k, v = kv[:, :n], kv[:, n:]
            else:
                k, v = (torch.randn(rows, n, generator=g, device="cuda").bfloat16() for _ in range(2))
            s["k_new"], s["v_new"] = k.unflatten(1, (hkv, d)), v.unflatten(1, (hkv, d))
            s["k"], s["v"] = (torch.zeros(blocks, hkv, PAGE, d, dtype=torch.bfloat16, device="cuda")
                              for _ in range(2))
        else:
            s["k"], s["v"] = (torch.randn(blocks, hkv, PAGE, d, generator=g, device="cuda").bfloat16()
                              for _ in range(2))
            s["k_out"], s["v_out"] = (torch.zeros(rows, hkv, d, dtype=torch.bfloat16, device="cuda")
                                      for _ in range(2))
        if own:
            import speculative_decoding_tree_build_gb300 as tv
            s["geom"] = tv.geom(hkv, hkv, d)
        return s
    nodes = _ragged(case["batch"], case["lo"], case["hi"])
    cu = [0]
    for n in nodes:
        cu.append(cu[-1] + n)
    rows = cu[-1]
    s["cu"], s["max_nodes"] = _i32(cu), case["hi"]
    s["logits"] = _logits(g, rows, case)
    asked = _settings(case)
    s["rows_of"] = []
    for setting in sorted(set(asked)):
        at = [r for b, got in enumerate(asked) if got == setting for r in range(cu[b], cu[b + 1])]
        s["rows_of"].append((setting, torch.tensor(at, device="cuda")))
    t, k, p, m = zip(*asked)
    s["t"] = torch.tensor(t, dtype=torch.float32, device="cuda")
    s["top_k"] = _i32(list(k))
    s["top_p"] = torch.tensor(p, dtype=torch.float32, device="cuda")
    s["min_p"] = torch.tensor(m, dtype=torch.float32, device="cuda")
    s["status"] = torch.zeros(case["batch"], dtype=torch.int32, device="cuda")
    if case["op"] == "sample":
        ld = -(-case["vocab"] // 4) * 4
        u = torch.rand(rows, ld, generator=g, device="cuda").clamp_(2.0 ** -25, 1 - 2.0 ** -24)
        s["gumbel"] = u.log_().neg_().log_().neg_()[:, :case["vocab"]]
        s["tokens"] = torch.empty(rows, dtype=torch.int32, device="cuda")
        s["logp"] = torch.empty(rows, device="cuda")
    else:
        ld = -(-case["vocab"] // 8) * 8
        s["out"] = torch.empty(rows, ld, dtype=s["logits"].dtype, device="cuda")[:, :case["vocab"]]
        s["kept"] = torch.empty(rows, dtype=torch.int32, device="cuda")
    return s


# ------------------------------------------------------------------- one pass


def run(s):
    return {"tables": _tables, "slots": _slots, "rows": _rows, "sample": _sample,
            "filter": _filter}[s["case"]["op"]](s)


def _tables(s):
    """The pages of the last step's trees go back, those of the next are taken
    (what the second call takes, the first one of the next pass returns)."""
    if own:
        import speculative_decoding_tree_build_gb300 as tv
        tv.block_tables(s["old"], s["table"], s["n_blocks"], s["free"], s["free_count"], s["status"],
                        s["released"], s["released_count"])
        tv.block_tables(s["end"], s["table"], s["n_blocks"], s["free"], s["free_count"], s["status"])
    else:
        _set_tables(s, s["old"], True)
        _set_tables(s, s["end"], False)
    return {"table": s["table"], "n_blocks": s["n_blocks"], "free": s["free"],
            "free_count": s["free_count"], "status": s["status"]}


def _push(s, ids):
    """Put `ids` on the list so that taking them off again starts with the first."""
    at = s["free_count"].long() + torch.arange(ids.numel(), device="cuda")
    s["free"][at] = ids.flip(0)
    s["free_count"] += ids.numel()


def _set_tables(s, want, released):
    good = s["status"] == 0
    column = torch.arange(s["table"].shape[1], device="cuda")[None]
    if released:
        take = (column < s["released_count"][:, None]) & good[:, None]
        _push(s, s["released"][take])
        s["released_count"][good] = 0
    need = (want + PAGE - 1) // PAGE
    drop = (column >= need[:, None]) & (column < s["n_blocks"][:, None]) & good[:, None]
    _push(s, s["table"][drop])
    s["table"][drop] = -1
    add = torch.where(good, (need - s["n_blocks"]).clamp(min=0), 0)
    fits = (add == 0) | (torch.cumsum(add, 0) <= s["free_count"])
    s["status"][~fits] |= NO_BLOCKS
    fill = (column >= s["n_blocks"][:, None]) & (column < need[:, None]) & (good & fits)[:, None]
    number = torch.cumsum(fill.flatten(), 0).view(fill.shape) - 1
    s["table"][fill] = s["free"][(s["free_count"] - 1 - number[fill])]
    s["free_count"] -= fill.sum()
    s["n_blocks"].copy_(torch.where(good & fits, need, s["n_blocks"]))


def _slots(s):
    if own:
        import speculative_decoding_tree_build_gb300 as tv
        tv.slot_map(s["cu"], s["old"], s["table"], s["n_blocks"], s["pool"], s["slots"], s["status"])
    else:
        row = torch.arange(s["slots"].shape[0], device="cuda")
        seq = torch.searchsorted(s["cu"].long(), row, right=True) - 1
        here = seq < s["old"].shape[0]
        seq = seq.clamp(max=s["old"].shape[0] - 1)
        slot = torch.where(here, s["old"].long()[seq] + row - s["cu"].long()[seq], 0)
        page = s["table"].long()[seq, slot // PAGE]
        s["slots"].copy_(torch.where(here, page * PAGE + slot % PAGE, -1))
    return {"slots": s["slots"], "status": s["status"]}


def _rows(s):
    write = s["case"]["to"] == "write"
    if own:
        import speculative_decoding_tree_build_gb300 as tv
        if write:
            tv.kv_rows_write(s["geom"], s["k_new"], s["v_new"], s["slots"], s["k"], s["v"])
        else:
            tv.kv_rows_read(s["geom"], s["slots"], s["k"], s["v"], s["k_out"], s["v_out"])
    else:
        row = (s["slots"] >= 0).nonzero().flatten()
        page, at = s["slots"][row] // PAGE, s["slots"][row] % PAGE
        for name in ("k", "v"):
            if write:
                s[name][page, :, at] = s[name + "_new"][row]
            else:
                s[name + "_out"][row] = s[name][page, :, at]
    return {n: s[n] for n in (("k", "v") if write else ("k_out", "v_out"))}


def _pieces(s):
    """(settings, rows that have them) in pieces of at most PIECE logits."""
    for setting, rows in s["rows_of"]:
        for part in rows.split(max(1, PIECE // s["case"]["vocab"])):
            yield setting, part


def _keep(x, setting):
    """Which entries of the rows a request's settings keep, and their weights
    and scaled logits in the vocabulary's order."""
    t, k, p, m = setting
    value, order = torch.sort(x, dim=-1, descending=True, stable=True)
    inv = torch.tensor(1.0, device="cuda") / torch.tensor(t, dtype=torch.float32, device="cuda")
    scaled = value * inv
    weight = torch.exp(scaled.double() - scaled[:, :1].double())
    keep = value > -math.inf
    if 0 < k < x.shape[-1]:
        keep[:, k:] = False
    if p < 1:
        weight = torch.where(keep, weight, 0.0)
        upto = torch.cumsum(weight, -1)
        keep &= upto - weight < torch.tensor(p, dtype=torch.float32).double().item() * upto[:, -1:]
        keep[:, 0] = True
    if m > 0:
        least = torch.tensor(m, dtype=torch.float32).double().log().item()
        keep &= scaled.double() - scaled[:, :1].double() >= least
    return torch.zeros_like(keep).scatter_(-1, order, keep), scaled[:, 0], x * inv


def _sample(s):
    if own:
        import speculative_decoding_tree_build_gb300 as tv
        tv.sample_filtered(s["logits"], s["gumbel"], s["cu"], s["t"], s["top_k"], s["top_p"],
                           s["min_p"], s["max_nodes"], s["tokens"], s["logp"], s["status"])
        return {"tokens": s["tokens"], "logp": s["logp"], "status": s["status"]}
    for setting, rows in _pieces(s):
        x = s["logits"][rows].float()
        if setting[0] == 0:
            s["tokens"][rows] = x.argmax(-1).to(torch.int32)
            s["logp"][rows] = 0.0
            continue
        keep, top, scaled = _keep(x, setting)
        token = torch.where(keep, scaled + s["gumbel"][rows], -math.inf).argmax(-1)
        far = scaled.double() - top.double()[:, None]
        total = torch.where(keep, far.exp(), 0.0).sum(-1)
        s["tokens"][rows] = token.to(torch.int32)
        s["logp"][rows] = (far.gather(1, token[:, None])[:, 0] - total.log()).float()
    return {"tokens": s["tokens"], "logp": s["logp"], "status": s["status"]}


def _filter(s):
    if own:
        import speculative_decoding_tree_build_gb300 as tv
        tv.filter_logits(s["logits"], s["cu"], s["t"], s["top_k"], s["top_p"], s["min_p"],
                         s["max_nodes"], s["out"], s["kept"], s["status"])
        return {"out": s["out"], "kept": s["kept"], "status": s["status"]}
    for setting, rows in _pieces(s):
        x = s["logits"][rows].float()
        if setting[0] == 0:
            keep = torch.zeros_like(x, dtype=torch.bool).scatter_(1, x.argmax(-1, keepdim=True), True)
        else:
            keep = _keep(x, setting)[0]
        s["out"][rows] = torch.where(keep, x, -math.inf).to(s["out"].dtype)
        s["kept"][rows] = keep.sum(-1).to(torch.int32)
    return {"out": s["out"], "kept": s["kept"], "status": s["status"]}


# ------------------------------------------------------------------- what a pass needs


def work(case):
    batch = case["batch"] if "batch" in case else 0
    if case["op"] in ("tables", "slots"):
        old, new = _spans(case)
        grow = sum(_pages_of(a + b) - _pages_of(a) for a, b in zip(old, new))
        if case["op"] == "tables":
            # every block that goes back and is taken again: an id read, an id written, twice;
            # what a request has and wants, what it gets
            return {"bytes": 16 * grow + 8 * case["released"] * batch + 2 * 16 * batch + 8, "flops": 0}
        rows = sum(new)
        return {"bytes": 8 * (rows + case["spare"]) + 4 * (grow + batch) + 16 * batch, "flops": 0}
    if case["op"] == "rows":
        return {"bytes": case["rows"] * (8 + 2 * 2 * case["hkv"] * case["d"] * 2), "flops": 0}
    nodes = _ragged(batch, case["lo"], case["hi"])
    size = 2 if case["type"] == "bf16" else 4
    entries = sum(nodes) * case["vocab"]
    if case["op"] == "filter":
        return {"bytes": 2 * entries * size + sum(nodes) * 4, "flops": entries}
    # the noise of a whole row is needed where nothing is filtered
    bare = sum(n for n, (t, k, p, m) in zip(nodes, _settings(case))
               if t > 0 and not 0 < k < case["vocab"] and p >= 1 and m == 0) * case["vocab"]
    return {"bytes": entries * size + bare * 4 + sum(nodes) * 8, "flops": entries + bare}


# ------------------------------------------------------------------- in 64 bits


def exact(case, seed):
    with torch.no_grad():
        s = prepare(case, seed)
        return {"tables": _exact_tables, "slots": _exact_slots, "rows": _exact_rows,
                "sample": _exact_kept, "filter": _exact_kept}[case["op"]](s, case)


def _exact_tables(s, case):
    """A list and its requests, one after the other."""
    old, end, n = s["old"].tolist(), s["end"].tolist(), s["n_blocks"].tolist()
    table = [row[:c] for row, c in zip(s["table"].tolist(), n)]
    count = s["free_count"].item()
    free, behind = s["free"].tolist()[:count], s["free"].tolist()[count:]
    for row, c in zip(reversed(s["released"].tolist()), reversed(s["released_count"].tolist())):
        free += reversed(row[:c])
    high = len(free)
    status = [0] * case["batch"]
    full = list(free)
    refused = False
    for b in range(case["batch"]):
        add = _pages_of(end[b]) - len(table[b])
        if add <= 0:
            continue
        refused = refused or add > len(free)
        if refused:
            status[b] = NO_BLOCKS
            continue
        for _ in range(add):
            table[b].append(free.pop())
    width = s["table"].shape[1]
    return {"table": torch.tensor([r + [-1] * (width - len(r)) for r in table]),
            "n_blocks": torch.tensor([len(r) for r in table]),
            "free": torch.tensor((full + behind[high - count:])),
            "free_count": torch.tensor([len(free)]), "status": torch.tensor(status)}


def _exact_slots(s, case):
    cu, old, table = s["cu"].tolist(), s["old"].tolist(), s["table"].tolist()
    got = []
    for b in range(case["batch"]):
        got += [table[b][i // PAGE] * PAGE + i % PAGE for i in range(old[b], old[b] + cu[b + 1] - cu[b])]
    got += [-1] * (s["slots"].numel() - len(got))
    return {"slots": torch.tensor(got), "status": torch.zeros(case["batch"], dtype=torch.int64)}


def _exact_rows(s, case):
    slots = s["slots"].tolist()
    row = torch.tensor([i for i, n in enumerate(slots) if n >= 0], dtype=torch.int64, device="cuda")
    slot = torch.tensor([n for n in slots if n >= 0], dtype=torch.int64, device="cuda")
    got = {}
    for name in ("k", "v"):
        by_slot = s[name].double().transpose(1, 2).flatten(0, 1)       # [slots][hkv][d]
        if case["to"] == "write":
            by_slot = by_slot.index_copy(0, slot, s[name + "_new"].double().index_select(0, row))
            got[name] = by_slot.unflatten(0, (-1, PAGE)).transpose(1, 2).contiguous()
        else:
            out = torch.zeros_like(s[name + "_out"], dtype=torch.float64)
            got[name + "_out"] = out.index_copy(0, row, by_slot.index_select(0, slot))
    return got


def _exact_kept(s, case):
    """The place where the kept entries end, found bit by bit in the order of
    (logit, index) without sorting."""
    vocab = case["vocab"]
    width = max(1, (vocab - 1).bit_length())
    index = torch.arange(vocab, device="cuda")
    total = s["logits"].shape[0]
    if case["op"] == "filter":
        got = {"out": torch.empty(total, vocab, device="cuda"),
               "kept": torch.empty(total, dtype=torch.int64, device="cuda")}
    else:
        got = {"tokens": torch.empty(total, dtype=torch.int64, device="cuda"),
               "logp": torch.empty(total, dtype=torch.float64, device="cuda")}
    for (t, k, p, m), rows in _pieces(s):
        x = s["logits"][rows].double()
        bits = x.float().where(x != 0, 0.0).view(torch.int32).long()
        key = torch.where(bits < 0, -1 - (bits & 0x7FFFFFFF), bits) + (1 << 31)
        place = (key << width) + ((1 << width) - 1 - index)            # the larger, the earlier
        if t == 0:
            scaled = x
            keep = place == place.amax(-1, keepdim=True)
        else:
            inv = (torch.ones((), device="cuda") / torch.tensor(t, dtype=torch.float32, device="cuda"))
            scaled = (x.float() * inv).double()                        # the definition's rounding
            far = scaled - scaled.amax(-1, keepdim=True)
            weight = far.exp()
            keep = x > -math.inf

            def end(amount, target):
                """The last place up to which `amount` has to be summed to reach target."""
                cut = torch.zeros(x.shape[0], 1, dtype=torch.int64, device="cuda")
                for bit in reversed(range(32 + width)):
                    trial = cut + (1 << bit)
                    reached = torch.where(place >= trial, amount, 0).sum(-1, keepdim=True)
                    cut = torch.where(reached >= target, trial, cut)
                return cut

            if 0 < k < vocab:
                keep &= place >= end(torch.ones_like(weight), k)
            if p < 1:
                weight = torch.where(keep, weight, 0.0)
                share = float(torch.tensor(p, dtype=torch.float32))
                keep &= place >= end(weight, share * weight.sum(-1, keepdim=True))
            if m > 0:
                keep &= far >= math.log(float(torch.tensor(m, dtype=torch.float32)))
        if case["op"] == "filter":
            got["out"][rows] = torch.where(keep, x, -math.inf).to(torch.float32)
            got["kept"][rows] = keep.sum(-1)
        elif t == 0:
            got["tokens"][rows], got["logp"][rows] = x.argmax(-1), 0.0
        else:
            token = torch.where(keep, scaled.float() + s["gumbel"][rows], -math.inf).argmax(-1)
            got["tokens"][rows] = token
            got["logp"][rows] = (far.gather(1, token[:, None])[:, 0] -
                                 torch.where(keep, far, -math.inf).logsumexp(-1))
    got["status"] = torch.zeros(case["batch"], dtype=torch.int64)
    return got
