"""Measured cases of the decode-step operators: rotary positions with several
axes, the 8-bit paged KV cache (written, read back) and attention of one new
token over a paged cache.

``run`` takes one pass through an operator. With ``own`` false it is the plain
form: elementary torch operations in 32 bits (angles in 64) on the same data.
With ``own`` true it is the library's call. ``exact`` restates the operator's
definition in 64 bits.
"""

import math

import torch

own = False

PAGE = 16                      # slots per page of the paged cache
E4M3_MAX, INT8_MAX = 448.0, 127.0
TINY = 2.0 ** -100             # floor of a row's largest magnitude / of an e4m3 scale
HELD = {"bf16": torch.bfloat16, "fp32": torch.float32, "e4m3": torch.float8_e4m3fn,
        "int8": torch.int8}


# ------------------------------------------------------------------- cases


def listed():
    return [
        # one decode step's new tokens of eight sequences: call latency counts
        {"name": "rope-step", "op": "rope", "rows": 8, "hq": 32, "hkv": 8, "d": 128, "type": "bf16",
         "style": 1, "order": 0, "s0": 16, "s1": 24, "s2": 24, "far": 32768, "fused": True},
        # one image of 37 x 37 patches in a vision encoder: rows and columns, no time
        {"name": "rope-image", "op": "rope", "rows": 1369, "hq": 16, "hkv": 16, "d": 80,
         "type": "fp32", "style": 1, "order": 0, "s0": 20, "s1": 20, "s2": 0, "far": 0,
         "fused": False},
        # a video prompt late in a long conversation: time, height, width in turn
        {"name": "rope-video", "op": "rope", "rows": 16201, "hq": 32, "hkv": 8, "d": 128,
         "type": "bf16", "style": 0, "order": 1, "s0": 24, "s1": 20, "s2": 20, "far": 1000000,
         "fused": True},
        # the new token of each of 64 sequences written to the cache
        {"name": "append-step", "op": "append", "batch": 64, "lo": 1, "hi": 1, "empty": 0,
         "held_lo": 4096, "held_hi": 32768, "hkv": 8, "d": 128, "held": "e4m3", "fused": True},
        # ragged prompt chunks (continuous batching), one sequence without new rows
        {"name": "append-ragged", "op": "append", "batch": 13, "lo": 1, "hi": 2500, "empty": 1,
         "held_lo": 0, "held_hi": 5000, "hkv": 8, "d": 64, "held": "int8", "fused": False},
        # whole prompts of four sequences
        {"name": "append-prompt", "op": "append", "batch": 4, "lo": 8000, "hi": 8191, "empty": 0,
         "held_lo": 0, "held_hi": 0, "hkv": 8, "d": 128, "held": "e4m3", "fused": True},
        # the rows that a step added, read back beside rows that were read before
        {"name": "read-step", "op": "read", "batch": 8, "lo": 1, "hi": 41, "empty": 0,
         "held_lo": 512, "held_hi": 2048, "hkv": 8, "d": 128, "held": "int8"},
        # one layer's whole cache read back for tree verification
        {"name": "read-layer", "op": "read", "batch": 32, "lo": 1024, "hi": 8192, "empty": 0,
         "held_lo": 0, "held_hi": 0, "hkv": 8, "d": 128, "held": "e4m3"},
        # eight short sequences: launch and split cost against 37 MB of cache
        {"name": "decode-short", "op": "decode", "batch": 8, "lo": 512, "hi": 2048, "empty": 0,
         "hq": 32, "hkv": 8, "d": 128, "held": "bf16"},
        # one long sequence: the length has to be split to fill the card
        {"name": "decode-one", "op": "decode", "batch": 1, "lo": 32768, "hi": 32768, "empty": 0,
         "hq": 32, "hkv": 8, "d": 128, "held": "bf16"},
        # eight query heads to a cached head
        {"name": "decode-wide", "op": "decode", "batch": 16, "lo": 2048, "hi": 4096, "empty": 0,
         "hq": 64, "hkv": 8, "d": 128, "held": "int8"},
        # a serving batch of ragged long sequences: bandwidth and balance
        {"name": "decode-ragged", "op": "decode", "batch": 64, "lo": 4096, "hi": 32768, "empty": 0,
         "hq": 32, "hkv": 8, "d": 128, "held": "e4m3"},
    ]


def _log(rng, lo, hi):
    """An integer spread evenly over the logarithm of [lo, hi]."""
    return min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    op = rng.choice(["rope", "append", "read", "decode", "decode"])
    if op == "rope":
        d = rng.choice([32, 64, 72, 80, 96, 128, 128, 256])
        hq = _log(rng, 1, 64)
        hkv = rng.choice([h for h in range(1, hq + 1) if hq % h == 0])
        half = d // 2
        s0 = rng.choice([half, half // 2, half // 4])
        s1 = rng.randint(0, (half - s0) // 2)
        s2 = rng.randint(0, half - s0 - s1) if s1 else 0
        rows = _log(rng, 1, max(1, 60000000 // ((hq + hkv) * d)))
        return {"op": op, "rows": rows, "hq": hq, "hkv": hkv, "d": d,
                "type": rng.choice(["bf16", "bf16", "fp32"]), "style": rng.randint(0, 1),
                "order": rng.randint(0, 1), "s0": s0, "s1": s1, "s2": s2,
                "far": _log(rng, 1, 4000000), "fused": rng.random() < 0.5}
    batch = _log(rng, 1, 96)
    hkv = rng.choice([1, 2, 3, 4, 5, 8, 8, 16])
    d = rng.choice([64, 128])
    empty = rng.randint(0, 2) if batch > 2 else 0
    # rows of all sequences together, by cost: at most a quarter of the largest listed case
    most = max(1, int(220000000 / (hkv * d * (batch + 1))))
    hi = _log(rng, 1, max(1, min(most, 65536)))
    lo = _log(rng, 1, hi)
    case = {"op": op, "batch": batch, "lo": lo, "hi": hi, "empty": empty, "hkv": hkv, "d": d}
    if op == "decode":
        case["hq"] = hkv * rng.choice([1, 2, 3, 4, 4, 5, 7, 8, 8, 12, 16])
        case["held"] = rng.choice(["bf16", "e4m3", "int8"])
        return case
    held_hi = rng.choice([0, _log(rng, 1, 20000 // batch + 1)])
    case.update(held=rng.choice(["e4m3", "int8"]), held_hi=held_hi,
                held_lo=rng.randint(0, held_hi))
    if op == "append":
        case["fused"] = rng.random() < 0.5
    return case


def _ragged(batch, lo, hi, empty=0):
    """`batch` lengths from lo to hi, spread over their logarithm (the first
    `empty` of them none at all)."""
    base = max(lo, 1)
    at = [i / (batch - 1) for i in range(batch)] if batch > 1 else [1.0]
    got = [round(base * (max(hi, 1) / base) ** x) for x in at]
    got = [min(hi, max(lo, n)) for n in got]
    return [0] * min(empty, batch) + got[min(empty, batch):]


def _spans(case):
    """(slots held before, slots the call is about) of each sequence."""
    new = _ragged(case["batch"], case["lo"], case["hi"], case["empty"])
    old = _ragged(case["batch"], case.get("held_lo", 0), case.get("held_hi", 0))[::-1]
    return old, new


# ------------------------------------------------------------------- inputs


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 2654435761 % (1 << 62) + 17)
    return g


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _quantise(x, held):
    """(codes, scales) of rows [..., D]: the cache's definition, in float32."""
    top = x.abs().amax(-1, keepdim=True)
    if held == "e4m3":
        # top = m 2^e with m in [0.5, 1): the smallest 2^n with top / 2^n <= 448 = 0.875 * 2^9
        m, e = torch.frexp(top.clamp(min=TINY))
        e = torch.where(m > 0.875, e - 8, e - 9).clamp(min=-100)
        scale = ((e + 127) << 23).view(torch.float32)
        code = (x / scale).to(torch.float8_e4m3fn)
    else:
        top = top.clamp(min=TINY)
        scale = top / torch.full_like(top, INT8_MAX)
        code = torch.round(x * INT8_MAX / top).to(torch.int8)
    return code, scale.squeeze(-1)


def _pages(g, slots, case, spare):
    """A shuffled block table that holds `slots` slots a sequence, and the pool's size."""
    need = [-(-n // PAGE) for n in slots]
    pool = sum(-(-n // PAGE) for part in _spans(case) for n in part) + spare
    order = torch.randperm(pool, generator=g, device="cuda").to(torch.int32)
    width = max(max(need), 1)
    table = torch.full((len(slots), width), -1, dtype=torch.int32, device="cuda")
    counts = torch.tensor(need, device="cuda")
    take = torch.arange(width, device="cuda")[None] < counts[:, None]
    table[take] = order[: sum(need)]
    return table, counts.to(torch.int32), pool


def _pool(g, pool, case, kind):
    """A filled pool: keys carry a few strong channels, values do not."""
    x = _randn(g, pool, case["hkv"], PAGE, case["d"])
    if kind == "k":
        x *= 1 + 3 * (torch.rand(case["d"], generator=g, device="cuda") < 0.05)
    if case["held"] == "bf16":
        return x.to(torch.bfloat16), None
    return _quantise(x.to(torch.bfloat16).float(), case["held"])


def prepare(case, seed):
    g = _gen(seed)
    s = {"case": case}
    if case["op"] == "rope":
        rows, d, t = case["rows"], case["d"], HELD[case["type"]]
        nq, nk = case["hq"] * d, case["hkv"] * d
        if case["fused"]:                        # slices of one fused projection's output
            qkv = _randn(g, rows, nq + 2 * nk).to(t)
            q, k = qkv[:, :nq], qkv[:, nq:nq + nk]
        else:
            q, k = _randn(g, rows, nq).to(t), _randn(g, rows, nk).to(t)
        s["q"], s["k"] = q.unflatten(1, (case["hq"], d)), k.unflatten(1, (case["hkv"], d))
        s["q_out"] = torch.empty(rows, case["hq"], d, dtype=t, device="cuda")
        s["k_out"] = torch.empty(rows, case["hkv"], d, dtype=t, device="cuda")
        axes = [n for n in (case["s0"], case["s1"], case["s2"]) if n]
        # patches of one or more frames in reading order, from a base position on
        side = max(1, math.isqrt(min(rows, 1400)))
        base = int(torch.randint(0, case["far"] + 1, (1,), generator=g, device="cuda"))
        i = torch.arange(rows, device="cuda")
        grid = [base + i // (side * side), base + i // side % side, base + i % side]
        s["pos"] = torch.stack(grid[-len(axes):] if len(axes) < 3 else grid).to(torch.int32)
        pairs = sum(axes)
        s["inv_freq"] = (10000.0 ** (-torch.arange(pairs, device="cuda", dtype=torch.float64) /
                                     pairs)).float()
        s["axis"] = torch.tensor(_axis_of_pair(axes, case["order"]), device="cuda")
        if own:
            import speculative_decoding_tree_build_gb300 as tv
            s["geom"] = tv.rope_axes_geom(case["hq"], case["hkv"], d, axes, case["style"],
                                          case["order"])
        return s
    old, new = _spans(case)
    at = torch.randperm(case["batch"], generator=torch.Generator().manual_seed(int(seed))).tolist()
    old, new = [old[i] for i in at], [new[i] for i in at]
    ends = [a + b for a, b in zip(old, new)]
    s["table"], s["n_blocks"], pool = _pages(g, ends, case, 3)
    s["status"] = torch.zeros(case["batch"], dtype=torch.int32, device="cuda")
    s["old"] = torch.tensor(old, dtype=torch.int32, device="cuda")
    s["end"] = torch.tensor(ends, dtype=torch.int32, device="cuda")
    shape = (pool, case["hkv"], PAGE, case["d"])
    if case["op"] == "append":
        rows, n = sum(new), case["hkv"] * case["d"]
        cu = [0]
        for c in new:
            cu.append(cu[-1] + c)
        s["cu"] = torch.tensor(cu, dtype=torch.int32, device="cuda")
        if case["fused"]:
            kv = _randn(g, rows, 2 * n).to(torch.bfloat16)
            k, v = kv[:, :n], kv[:, n:]
        else:
            k, v = (_randn(g, rows, n).to(torch.bfloat16) for _ in range(2))
        s["k_new"], s["v_new"] = (x.unflatten(1, (case["hkv"], case["d"])) for x in (k, v))
        s["k"], s["v"] = (torch.zeros(shape, dtype=torch.int8, device="cuda").view(HELD[case["held"]])
                          for _ in range(2))
        s["ks"], s["vs"] = (torch.zeros(shape[:3], device="cuda") for _ in range(2))
    else:
        s["k"], s["ks"] = _pool(g, pool, case, "k")
        s["v"], s["vs"] = _pool(g, pool, case, "v")
    if case["op"] == "read":
        s["to_table"], s["to_n_blocks"], to_pool = _pages(g, ends, case, 5)
        s["k_out"], s["v_out"] = (torch.zeros(to_pool, *shape[1:], dtype=torch.bfloat16,
                                              device="cuda") for _ in range(2))
    if case["op"] == "decode":
        s["q"] = _randn(g, case["batch"], case["hq"], case["d"]).to(torch.bfloat16)
        s["out"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty(case["batch"], case["hq"], device="cuda")
    if own:
        import speculative_decoding_tree_build_gb300 as tv
        s["geom"] = tv.geom(case.get("hq", case["hkv"]), case["hkv"], case["d"])
        if case["op"] == "decode":
            s["work"] = torch.empty(tv.decode_workspace_bytes(s["geom"], case["batch"]),
                                    dtype=torch.uint8, device="cuda")
    return s


# ------------------------------------------------------------------- one pass


def run(s):
    return {"rope": _rope, "append": _append, "read": _read, "decode": _decode}[s["case"]["op"]](s)


def _axis_of_pair(sections, order):
    """Which axis each rotated pair takes its position from: one axis after
    the other, or the axes in turn while they have pairs left."""
    if order == 0:
        return [a for a, n in enumerate(sections) for _ in range(n)]
    turns = sorted((turn, a) for a, n in enumerate(sections) for turn in range(n))
    return [a for _, a in turns]


def _rope(s):
    if own:
        import speculative_decoding_tree_build_gb300 as tv
        tv.rope_axes(s["geom"], s["q"], s["k"], s["pos"], s["inv_freq"], s["q_out"], s["k_out"])
        return {"q": s["q_out"], "k": s["k_out"]}
    angle = s["pos"].double()[s["axis"]].t() * s["inv_freq"].double()      # [rows, pairs]
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
    pairs = cos.shape[-1]

    def turn(x):
        y = x.float().clone()
        a, b = ((y[..., :pairs], y[..., pairs:2 * pairs]) if s["case"]["style"] else
                (y[..., 0:2 * pairs:2], y[..., 1:2 * pairs:2]))
        ra, rb = a * cos - b * sin, b * cos + a * sin
        a.copy_(ra)
        b.copy_(rb)
        return y.to(x.dtype)

    return {"q": turn(s["q"]), "k": turn(s["k"])}


def _append(s):
    if own:
        import speculative_decoding_tree_build_gb300 as tv
        tv.kv_quant_append(s["geom"], s["k_new"], s["v_new"], s["cu"], s["old"], s["table"],
                           s["n_blocks"], s["k"], s["v"], s["ks"], s["vs"], s["status"])
    else:
        row = torch.arange(s["k_new"].shape[0], device="cuda")
        seq = torch.searchsorted(s["cu"].long(), row, right=True) - 1
        slot = s["old"].long()[seq] + row - s["cu"].long()[seq]
        page, at = s["table"].long()[seq, slot // PAGE], slot % PAGE
        kc, ks = _quantise(s["k_new"].float(), s["case"]["held"])
        vc, vs = _quantise(s["v_new"].float(), s["case"]["held"])
        s["k"].view(torch.int8)[page, :, at] = kc.view(torch.int8)
        s["v"].view(torch.int8)[page, :, at] = vc.view(torch.int8)
        s["ks"][page, :, at], s["vs"][page, :, at] = ks, vs
    # the codes are returned as the numbers they are, each row's unit beside them
    return {"k": s["k"], "v": s["v"], "ks": s["ks"], "vs": s["vs"], "status": s["status"]}


def _read(s):
    if own:
        import speculative_decoding_tree_build_gb300 as tv
        tv.kv_quant_read(s["geom"], s["old"], s["end"], s["table"], s["n_blocks"], s["k"], s["v"],
                         s["ks"], s["vs"], s["to_table"], s["to_n_blocks"], s["k_out"], s["v_out"],
                         s["status"])
    else:
        width = s["table"].shape[1] * PAGE
        slot = torch.arange(width, device="cuda")
        take = (slot >= s["old"][:, None]) & (slot < s["end"][:, None])
        seq, slot = take.nonzero(as_tuple=True)
        at = slot % PAGE
        page, to = s["table"].long()[seq, slot // PAGE], s["to_table"].long()[seq, slot // PAGE]
        k = s["k"].view(torch.int8)[page, :, at].view(s["k"].dtype).float() * s["ks"][page, :, at][..., None]
        v = s["v"].view(torch.int8)[page, :, at].view(s["v"].dtype).float() * s["vs"][page, :, at][..., None]
        s["k_out"][to, :, at] = k.to(torch.bfloat16)
        s["v_out"][to, :, at] = v.to(torch.bfloat16)
    return {"k": s["k_out"], "v": s["v_out"], "status": s["status"]}


def _decode(s):
    if own:
        import speculative_decoding_tree_build_gb300 as tv
        tv.decode_attention(s["geom"], s["q"], s["end"], s["table"], s["n_blocks"], s["k"], s["v"],
                            s["ks"], s["vs"], s["out"], s["lse"], s["work"], s["status"])
        return {"out": s["out"], "lse": s["lse"], "status": s["status"]}
    case = s["case"]
    page = s["table"].long().clamp(min=0)                    # pages not held are masked below

    def fetch(x, scale):
        y = x.view(torch.int16 if x.dtype == torch.bfloat16 else torch.int8)[page].view(x.dtype).float()
        if scale is not None:
            y *= scale[page][..., None]
        return y.transpose(1, 2).flatten(2, 3)               # [batch, hkv, slots, d]

    group = case["hq"] // case["hkv"]
    q = s["q"].float().unflatten(1, (case["hkv"], group))
    score = (q @ fetch(s["k"], s["ks"]).transpose(2, 3)) / math.sqrt(case["d"])
    seen = torch.arange(score.shape[-1], device="cuda") < s["end"][:, None, None, None]
    score = torch.where(seen, score, -math.inf)
    top = score.amax(-1, keepdim=True)
    base = torch.where(top > -math.inf, top, 0.0)
    p = torch.exp(score - base)
    total = p.sum(-1, keepdim=True)
    out = (p @ fetch(s["v"], s["vs"])) / torch.where(total > 0, total, 1.0)
    lse = (base + total.log()).flatten(1)
    return {"out": out.flatten(1, 2).to(torch.bfloat16), "lse": lse, "status": s["status"]}


# ------------------------------------------------------------------- what a pass needs


def work(case):
    d, hkv = case["d"], case["hkv"]
    if case["op"] == "rope":
        size = 2 if case["type"] == "bf16" else 4
        axes = sum(1 for n in (case["s0"], case["s1"], case["s2"]) if n)
        pairs = case["s0"] + case["s1"] + case["s2"]
        values = case["rows"] * (case["hq"] + hkv)
        return {"bytes": values * d * 2 * size + case["rows"] * axes * 4 + pairs * 4,
                "flops": values * pairs * 6}
    old, new = _spans(case)
    rows = sum(new)
    tables = case["batch"] * 12 + sum(-(-(a + b) // PAGE) - a // PAGE for a, b in zip(old, new)) * 4
    held = 2 * rows * hkv * ((d * 2) if case["held"] == "bf16" else d + 4)
    if case["op"] == "decode":
        ends = case["batch"] * case["hq"] * (2 * d * 2 + 4)
        return {"bytes": held + ends + tables, "flops": 4 * rows * case["hq"] * d}
    plain = 2 * rows * hkv * d * 2
    return {"bytes": held + plain + tables * (2 if case["op"] == "read" else 1),
            "flops": 2 * rows * hkv * d * 2}


# ------------------------------------------------------------------- in 64 bits


def exact(case, seed):
    with torch.no_grad():
        s = prepare(case, seed)
        return {"rope": _exact_rope, "append": _exact_append, "read": _exact_read,
                "decode": _exact_decode}[case["op"]](s, case)


def _exact_rope(s, case):
    axes = [n for n in (case["s0"], case["s1"], case["s2"]) if n]
    left, axis, a = list(axes), [], 0
    while sum(left):
        a %= len(axes)
        if left[a]:
            axis.append(a)
            left[a] -= 1
            a += case["order"]
        else:
            a += 1
    pairs = len(axis)
    angle = torch.stack([s["pos"][axis[i]].double() * s["inv_freq"][i].double()
                         for i in range(pairs)], 1)
    unit = torch.polar(torch.ones_like(angle), angle)[:, None]

    def turn(x):
        y = x.double().clone()
        if case["style"]:
            z = torch.complex(y[..., :pairs].contiguous(), y[..., pairs:2 * pairs].contiguous()) * unit
            y[..., :pairs], y[..., pairs:2 * pairs] = z.real, z.imag
        else:
            z = torch.view_as_complex(y[..., :2 * pairs].unflatten(-1, (pairs, 2)).contiguous()) * unit
            y[..., :2 * pairs] = torch.view_as_real(z).flatten(-2)
        return y

    return {"q": turn(s["q"]), "k": turn(s["k"])}


def _exact_append(s, case):
    def two_to(n):
        return ((n + 1023) << 52).view(torch.float64)

    def coded(x):
        y = x.double()
        top = y.abs().amax(-1)
        if case["held"] == "int8":
            scale = top.clamp(min=TINY) / 127
            return None, scale
        # the smallest power of two, from 2^-100 on, under which the row fits
        _, e = torch.frexp(top.clamp(min=TINY))
        power = (e.long() - 10).clamp(min=-100)
        for _ in range(3):
            power = torch.where(top > 448 * two_to(power), power + 1, power)
        y = y / two_to(power)[..., None]
        _, e = torch.frexp(y)                    # 4 bits of significand, down to 2^-9
        step = two_to(e.long().clamp(min=-5) - 4)
        return torch.round(y / step) * step, two_to(power)

    got = {"status": None}
    cu, old, table = s["cu"].tolist(), s["old"].tolist(), s["table"].tolist()
    page, at = [], []
    for b in range(case["batch"]):
        slots = range(old[b], old[b] + cu[b + 1] - cu[b])
        page += [table[b][i // PAGE] for i in slots]
        at += [i % PAGE for i in slots]
    page, at = torch.tensor(page, device="cuda"), torch.tensor(at, device="cuda")
    for name in ("k", "v"):
        code, scale = coded(s[name + "_new"])
        full = torch.zeros(s[name + "s"].shape, dtype=torch.float64, device="cuda")
        full[page, :, at] = scale
        got[name + "s"], got[name] = full, None
        if code is not None:
            full = torch.zeros(s[name].shape, dtype=torch.float64, device="cuda")
            full[page, :, at] = code
            got[name] = full
    return got


def _rows_of(s, b, first, last, name):
    """Sequence b's rows first..last-1 of the cache in 64 bits, [rows, hkv, d]."""
    slots = torch.arange(first, last, device="cuda")
    page, at = s["table"][b].long()[slots // PAGE], slots % PAGE
    x = s[name].view(torch.int8 if s[name + "s"] is not None else torch.int16)[page, :, at]
    x = x.view(s[name].dtype).double()
    return x if s[name + "s"] is None else x * s[name + "s"][page, :, at].double()[..., None]


def _exact_read(s, case):
    got = {"status": None}
    for name in ("k", "v"):
        full = torch.zeros(s[name + "_out"].shape, dtype=torch.float64, device="cuda")
        for b, (first, last) in enumerate(zip(s["old"].tolist(), s["end"].tolist())):
            slots = torch.arange(first, last, device="cuda")
            full[s["to_table"][b].long()[slots // PAGE], :, slots % PAGE] = _rows_of(s, b, first, last, name)
        got[name] = full
    return got


def _exact_decode(s, case):
    group, d = case["hq"] // case["hkv"], case["d"]
    outs, lses = [], []
    for b, n in enumerate(s["end"].tolist()):
        if n == 0:
            outs.append(torch.zeros(case["hq"], d, dtype=torch.float64, device="cuda"))
            lses.append(torch.full((case["hq"],), -math.inf, dtype=torch.float64, device="cuda"))
            continue
        k, v = (_rows_of(s, b, 0, n, name).permute(1, 0, 2) for name in ("k", "v"))
        q = s["q"][b].double().view(case["hkv"], group, d)
        score = torch.einsum("hgd,hnd->hgn", q, k) * d ** -0.5
        lse = torch.logsumexp(score, -1)
        outs.append(torch.einsum("hgn,hnd->hgd", torch.exp(score - lse[..., None]), v).flatten(0, 1))
        lses.append(lse.flatten())
    return {"out": torch.stack(outs), "lse": torch.stack(lses), "status": None}
