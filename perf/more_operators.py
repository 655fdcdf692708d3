"""Operators of an 8-bit paged KV cache, as they are called while a model serves: new K and V rows quantised as they are written, attention
of single tokens and of chunks of new tokens over the quantised blocks, the two in one call, and rows read back.

The cache holds each K and V row of a token and kv head as D codes in e4m3 and one scale byte s: value = code * 2^(s - 127). A row's
exponent is the least e >= -117 whose 448 * 2^e reaches the row's largest magnitude, so that dividing by the scale is exact.

A case's "batch" lists the step's requests as "[COUNTx]NEW@CACHED, ...", NEW and CACHED a number or a range "LO-HI": NEW tokens are
computed over CACHED tokens that the cache holds already. The lengths follow from the case; values and block numbers from the seed.
"""

import math
import random

import torch

own = False

DEVICE = "cuda"
LEAST = -117  # the smallest exponent of a scale: below it codes would leave bf16's normal numbers


# ------------------------------------------------------------------ cases
def listed():
    llama = {"hq": 32, "hkv": 8, "d": 128, "block": 16}
    none = {"softcap": 0.0, "mask": "none", "span": 0}
    return [
        # a decode step's new rows: latency is all there is
        {"name": "write-64", "op": "write", "rows": 64, "padding": 0, "hkv": 8, "d": 128, "block": 16},
        # the rows of a long prompt, some of them padding
        {"name": "write-16k", "op": "write", "rows": 16001, "padding": 383, "hkv": 8, "d": 128, "block": 16},
        # a conversation's rows read back, to be kept elsewhere
        {"name": "read-2k", "op": "read", "rows": 2047, "padding": 0, "hkv": 2, "d": 64, "block": 8},
        # the contexts of preempted requests read back
        {"name": "read-128k", "op": "read", "rows": 131072, "padding": 0, "hkv": 8, "d": 128, "block": 16},
        # a handful of short chats on a small model, one token each
        {"name": "decode-4", "op": "attention", "batch": "1@4, 1@15, 1@16, 1@39", "hq": 4, "hkv": 2, "d": 64, "block": 16, **none},
        # the steady state of a chat server
        {"name": "decode-64", "op": "attention", "batch": "64x1@511-4095", **llama, **none},
        # a few very long conversations
        {"name": "decode-long", "op": "attention", "batch": "8x1@32767-131071", **llama, **none},
        # a few guessed tokens of each request are checked at once
        {"name": "verify-64", "op": "attention", "batch": "64x5@511-4095", **llama, **none},
        # prompt processing at scale
        {"name": "chunks-2048", "op": "attention", "batch": "4x2048@6144", **llama, **none},
        # one chunk over a long context, and decodes on a layer that sees the last tokens only, all q heads on one kv head
        {"name": "window-odd", "op": "attention", "batch": "517@20001, 1001@0, 3@77, 40x1@63-30000", "hq": 8, "hkv": 1, "d": 64, "block": 32,
         "softcap": 30.0, "mask": "window", "span": 2000},
        # a continuous-batching step, written and attended in one call: a chunk of a long prompt, short prompts, decodes
        {"name": "step-mixed", "op": "step", "batch": "512@1536, 8x64@0, 320x1@127-2047", **llama, **none},
        # the same of a model with a kv head per q head
        {"name": "step-heads", "op": "step", "batch": "30x1@0-900, 133@250, 2@15", "hq": 12, "hkv": 12, "d": 64, "block": 16, **none},
    ]


def _logint(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["attention"] * 5 + ["step", "step", "write", "read"])
    d, block = rng.choice([64, 128]), rng.choice([8, 16, 16, 32])
    group = rng.choice([1, 2, 4, 8])
    hkv = rng.choice([1, 2, 3, 4, 8]) if group > 1 else rng.choice([2, 4, 8, 12, 16])
    if op in ("write", "read"):
        rows = _logint(rng, 1, 20000)
        return {"op": op, "rows": rows, "padding": rng.choice([0, _logint(rng, 1, rows)]), "hkv": hkv, "d": d, "block": block}
    kind = rng.choice(["decode", "chunks", "mixed", "guesses"])
    top = _logint(rng, 16, 65535 if op == "attention" else 8191)
    most = max(1, min(256, (1 << (19 if op == "attention" else 17)) // top))
    parts = []
    if kind in ("decode", "mixed"):
        parts.append("%dx1@%d-%d" % (_logint(rng, 1, most), rng.randint(0, top // 2), top))
    if kind == "guesses":
        parts.append("%dx%d-%d@%d-%d" % (_logint(rng, 1, most), rng.randint(1, 3), rng.randint(3, 8), rng.randint(0, top // 2), top))
    if kind in ("chunks", "mixed"):
        for _ in range(rng.randint(1, 3)):
            new = _logint(rng, 2, 2300)
            parts.insert(rng.randint(0, len(parts)), "%d@%d" % (new, rng.choice([0, _logint(rng, 1, 6000)])))
    mask = rng.choice(["none", "none", "none", "documents", "window"])
    return {"op": op, "batch": ", ".join(parts), "hq": hkv * group, "hkv": hkv, "d": d, "block": block,
            "softcap": rng.choice([0.0, 0.0, 0.0, 15.0, 50.0]), "mask": mask, "span": 0 if mask == "none" else _logint(rng, 3, 4096)}


def _rng_of(case):
    return random.Random(repr(sorted((k, v) for k, v in case.items() if k != "name")))


def _range(text, rng):
    lo, _, hi = text.partition("-")
    return rng.randint(int(lo), int(hi)) if hi else int(lo)


def _requests(case):
    """[(new, cached)] of the case's batch."""
    rng, out = _rng_of(case), []
    for part in case["batch"].split(","):
        count, times, rest = part.strip().partition("x")
        if not times:
            count, rest = "1", part.strip()
        new, _, cached = rest.partition("@")
        for _ in range(int(count)):
            out.append((_range(new, rng), _range(cached, rng)))
    return out


def _ranges(case, reqs):
    """Per request the keys that each new token sees: lists (begin, end), key j seen where begin <= j < end."""
    rng, out, mask, span = _rng_of(case), [], case["mask"], case["span"]
    for n, c in reqs:
        pos, last = range(c, c + n), c + n
        if mask == "window":
            out.append(([max(0, p - span + 1) for p in pos], [p + 1 for p in pos]))
        elif mask == "documents":  # packed into one sequence; one in eight is padding that sees nothing
            stops, at = [], 0
            while at < last:
                at += rng.randint(1, 2 * span)
                stops.append((min(at, last), rng.random() < 0.125 and at < last))
            begin, end, k = [], [], 0
            for p in pos:
                while stops[k][0] <= p:
                    k += 1
                begin.append(stops[k - 1][0] if k else 0)
                end.append(begin[-1] if stops[k][1] else p + 1)
            out.append((begin, end))
        else:
            out.append(([0] * n, [p + 1 for p in pos]))
    return out


def _i32(values):
    return torch.tensor(values, dtype=torch.int32, device=DEVICE)


# ------------------------------------------------------------------ the format
def _exponents(top):
    """The least e >= LEAST with top <= 448 * 2^e = 0.875 * 2^(9 + e), for fp32 magnitudes."""
    m, e = torch.frexp(top)
    return torch.where(top == 0, LEAST, e - 9 + (m > 0.875).int()).clamp(min=LEAST)


def _power(e):
    """2^e in fp32 for whole numbers -126 <= e <= 127, exactly."""
    return ((e.int() + 127) << 23).view(torch.float32)


def _quantise(x):
    """bf16 rows [..., d] -> (codes in e4m3 [..., d], scale bytes [...])."""
    x = x.float()
    e = _exponents(x.abs().amax(-1))
    return (x * _power(-e).unsqueeze(-1)).to(torch.float8_e4m3fn), (e + 127).to(torch.uint8)


def _values(codes, scales):
    """fp32 values of codes [..., d] under scale bytes [...]."""
    return codes.float() * _power(scales.int() - 127).unsqueeze(-1)


# ------------------------------------------------------------------ inputs
def _rows(shape, g, keys):
    """bf16 rows as projections give them: a few strong channels in K, tokens of unlike size in V."""
    x = torch.empty(shape, dtype=torch.bfloat16, device=DEVICE).normal_(generator=g)
    if keys:
        gain = torch.ones(shape[-1], dtype=torch.bfloat16, device=DEVICE)
        gain[torch.randperm(shape[-1], generator=g, device=DEVICE)[:3]] = 4.0
        return x.mul_(gain)
    size = torch.empty(shape[:-1], dtype=torch.float32, device=DEVICE).normal_(generator=g).mul_(0.5).exp_()
    return x.mul_(size.unsqueeze(-1).bfloat16())


def _pool(blocks, B, hkv, d, g):
    """A quantised pool that holds rows everywhere."""
    codes = torch.empty(blocks, 2, B, hkv, d, dtype=torch.float8_e4m3fn, device=DEVICE)
    scales = torch.empty(blocks, 2, B, hkv, dtype=torch.uint8, device=DEVICE)
    step = max(1, (1 << 26) // (B * hkv * d))
    for b in range(0, blocks, step):
        for i in (0, 1):
            c, s = _quantise(_rows((min(step, blocks - b), B, hkv, d), g, i == 0))
            codes[b:b + step, i], scales[b:b + step, i] = c, s
    return codes, scales


def prepare(case, seed):
    g = torch.Generator(device=DEVICE)
    g.manual_seed(int(seed))
    return (_prepare_rows if case["op"] in ("write", "read") else _prepare_attention)(case, g)


def _prepare_rows(case, g):
    B, hkv, d, T = case["block"], case["hkv"], case["d"], case["rows"]
    blocks = -(-T // B) + 7
    codes, scales = _pool(blocks, B, hkv, d, g)
    slots = torch.randperm(blocks * B, generator=g, device=DEVICE)[:T]
    slots[torch.randperm(T, generator=g, device=DEVICE)[:case["padding"]]] = -1
    s = {"case": case, "codes": codes, "scales": scales, "slots": slots}
    if case["op"] == "write":
        # the projection's rows hold k and v side by side
        kv = torch.cat([_rows((T, hkv, d), g, True).flatten(1), _rows((T, hkv, d), g, False).flatten(1)], 1)
        s["k"], s["v"] = kv[:, :hkv * d].view(T, hkv, d), kv[:, hkv * d:].view(T, hkv, d)
    else:  # rows of padding stay as they are
        s["k"] = torch.full((T, hkv, d), 7.0, dtype=torch.bfloat16, device=DEVICE)
        s["v"] = torch.full((T, hkv, d), -7.0, dtype=torch.bfloat16, device=DEVICE)
    return s


def _prepare_attention(case, g):
    reqs = _requests(case)
    B, hq, hkv, d = case["block"], case["hq"], case["hkv"], case["d"]
    qsl, T = [0], sum(n for n, _ in reqs)
    for n, _ in reqs:
        qsl.append(qsl[-1] + n)
    lens = [n + c for n, c in reqs]
    used = [-(-L // B) for L in lens]
    blocks = int(sum(used) * 1.05) + 1
    order = torch.randperm(blocks, generator=g, device=DEVICE).to(torch.int32)
    table = torch.full((len(reqs), max(used)), -1, dtype=torch.int32, device=DEVICE)
    at = 0
    for r, u in enumerate(used):
        table[r, :u] = order[at:at + u]
        at += u
    codes, scales = _pool(blocks, B, hkv, d, g)
    # the projection's rows hold q, k and v side by side. Trained q and k give scores of some size
    q = torch.empty(T, hq * d, dtype=torch.bfloat16, device=DEVICE).normal_(generator=g).mul_(3.0 if case["softcap"] else 1.5)
    qkv = torch.cat([q, _rows((T, hkv, d), g, True).flatten(1), _rows((T, hkv, d), g, False).flatten(1)], 1)
    s = {"case": case, "reqs": reqs, "codes": codes, "scales": scales, "table": table, "qsl_host": qsl, "scale": d ** -0.5,
         "q": qkv[:, :hq * d].view(T, hq, d), "k": qkv[:, hq * d:(hq + hkv) * d].view(T, hkv, d),
         "v": qkv[:, (hq + hkv) * d:].view(T, hkv, d), "begin": None, "end": None}
    if case["mask"] != "none":
        ranges = _ranges(case, reqs)
        s["begin"] = _i32([b for r in ranges for b in r[0]])
        if case["mask"] == "documents":
            s["end"] = _i32([e for r in ranges for e in r[1]])
    s["seq_lens"], s["qsl"], s["computed"] = _i32(lens), _i32(qsl), _i32([c for _, c in reqs])
    if own:
        from paged_kv_cache_hkv_gb300 import binding
        s["out"] = torch.zeros(T, hq, d, dtype=torch.bfloat16, device=DEVICE)
        s["slots"] = torch.empty(T, dtype=torch.int64, device=DEVICE)
        s["workspace"] = torch.empty(binding.pkv_quant_attention_workspace_size(
            len(reqs), hq, codes, max_blocks_per_req=max(used), chunk_keys=binding.quant_chunk_keys([n for n, _ in reqs], lens, hq // hkv, B)),
            dtype=torch.uint8, device=DEVICE)
        s["calls"] = binding.StepCalls(
            slot_mapping=s["slots"], block_table=table, query_start_loc=s["qsl"], num_computed_tokens=s["computed"], kv_cache=codes,
            kv_scales=scales, key=s["k"], value=s["v"], out=s["out"], q=s["q"], seq_lens=s["seq_lens"], max_query_len=max(n for n, _ in reqs),
            max_seq_len=max(lens), scale=s["scale"], workspace=s["workspace"], softcap=case["softcap"], key_begin=s["begin"],
            key_end=s["end"], write_in_attention=True)
    return s


# ------------------------------------------------------------------ the operators
def run(s):
    op = s["case"]["op"]
    if op == "write":
        if own:
            from paged_kv_cache_hkv_gb300 import binding
            binding.pkv_quant_kv_write(s["codes"], s["scales"], s["k"], s["v"], s["slots"])
        else:
            _write(s, s["slots"])
        return {"kv_cache": s["codes"], "kv_scales": s["scales"]}
    if op == "read":
        if own:
            from paged_kv_cache_hkv_gb300 import binding
            binding.pkv_quant_kv_read(s["k"], s["v"], s["codes"], s["scales"], s["slots"])
        else:
            _read(s)
        return {"key": s["k"], "value": s["v"]}
    if op == "step":
        if own:
            s["calls"].run()
            return {"out": s["out"], "slot_mapping": s["slots"], "kv_cache": s["codes"], "kv_scales": s["scales"]}
        slots = _slots(s)
        _write(s, slots)
        return {"out": _attention(s), "slot_mapping": slots, "kv_cache": s["codes"], "kv_scales": s["scales"]}
    if own:
        s["calls"].attend()
        return s["out"]
    return _attention(s)


def _write(s, slots):
    B, hkv, d = s["case"]["block"], s["case"]["hkv"], s["case"]["d"]
    at = slots[slots >= 0]
    for i, x in enumerate((s["k"], s["v"])):
        codes, scales = _quantise(x[slots >= 0])
        s["codes"].view(torch.uint8)[at // B, i, at % B] = codes.view(torch.uint8)
        s["scales"][at // B, i, at % B] = scales


def _read(s):
    B = s["case"]["block"]
    rows = s["slots"] >= 0
    at = s["slots"].clamp(min=0)
    for i, x in enumerate((s["k"], s["v"])):
        codes = s["codes"].view(torch.uint8)[at // B, i, at % B].view(torch.float8_e4m3fn)
        x.copy_(torch.where(rows.view(-1, 1, 1), _values(codes, s["scales"][at // B, i, at % B]).bfloat16(), x))


def _slots(s):
    B, T = s["case"]["block"], s["q"].shape[0]
    t = torch.arange(T, device=s["q"].device)
    r = torch.searchsorted(s["qsl"][1:].long(), t, right=True)
    pos = s["computed"][r].long() + t - s["qsl"][r]
    return s["table"][r, pos // B].long() * B + pos % B


def _weights(scores, s, key, begin, end):
    """Scores [..., rows, keys] over keys numbered key -> softmax numerators and their sums; a row that sees nothing has sum 0."""
    cap = s["case"]["softcap"]
    if cap:
        scores = torch.tanh(scores / cap) * cap
    scores = torch.where((key >= begin) & (key < end), scores, -math.inf)
    top = scores.amax(-1, keepdim=True)
    e = torch.exp(scores - torch.where(top == -math.inf, 0.0, top))
    return e, e.sum(-1, keepdim=True)


def _blocks(s, ids):
    """fp32 values of the blocks ids [...]: [..., 2, B, hkv, d]."""
    return _values(s["codes"].view(torch.uint8)[ids].view(torch.float8_e4m3fn), s["scales"][ids])


def _attention(s):
    case, reqs, qsl = s["case"], s["reqs"], s["qsl_host"]
    B, hq, hkv, d = case["block"], case["hq"], case["hkv"], case["d"]
    group = hq // hkv
    q, table = s["q"], s["table"]
    out = torch.zeros(q.shape[0], hq, d, dtype=torch.bfloat16, device=q.device)
    # requests of one to eight new tokens in batches of like length and as many rows, padded to the longest of each
    few = sorted((r for r, (n, _) in enumerate(reqs) if n <= 8), key=lambda r: (reqs[r][0], reqs[r][1]))
    while few:
        n, longest = reqs[few[-1]][0], sum(reqs[few[-1]])
        take = max(1, min(len(few), (1 << 20) // longest))
        while reqs[few[-take]][0] != n:
            take -= 1
        batch, few = few[-take:], few[:-take]
        ids = torch.tensor(batch, device=q.device)
        rows = torch.tensor([qsl[r] for r in batch], device=q.device).view(-1, 1) + torch.arange(n, device=q.device)
        last = s["seq_lens"][ids].long().view(-1, 1)
        end = last - n + 1 + torch.arange(n, device=q.device)
        begin = torch.zeros_like(end) if s["begin"] is None else s["begin"][rows].long()
        if s["end"] is not None:
            end = torch.minimum(last, s["end"][rows].long())
        used = -(-longest // B)
        first = 0
        if case["mask"] == "window" and take == 1:  # blocks before every row's window are left alone
            first = max(0, reqs[batch[0]][1] + 1 - case["span"]) // B
        blocks = _blocks(s, table[ids, first:used].clamp(min=0).long())  # [reqs, blocks, 2, B, hkv, d]
        k = blocks[:, :, 0].flatten(1, 2).permute(0, 2, 3, 1)  # [reqs, hkv, d, keys]
        v = blocks[:, :, 1].flatten(1, 2).permute(0, 2, 1, 3)  # [reqs, hkv, keys, d]
        key = torch.arange(first * B, used * B, device=q.device)
        x = q[rows].float().view(-1, n, hkv, group, d).permute(0, 2, 3, 1, 4).flatten(2, 3)  # [reqs, hkv, group * n, d]
        scores = (x @ k * s["scale"]).unflatten(2, (group, n))
        e, total = _weights(scores, s, key, begin.view(-1, 1, 1, n, 1), end.view(-1, 1, 1, n, 1))
        o = (e.flatten(2, 3) @ v).unflatten(2, (group, n)) / torch.where(total == 0, 1.0, total)
        out[rows] = o.permute(0, 3, 1, 2, 4).reshape(-1, n, hq, d).to(torch.bfloat16)
        del blocks, k, v, scores, e
    for r, (n, c) in enumerate(reqs):
        if n <= 8:
            continue
        L, t0 = n + c, qsl[r]
        blocks = _blocks(s, table[r, :-(-L // B)].long())
        k = blocks[:, 0].flatten(0, 1)[:L].permute(1, 2, 0)  # [hkv, d, keys]
        v = blocks[:, 1].flatten(0, 1)[:L].permute(1, 0, 2)  # [hkv, keys, d]
        key = torch.arange(L, device=q.device)
        for i0 in range(0, n, 2048):
            i1 = min(n, i0 + 2048)
            pos = torch.arange(c + i0, c + i1, device=q.device).view(-1, 1)
            begin = torch.zeros_like(pos) if s["begin"] is None else s["begin"][t0 + i0:t0 + i1].long().view(-1, 1)
            end = pos + 1 if s["end"] is None else s["end"][t0 + i0:t0 + i1].long().clamp(max=L).view(-1, 1)
            rows = q[t0 + i0:t0 + i1].float().view(-1, hkv, group, d).permute(1, 2, 0, 3)  # [hkv, group, rows, d]
            scores = rows.flatten(1, 2) @ k * s["scale"]
            e, total = _weights(scores.view(hkv, group, i1 - i0, L), s, key, begin, end)
            o = (e.view(hkv, -1, L) @ v).view(hkv, group, i1 - i0, d) / torch.where(total == 0, 1.0, total)
            out[t0 + i0:t0 + i1] = o.permute(2, 0, 1, 3).reshape(-1, hq, d).to(torch.bfloat16)
    return out


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    hkv, d = case["hkv"], case["d"]
    wide, narrow = 4 * hkv * d, 2 * hkv * (d + 1)  # bytes of a token's K and V rows in bf16 and in the cache
    if case["op"] in ("write", "read"):
        return {"bytes": (case["rows"] - case["padding"]) * (wide + narrow) + 8 * case["rows"], "flops": 0}
    reqs, hq = _requests(case), case["hq"]
    rows, keys, pairs, entries = 0, 0, 0, 0
    for (n, c), (begin, end) in zip(reqs, _ranges(case, reqs)):
        rows += n
        pairs += sum(max(0, e - b) for b, e in zip(begin, end))
        at = 0  # keys that some row sees
        for b, e in sorted((b, e) for b, e in zip(begin, end) if e > b):
            keys += max(0, e - max(b, at))
            entries += max(0, -(-e // case["block"]) - max(b, at) // case["block"])
            at = max(at, e)
    masks = {"none": 0, "window": 1, "documents": 2}[case["mask"]]
    total = 4 * rows * hq * d + keys * narrow + 4 * entries + 12 * len(reqs) + 4 * masks * rows
    if case["op"] == "step":  # the new rows in and their slots out; their codes and scales are among the keys
        total += rows * (wide + 8)
    return {"bytes": total, "flops": 4 * d * hq * pairs}


# ------------------------------------------------------------------ the same from the definitions, in 64 bits
def _power64(e):
    return ((e.long() + 1023) << 52).view(torch.float64)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "write":
        _exact_write(s, s["slots"].tolist())
        return {"kv_cache": s["codes"], "kv_scales": s["scales"]}
    if case["op"] == "read":
        out = {"key": s["k"].double(), "value": s["v"].double()}
        B = case["block"]
        rows = torch.nonzero(s["slots"] != -1).flatten()
        block, off = torch.div(s["slots"][rows], B, rounding_mode="floor"), s["slots"][rows] % B
        for i, x in enumerate(out.values()):
            power = _power64(s["scales"][block, i, off].long() - 127)
            x[rows] = s["codes"].view(torch.uint8)[block, i, off].view(torch.float8_e4m3fn).double() * power[:, :, None]
        return out
    if case["op"] == "step":
        slots, table = [], s["table"].tolist()
        for r, (n, c) in enumerate(s["reqs"]):
            slots += [table[r][p // case["block"]] * case["block"] + p % case["block"] for p in range(c, c + n)]
        _exact_write(s, slots)
        return {"out": _exact_attention(s), "slot_mapping": torch.tensor(slots), "kv_cache": s["codes"], "kv_scales": s["scales"]}
    return _exact_attention(s)


def _exact_write(s, slots):
    """Every value to the nearest of the codes, ties to the even one: the codes of one binade are 2^(b - 3) apart, those below 2^-6 2^-9."""
    B = s["case"]["block"]
    rows = torch.tensor([t for t, x in enumerate(slots) if x >= 0], dtype=torch.int64, device=s["codes"].device)
    block = torch.tensor([x // B for x in slots if x >= 0], dtype=torch.int64, device=rows.device)
    off = torch.tensor([x % B for x in slots if x >= 0], dtype=torch.int64, device=rows.device)
    if not rows.numel():
        return
    for i, x in enumerate((s["k"], s["v"])):
        x = x[rows].double()
        top = x.abs().max(-1).values
        e = torch.full_like(top, LEAST, dtype=torch.int64)
        for _ in range(260):  # up until 448 * 2^e reaches the row's largest
            short = 448.0 * _power64(e) < top
            if not bool(short.any()):
                break
            e = e + short.long()
        y = x / _power64(e)[..., None]
        binade = torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))).long().clamp(-6, 8)
        binade = torch.where(_power64(binade) > y.abs().clamp(min=2.0 ** -6), binade - 1, binade)
        binade = torch.where(_power64(binade + 1) <= y.abs(), binade + 1, binade)
        apart = _power64(binade - 3)
        s["codes"].view(torch.uint8)[block, i, off] = (torch.round(y / apart) * apart).to(torch.float8_e4m3fn).view(torch.uint8)
        s["scales"][block, i, off] = (e + 127).to(torch.uint8)


def _exact_attention(s):
    case = s["case"]
    B, hq, hkv, cap = case["block"], case["hq"], case["hkv"], case["softcap"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=s["q"].device)
    codes = s["codes"].view(torch.uint8)
    t0 = 0
    for r, ((n, c), (begin, end)) in enumerate(zip(s["reqs"], _ranges(case, s["reqs"]))):
        lo = torch.tensor(begin, device=out.device)
        hi = torch.tensor(end, device=out.device)
        for g in range(hkv):
            for i0 in range(0, n, 512):
                i1 = min(n, i0 + 512)
                first, past = min(begin[i0:i1]), max(max(end[i0:i1]), min(begin[i0:i1]) + 1)
                j = torch.arange(first, past, device=out.device)
                block, off = s["table"][r, j // B].long(), j % B
                keys, vals = (codes[block, i, off, g].view(torch.float8_e4m3fn).double()
                              * _power64(s["scales"][block, i, off, g].long() - 127)[:, None] for i in (0, 1))
                hidden = (j[None, :] < lo[i0:i1, None]) | (j[None, :] >= hi[i0:i1, None])
                for h in range(g * hq // hkv, (g + 1) * hq // hkv):
                    x = torch.einsum("id,jd->ij", s["q"][t0 + i0:t0 + i1, h].double(), keys).mul_(s["scale"])
                    if cap:
                        x = x.div_(cap).tanh_().mul_(cap)
                    x.masked_fill_(hidden, -math.inf)
                    x = x.sub_(torch.logsumexp(x, 1, keepdim=True)).exp_()
                    out[t0 + i0:t0 + i1, h] = torch.einsum("ij,jd->id", torch.nan_to_num_(x, nan=0.0), vals)
        t0 += n
    return out
