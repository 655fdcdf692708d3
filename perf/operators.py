"""Operators around the paged KV cache, as they are called while a model serves: attention whose scores are capped or biased by
distance, attention under masks that leave each row a range of keys, and the block tables, slot maps and free blocks of a step.

A case's "batch" lists the step's requests as "[COUNTx]NEW@CACHED, ...", NEW and CACHED a number or a range "LO-HI": NEW tokens are
computed over CACHED tokens that the cache holds already. The lengths follow from the case; values and block numbers from the seed.
"""

import math
import random
from collections import deque

import torch

own = False

DEVICE = "cuda"


# ------------------------------------------------------------------ cases
def listed():
    llama = {"hq": 32, "hkv": 8, "d": 128, "block": 16}
    return [
        # a handful of short chats on a small model, one token each: latency is all there is
        {"name": "cap-decode-4", "op": "attention", "batch": "1@4, 1@15, 1@16, 1@39", "hq": 4, "hkv": 2, "d": 64, "block": 16,
         "softcap": 30.0, "alibi": False, "mask": "none", "span": 0},
        # the steady state of a chat server with capped scores
        {"name": "cap-decode-64", "op": "attention", "batch": "64x1@511-4095", **llama,
         "softcap": 50.0, "alibi": False, "mask": "none", "span": 0},
        # a step of a model with distance biases and a kv head per q head: one chunk of a long prompt, short prompts, decodes
        {"name": "alibi-mixed", "op": "attention", "batch": "512@1536, 7x64@0, 61@3, 193x1@127-2047", "hq": 16, "hkv": 16, "d": 64, "block": 16,
         "softcap": 0.0, "alibi": True, "mask": "none", "span": 0},
        # a few very long conversations, capped and biased
        {"name": "cap-alibi-long", "op": "attention", "batch": "8x1@32767-131071", **llama,
         "softcap": 30.0, "alibi": True, "mask": "none", "span": 0},
        # prompt processing at scale with capped scores
        {"name": "cap-prefill", "op": "attention", "batch": "4x2048@6144", **llama,
         "softcap": 50.0, "alibi": False, "mask": "none", "span": 0},
        # short documents packed into one prompt, some of them padding that sees nothing
        {"name": "documents-8k", "op": "attention", "batch": "8191@0", **llama,
         "softcap": 0.0, "alibi": False, "mask": "documents", "span": 400},
        # prompts whose head (an image, an instruction) is seen in both directions, all q heads on one kv head
        {"name": "prefix-odd", "op": "attention", "batch": "3x1001-1499@0, 517@301, 40x1@63-2047", "hq": 8, "hkv": 1, "d": 64, "block": 32,
         "softcap": 0.0, "alibi": False, "mask": "prefix", "span": 700},
        # long conversations on a layer that sees the last tokens only
        {"name": "window-long", "op": "attention", "batch": "16x1@32767-131071", **llama,
         "softcap": 0.0, "alibi": False, "mask": "window", "span": 4096},
        # the tables of a decode step
        {"name": "tables-64", "op": "tables", "batch": "64x1@511-4095", "block": 16, "short": False},
        # a large step: thousands of decodes, chunks and new prompts, more than the pool has blocks for
        {"name": "tables-4096", "op": "tables", "batch": "32x2048@0-6144, 64x1-1023@0, 4000x1@127-4095", "block": 16, "short": True},
        # a few requests end, two of them with a prompt in common
        {"name": "release-8", "op": "release", "batch": "64x1@511-4095", "rows": 8, "prefix": 256, "block": 16},
        # a large batch is preempted: every request of a prefix-sharing group and many others
        {"name": "release-1024", "op": "release", "batch": "4096x1@1039-4095", "rows": 1024, "prefix": 1024, "block": 16},
    ]


def _logint(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["attention"] * 6 + ["tables", "tables", "release"])
    block = rng.choice([8, 16, 16, 32])
    if op == "tables":
        n = _logint(rng, 1, 4096)
        parts = ["%dx1@%d-%d" % (n, rng.randint(0, 500), rng.randint(500, 4095))]
        if rng.random() < 0.7:
            parts.insert(rng.randint(0, 1), "%dx%d-%d@0-%d" % (_logint(rng, 1, 32), rng.randint(1, 64), rng.randint(64, 2047), rng.randint(1, 4000)))
        return {"op": op, "batch": ", ".join(parts), "block": block, "short": rng.random() < 0.4}
    if op == "release":
        n = _logint(rng, 1, 4096)
        prefix = block * rng.choice([0, 0, rng.randint(1, 64)])
        return {"op": op, "batch": "%dx1@%d-%d" % (n, prefix + rng.randint(0, 300), prefix + rng.randint(300, 3000)),
                "rows": _logint(rng, 1, min(n, 1024)), "prefix": prefix, "block": block}
    d = rng.choice([64, 128])
    group = rng.choice([1, 2, 4, 8])
    hkv = rng.choice([1, 2, 3, 4, 8]) if group > 1 else rng.choice([2, 4, 8, 12, 16])
    kind = rng.choice(["decode", "prefill", "mixed"])
    parts = []
    if kind != "prefill":
        top = _logint(rng, 16, 65535)
        parts.append("%dx1@%d-%d" % (_logint(rng, 1, max(1, min(256, (1 << 19) // top))), rng.randint(0, top // 2), top))
    if kind != "decode":
        for _ in range(rng.randint(1, 3)):
            new = _logint(rng, 2, 2300)
            parts.insert(rng.randint(0, len(parts)), "%d@%d" % (new, rng.choice([0, _logint(rng, 1, 6000)])))
    mask = rng.choice(["none", "none", "documents", "prefix", "window"])
    mods = rng.choice([(1, 0), (0, 1), (1, 1)]) if mask == "none" else rng.choice([(0, 0), (0, 0), (1, 0), (0, 1)])
    return {"op": op, "batch": ", ".join(parts), "hq": hkv * group, "hkv": hkv, "d": d, "block": block,
            "softcap": rng.choice([15.0, 30.0, 50.0]) if mods[0] else 0.0, "alibi": bool(mods[1]), "mask": mask,
            "span": 0 if mask == "none" else _logint(rng, 3, 4096)}


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
        elif mask == "documents":
            begin, end, start, blank, stop = [], [], 0, False, 0
            stops, at = [], 0
            while at < last:  # the documents of the whole sequence; one in eight is padding, and the last is none
                at += rng.randint(1, 2 * span)
                stops.append((min(at, last), rng.random() < 0.125 and at < last))
            k = 0
            for p in pos:
                while stops[k][0] <= p:
                    k += 1
                start = stops[k - 1][0] if k else 0
                stop, blank = stops[k]
                begin.append(start)
                end.append(start if blank else p + 1)
            out.append((begin, end))
        elif mask == "prefix":
            head = min(last, rng.randint(span // 2, span + span // 2))
            out.append(([0] * n, [max(p + 1, head) for p in pos]))
        else:
            out.append(([0] * n, [p + 1 for p in pos]))
    return out


def _i32(values):
    return torch.tensor(values, dtype=torch.int32, device=DEVICE)


def _starts(reqs):
    qsl = [0]
    for n, _ in reqs:
        qsl.append(qsl[-1] + n)
    return qsl


# ------------------------------------------------------------------ inputs
def prepare(case, seed):
    g = torch.Generator(device=DEVICE)
    g.manual_seed(int(seed))
    return {"attention": _prepare_attention, "tables": _prepare_tables, "release": _prepare_release}[case["op"]](case, g)


def _prepare_attention(case, g):
    reqs = _requests(case)
    B, hq, hkv, d = case["block"], case["hq"], case["hkv"], case["d"]
    qsl, T = _starts(reqs), sum(n for n, _ in reqs)
    lens = [n + c for n, c in reqs]
    used = [-(-L // B) for L in lens]
    width = max(used)
    blocks = int(sum(used) * 1.1) + 1
    order = torch.randperm(blocks, generator=g, device=DEVICE).to(torch.int32)
    table = torch.full((len(reqs), width), -1, dtype=torch.int32, device=DEVICE)
    at = 0
    for r, u in enumerate(used):
        table[r, :u] = order[at:at + u]
        at += u
    kv = torch.empty(blocks, 2, B, hkv, d, dtype=torch.bfloat16, device=DEVICE)
    kv.normal_(generator=g)
    # the projection's rows hold q, k and v side by side: q is a strided view. Trained q and k give scores of some size
    qkv = torch.empty(T, (hq + 2 * hkv) * d, dtype=torch.bfloat16, device=DEVICE)
    qkv.normal_(generator=g).mul_(3.0 if case["softcap"] else 1.5)
    q = qkv[:, :hq * d].view(T, hq, d)
    s = {"case": case, "reqs": reqs, "q": q, "kv": kv, "table": table, "qsl_host": qsl, "scale": d ** -0.5,
         "slopes": None, "begin": None, "end": None}
    if case["alibi"]:
        s["slopes"] = torch.tensor([2.0 ** (-8.0 * (h + 1) / hq) for h in range(hq)], dtype=torch.float32, device=DEVICE)
    if case["mask"] != "none":
        ranges = _ranges(case, reqs)
        if case["mask"] != "prefix":
            s["begin"] = _i32([b for r in ranges for b in r[0]])
        if case["mask"] != "window":
            s["end"] = _i32([e for r in ranges for e in r[1]])
    s["seq_lens"], s["qsl"], s["computed"] = _i32(lens), _i32(qsl), _i32([c for _, c in reqs])
    if own:
        from paged_kv_cache_hkv_gb300 import binding
        s["out"] = torch.zeros(T, hq, d, dtype=torch.bfloat16, device=DEVICE)
        s["slots"] = torch.empty(T, dtype=torch.int64, device=DEVICE)
        s["workspace"] = torch.empty(max(256, binding.pkv_attention_workspace_size(len(reqs), hq, kv)), dtype=torch.uint8, device=DEVICE)
        k = qkv[:, hq * d:(hq + hkv) * d].view(T, hkv, d)
        v = qkv[:, (hq + hkv) * d:].view(T, hkv, d)
        s["calls"] = binding.StepCalls(
            slot_mapping=s["slots"], block_table=table, query_start_loc=s["qsl"], num_computed_tokens=s["computed"], kv_cache=kv, key=k, value=v,
            out=s["out"], q=q, seq_lens=s["seq_lens"], max_query_len=max(n for n, _ in reqs), max_seq_len=max(lens), scale=s["scale"],
            workspace=s["workspace"], softcap=case["softcap"], alibi_slopes=s["slopes"], key_begin=s["begin"], key_end=s["end"])
    return s


def _pool_tables(case, reqs, g, extra):
    """A pool's tables before the step: blocks of the cached tokens handed out in a seeded order, the others in the free queue (a ring)."""
    B = case["block"]
    prefix = case.get("prefix", 0) // B
    have = [-(-c // B) for _, c in reqs]
    total = [-(-(n + c) // B) for n, c in reqs]
    blocks = sum(total) + prefix + extra
    order = torch.randperm(blocks, generator=g, device=DEVICE).to(torch.int32).cpu()
    table = torch.full((len(reqs), max(total) + 1), -1, dtype=torch.int32)
    ref = torch.zeros(blocks, dtype=torch.int32)
    at = prefix
    shared = order[:prefix]
    for r, u in enumerate(have):
        if prefix and r % 4 != 3:
            table[r, :prefix] = shared
            ref[shared.long()] += 1
            first = prefix
        else:
            first = 0
        table[r, first:u] = order[at:at + u - first]
        ref[order[at:at + u - first].long()] = 1
        at += u - first
    free = order[at:]
    if prefix and int(ref[shared.long()].max()) == 0:  # nobody shares it
        free = torch.cat([shared, free])
    queue = torch.roll(torch.cat([free, order[:blocks - len(free)]]), 17)  # the ring starts in the middle
    return table.to(DEVICE), ref.to(DEVICE), queue.to(DEVICE), 17 % blocks, len(free)


def _prepare_tables(case, g):
    reqs = _requests(case)
    B, R, T = case["block"], len(reqs), sum(n for n, _ in reqs)
    table, ref, queue, head, count = _pool_tables(case, reqs, g, 100)
    need = sum(-(-(n + c) // B) - -(-c // B) for n, c in reqs)
    if case["short"]:
        count = min(count, need * 3 // 4)
    s = {"case": case, "T": T, "table": table, "ref": ref, "queue": queue, "state": _i32([head, count]),
         "computed": _i32([c for _, c in reqs]), "new": _i32([n for n, _ in reqs]), "reqs": reqs}
    if own:
        from paged_kv_cache_hkv_gb300 import binding
        s["qsl"], s["lens"] = _i32([0] * (R + 1)), _i32([0] * R)
        s["slots"] = torch.empty(T, dtype=torch.int64, device=DEVICE)
        s["state_out"] = torch.zeros_like(s["state"])
        s["calls"] = binding.TableCalls(
            block_table=table, query_start_loc=s["qsl"], seq_lens=s["lens"], slot_mapping=s["slots"], num_computed_tokens=s["computed"],
            query_lens=s["new"], free_queue=queue, free_state=s["state"], free_state_out=s["state_out"], ref_cnt=ref, block_size=B)
    return s


def _prepare_release(case, g):
    reqs = _requests(case)
    held = [n + c for n, c in reqs]
    table, ref, queue, head, count = _pool_tables(case, [(0, h) for h in held], g, 10)
    rows = torch.randperm(len(reqs), generator=g, device=DEVICE)[:case["rows"]].to(torch.int32)
    s = {"case": case, "table": table, "ref0": ref, "queue": queue, "state": _i32([head, count]), "held": _i32(held), "rows": rows}
    if own:
        from paged_kv_cache_hkv_gb300 import binding
        s["ref"], s["state_out"] = ref.clone(), torch.zeros_like(s["state"])
        s["calls"] = binding.TableCalls(block_table=table, free_queue=queue, free_state=s["state"], free_state_out=s["state_out"], ref_cnt=s["ref"],
                                        block_size=case["block"], release_rows=rows, release_tokens=s["held"])
    return s


# ------------------------------------------------------------------ the operators
def run(s):
    op = s["case"]["op"]
    if own:
        if op == "attention":
            s["calls"].attend()
            return s["out"]
        if op == "tables":
            s["calls"].build()
            return {"block_table": s["table"], "query_start_loc": s["qsl"], "seq_lens": s["lens"], "slot_mapping": s["slots"],
                    "free_state": s["state_out"], "ref_cnt": s["ref"]}
        s["ref"].copy_(s["ref0"])  # a release counts down in place: each pass starts from the same counts
        s["calls"].release()
        return {"free_queue": s["queue"], "free_state": s["state_out"], "ref_cnt": s["ref"]}
    return {"attention": _attention, "tables": _tables, "release": _release}[op](s)


def _weights(scores, s, pos, key, begin, end):
    """Scores [..., rows, keys] of rows at positions pos over keys numbered key -> softmax numerators and their sums; a row that sees nothing has sum 0."""
    cap, slopes = s["case"]["softcap"], s["slopes"]
    if cap:
        scores = torch.tanh(scores / cap) * cap
    if slopes is not None:
        # distances to the nearest key that the row sees: a constant per row leaves the softmax, and keeps far rows exact
        near = torch.minimum(torch.maximum(pos, begin), end - 1)
        scores = scores - slopes.view(s["case"]["hkv"], -1, 1, 1) * (near - key).abs().float()
    seen = (key >= begin) & (key < end)
    scores = torch.where(seen, scores, -math.inf)
    top = scores.amax(-1, keepdim=True)
    e = torch.exp(scores - torch.where(top == -math.inf, 0.0, top))
    return e, e.sum(-1, keepdim=True)


def _attention(s):
    case, reqs, qsl = s["case"], s["reqs"], s["qsl_host"]
    B, hq, hkv, d = case["block"], case["hq"], case["hkv"], case["d"]
    group = hq // hkv
    q, kv, table = s["q"], s["kv"], s["table"]
    T = q.shape[0]
    out = torch.zeros(T, hq, d, dtype=torch.bfloat16, device=q.device)
    single = [r for r, (n, _) in enumerate(reqs) if n == 1]
    # the decodes in batches of like length, padded to the longest of each
    single.sort(key=lambda r: reqs[r][1])
    while single:
        longest = reqs[single[-1]][1] + 1
        take = max(1, min(len(single), (1 << 20) // longest))
        batch, single = single[-take:], single[:-take]
        rows = torch.tensor([qsl[r] for r in batch], device=q.device)
        ids = torch.tensor(batch, device=q.device)
        end = s["seq_lens"][ids].long()
        pos = end - 1
        begin = torch.zeros_like(end) if s["begin"] is None else s["begin"][rows].long()
        if s["end"] is not None:
            end = torch.minimum(end, s["end"][rows].long())
        used = -(-longest // B)
        first = 0
        if case["mask"] == "window":  # blocks before every row's window are left alone
            first = max(0, reqs[batch[0]][1] + 1 - case["span"]) // B if take == 1 else 0
        blocks = kv[table[ids, first:used].clamp(min=0).long()]  # [rows, blocks, 2, B, hkv, d]
        k = blocks[:, :, 0].flatten(1, 2).permute(0, 2, 3, 1).float()  # [rows, hkv, d, keys]
        v = blocks[:, :, 1].flatten(1, 2).permute(0, 2, 1, 3).float()  # [rows, hkv, keys, d]
        del blocks
        key = torch.arange(first * B, used * B, device=q.device)
        scores = (q[rows].float().view(-1, hkv, group, d) @ k * s["scale"]).unsqueeze(3)  # [rows, hkv, group, 1, keys]
        at = [x.view(-1, 1, 1, 1, 1) for x in (pos, begin, end)]
        e, total = _weights(scores, s, at[0], key, at[1], at[2])
        o = e.squeeze(3) @ v / torch.where(total == 0, 1.0, total).squeeze(3)
        out[rows] = o.reshape(-1, hq, d).to(torch.bfloat16)
        del k, v, scores, e
    for r, (n, c) in enumerate(reqs):
        if n < 2:
            continue
        L, t0 = n + c, qsl[r]
        blocks = kv[table[r, :-(-L // B)].long()]
        k = blocks[:, 0].flatten(0, 1)[:L].permute(1, 2, 0).float()  # [hkv, d, keys]
        v = blocks[:, 1].flatten(0, 1)[:L].permute(1, 0, 2).float()  # [hkv, keys, d]
        key = torch.arange(L, device=q.device)
        for i0 in range(0, n, 2048):
            i1 = min(n, i0 + 2048)
            pos = torch.arange(c + i0, c + i1, device=q.device).view(-1, 1)
            begin = torch.zeros_like(pos) if s["begin"] is None else s["begin"][t0 + i0:t0 + i1].long().view(-1, 1)
            end = pos + 1 if s["end"] is None else s["end"][t0 + i0:t0 + i1].long().clamp(max=L).view(-1, 1)
            rows = q[t0 + i0:t0 + i1].float().view(-1, hkv, group, d).permute(1, 2, 0, 3)  # [hkv, group, rows, d]
            scores = rows.flatten(1, 2) @ k * s["scale"]
            e, total = _weights(scores.view(hkv, group, i1 - i0, L), s, pos, key, begin, end)
            o = (e.view(hkv, -1, L) @ v).view(hkv, group, i1 - i0, d) / torch.where(total == 0, 1.0, total)
            out[t0 + i0:t0 + i1] = o.permute(2, 0, 1, 3).reshape(-1, hq, d).to(torch.bfloat16)
    return out


def _tables(s):
    B, T, queue, table = s["case"]["block"], s["T"], s["queue"], s["table"]
    c, n = s["computed"].long(), s["new"].long()
    R, blocks = c.numel(), queue.numel()
    head, count = s["state"][0].long(), s["state"][1].long()
    have, total = (c + B - 1) // B, (c + n + B - 1) // B
    need = total - have
    through = torch.cumsum(need, 0)
    granted = (need == 0) | (through <= count)
    taken = torch.where(through <= count, through, 0).amax()
    col = torch.arange(table.shape[1], device=table.device)
    fresh = queue[(head + (through - need).view(-1, 1) + col - have.view(-1, 1)) % blocks]
    fresh = torch.where(granted.view(-1, 1), fresh, -1)
    new_table = torch.where((col >= have.view(-1, 1)) & (col < total.view(-1, 1)), fresh, table)
    qsl = torch.zeros(R + 1, dtype=torch.int64, device=table.device)
    qsl[1:] = torch.cumsum(n, 0)
    lens = torch.where(granted, c + n, 0)
    t = torch.arange(T, device=table.device)
    r = torch.searchsorted(qsl[1:], t, right=True)
    pos = c[r] + t - qsl[r]
    entry = new_table[r, pos // B].long()
    slots = torch.where(granted[r] & (entry >= 0), entry * B + pos % B, -1)
    place = torch.arange(blocks, device=table.device)
    ref = s["ref"].clone()
    ids = queue[(head + place) % blocks].long()
    ref = torch.where(torch.zeros_like(ref).index_add(0, ids, (place < taken).int()) > 0, 1, ref)
    state = torch.stack([(head + taken) % blocks, count - taken])
    return {"block_table": new_table, "query_start_loc": qsl.int(), "seq_lens": lens.int(), "slot_mapping": slots,
            "free_state": state.int(), "ref_cnt": ref.int()}


def _release(s):
    B, table, queue, ref = s["case"]["block"], s["table"], s["queue"], s["ref0"]
    blocks, width = queue.numel(), table.shape[1]
    head, count = s["state"][0].long(), s["state"][1].long()
    rows = s["rows"].long()
    used = (s["held"][rows].long() + B - 1) // B
    # the order of release: row after row, each from its last block to its first
    col = torch.arange(width - 1, -1, -1, device=table.device)
    ids = table[rows].flip(1).long()
    mask = (col < used.view(-1, 1)).flatten()
    ids = torch.where(mask, ids.flatten(), blocks)
    left = torch.cat([ref, ref.new_zeros(1)]).index_add(0, ids, -mask.int())
    at = torch.arange(ids.numel(), device=table.device)
    last = torch.full((blocks + 1,), -1, device=table.device).scatter_reduce(0, ids, at, "amax")
    gone = mask & (left[ids] == 0) & (last[ids] == at)
    rank = torch.cumsum(gone, 0) - 1
    to = torch.where(gone, (head + count + rank) % blocks, blocks)
    new_queue = torch.cat([queue, queue.new_zeros(1)]).scatter(0, to, ids.int())[:blocks]
    return {"free_queue": new_queue, "free_state": torch.stack([head, count + gone.sum()]).int(), "ref_cnt": left[:blocks]}


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    reqs = _requests(case)
    B = case["block"]
    if case["op"] == "attention":
        hq, hkv, d = case["hq"], case["hkv"], case["d"]
        rows, keys, pairs, entries = 0, 0, 0, 0
        for (n, c), (begin, end) in zip(reqs, _ranges(case, reqs)):
            rows += n
            pairs += sum(max(0, e - b) for b, e in zip(begin, end))
            seen = [(b, e) for b, e in zip(begin, end) if e > b]
            at = 0  # keys that some row sees
            for b, e in sorted(seen):
                keys += max(0, e - max(b, at))
                entries += max(0, -(-e // B) - max(b, at) // B)
                at = max(at, e)
        masks = (case["mask"] in ("window", "documents")) + (case["mask"] in ("documents", "prefix"))
        return {"bytes": 4 * rows * hq * d + 4 * keys * hkv * d + 4 * entries + 12 * len(reqs) + 4 * masks * rows + 4 * hq * case["alibi"],
                "flops": 4 * d * hq * pairs}
    if case["op"] == "tables":
        T = sum(n for n, _ in reqs)
        need = sum(-(-(n + c) // B) - -(-c // B) for n, c in reqs)
        need = need * 3 // 4 if case["short"] else need
        # lengths in, starts and lengths out, a table entry where a request goes on in a block it has; queue in, table and count out; slots out
        return {"bytes": 16 * len(reqs) + 4 * sum(1 for n, c in reqs if c % B) + 12 * need + 8 * T, "flops": 0}
    held = sum(n + c for n, c in reqs) / len(reqs) * case["rows"]
    entries = held / B
    shared = case["prefix"] / B * case["rows"] * 3 / 4
    # entries in; each released block's count in and out, and its place in the queue out
    return {"bytes": int(8 * case["rows"] + 4 * entries + 12 * max(0, entries - shared)), "flops": 0}


# ------------------------------------------------------------------ the same from the definitions, in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    return {"attention": _exact_attention, "tables": _exact_tables, "release": _exact_release}[case["op"]](s)


def _exact_attention(s):
    case = s["case"]
    B, hq, hkv, d, cap = case["block"], case["hq"], case["hkv"], case["d"], case["softcap"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=s["q"].device)
    ranges = _ranges(case, s["reqs"])
    t0 = 0
    for r, ((n, c), (begin, end)) in enumerate(zip(s["reqs"], ranges)):
        lo = torch.tensor(begin, device=out.device)
        hi = torch.tensor(end, device=out.device)
        for g in range(hkv):
            for i0 in range(0, n, 512):
                i1 = min(n, i0 + 512)
                first, past = min(begin[i0:i1]), max(max(end[i0:i1]), min(begin[i0:i1]) + 1)
                j = torch.arange(first, past, device=out.device)
                block, off = s["table"][r, j // B].long(), j % B
                keys, vals = s["kv"][block, 0, off, g].double(), s["kv"][block, 1, off, g].double()
                p = torch.arange(c + i0, c + i1, device=out.device)
                hidden = (j[None, :] < lo[i0:i1, None]) | (j[None, :] >= hi[i0:i1, None])
                for h in range(g * hq // hkv, (g + 1) * hq // hkv):
                    x = torch.einsum("id,jd->ij", s["q"][t0 + i0:t0 + i1, h].double(), keys).mul_(s["scale"])
                    if cap:
                        x = x.div_(cap).tanh_().mul_(cap)
                    if s["slopes"] is not None:
                        x = x.sub_(float(s["slopes"][h]) * (p[:, None] - j[None, :]).abs())
                    x.masked_fill_(hidden, -math.inf)
                    x = x.sub_(torch.logsumexp(x, 1, keepdim=True)).exp_()
                    out[t0 + i0:t0 + i1, h] = torch.einsum("ij,jd->id", torch.nan_to_num_(x, nan=0.0), vals)
        t0 += n
    return out


def _exact_tables(s):
    B, blocks = s["case"]["block"], s["queue"].numel()
    queue, table, ref = s["queue"].tolist(), s["table"].cpu().clone(), s["ref"].tolist()
    head, count = s["state"].tolist()
    free = deque(queue[(head + i) % blocks] for i in range(count))
    qsl, lens, slots, full = [0], [], [], False
    for r, (n, c) in enumerate(s["reqs"]):
        qsl.append(qsl[-1] + n)
        have, total = (c + B - 1) // B, (c + n + B - 1) // B
        if total > have and (full or total - have > len(free)):
            full = True  # first come, first served: nobody behind takes blocks before this one
            table[r, have:total] = -1
            lens.append(0)
            slots += [-1] * n
            continue
        for e in range(have, total):
            b = free.popleft()
            table[r, e] = b
            ref[b] = 1
        lens.append(c + n)
        row = table[r].tolist()
        slots += [row[p // B] * B + p % B for p in range(c, c + n)]
    taken = count - len(free)
    return {"block_table": table, "query_start_loc": torch.tensor(qsl, dtype=torch.int32), "seq_lens": torch.tensor(lens, dtype=torch.int32),
            "slot_mapping": torch.tensor(slots), "free_state": torch.tensor([(head + taken) % blocks, count - taken], dtype=torch.int32),
            "ref_cnt": torch.tensor(ref, dtype=torch.int32)}


def _exact_release(s):
    B, blocks = s["case"]["block"], s["queue"].numel()
    queue, table, ref, held = s["queue"].tolist(), s["table"].tolist(), s["ref0"].tolist(), s["held"].tolist()
    head, count = s["state"].tolist()
    for r in s["rows"].tolist():
        for e in range((held[r] + B - 1) // B - 1, -1, -1):
            b = table[r][e]
            ref[b] -= 1
            if ref[b] == 0:
                queue[(head + count) % blocks] = b
                count += 1
    return {"free_queue": torch.tensor(queue, dtype=torch.int32), "free_state": torch.tensor([head, count], dtype=torch.int32),
            "ref_cnt": torch.tensor(ref, dtype=torch.int32)}
