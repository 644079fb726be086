"""The paged-cache operators as measured work: plain forms in elementary torch
operations, and (``own``) the library's calls a user's program makes.

Operators: rope_append (rotary positions and the append to the pages),
attention_paged (one new token per row over the pages), pages_fork and
pages_compact (bookkeeping and page copies), beam_select (the best beams over
beams x vocabulary).
"""
import random

import torch

own = False

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZES = {"f32": 4, "f16": 2, "bf16": 2}
# (query heads, KV heads, head size): the repository's 135M and 7B shapes, then
# ungrouped, wide and odd groups
HEADS = [(9, 3, 64), (32, 8, 128), (8, 8, 64), (16, 2, 128), (5, 5, 128), (14, 2, 64), (6, 1, 64), (7, 1, 128)]


# ------------------------------------------------------------------ the cases

def listed():
    return [
        # four beams of one prompt, one new token each, the 135M model's heads: a call whose latency counts
        dict(name="rope_step_135m", op="rope", rows=4, seqs=4, heads=9, kv=3, dim=64, rot=64, style=0, page=16,
             type="f32", far=331, stretch=1.0),
        # prompts of three sequences appended together, half-layout rotation of half of each head, positions
        # behind a long context with stretched frequencies
        dict(name="rope_prompts_7b", op="rope", rows=8195, seqs=3, heads=32, kv=8, dim=128, rot=64, style=1, page=64,
             type="bf16", far=120000, stretch=8.0),
        # one sequence at the end of the repository's 203-token prompt and 128 steps
        dict(name="attn_one_135m", op="attention", rows=1, heads=9, kv=3, dim=64, page=16, type="f32", max_len=331,
             window=0, empties=False),
        # a served batch of the 135M model up to its 4096 positions, in the framework's f32
        dict(name="attn_batch_135m", op="attention", rows=48, heads=9, kv=3, dim=64, page=32, type="f32",
             max_len=4096, window=0, empties=True),
        # one long document on the 7B heads: the length has to be split
        dict(name="attn_long_7b", op="attention", rows=1, heads=32, kv=8, dim=128, page=64, type="bf16",
             max_len=131071, window=0, empties=False),
        # a served batch on the 7B heads, ragged, some rows empty
        dict(name="attn_batch_7b", op="attention", rows=64, heads=32, kv=8, dim=128, page=16, type="f16",
             max_len=8191, window=0, empties=True),
        # four groups of four beams of the 135M model after a step
        dict(name="fork_135m", op="fork", groups=4, beams=4, layers=30, kv=3, dim=64, page=16, type="f32",
             max_len=331, reserve=1),
        # sixteen groups of four beams on the 7B heads
        dict(name="fork_7b", op="fork", groups=16, beams=4, layers=32, kv=8, dim=128, page=64, type="bf16",
             max_len=400, reserve=1),
        # a small pool after half of its sequences ended
        dict(name="compact_135m", op="compact", rows=24, layers=30, kv=3, dim=64, page=16, type="f32", max_len=331,
             drop=2),
        # a pool of the 7B heads after a third of its sequences ended
        dict(name="compact_7b", op="compact", rows=36, layers=32, kv=8, dim=128, page=64, type="f16", max_len=509,
             drop=3),
        # four beams over the 135M vocabulary
        dict(name="beam_135m", op="beam", groups=1, beams=4, vocab=49152, n_out=8),
        # a batch of beam groups over a large, odd vocabulary
        dict(name="beam_batch", op="beam", groups=48, beams=5, vocab=100003, n_out=10),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, round(lo * (hi / lo) ** rng.random())))


def draw(rng):
    most = {}
    for c in listed():
        w = work(c)
        most[c["op"]] = max(most.get(c["op"], 0), w["bytes"])
    op = rng.choice(["rope", "attention", "attention", "fork", "compact", "beam"])
    while True:
        heads, kv, dim = rng.choice(HEADS)
        kind, page = rng.choice(sorted(TYPES)), rng.choice([8, 16, 32, 64, 128])
        if op == "rope":
            rows = _log(rng, 1, 8195)
            c = dict(op=op, rows=rows, seqs=rng.randint(1, min(rows, 64)), heads=heads, kv=kv, dim=dim,
                     rot=rng.choice([dim, dim // 2, dim // 4]), style=rng.randint(0, 1), page=page, type=kind,
                     far=_log(rng, 1, 200000), stretch=rng.choice([1.0, 2.0, 8.0]))
        elif op == "attention":
            rows, max_len = _log(rng, 1, 64), _log(rng, 1, 131071)
            c = dict(op=op, rows=rows, heads=heads, kv=kv, dim=dim, page=page, type=kind, max_len=max_len,
                     window=rng.choice([0, 0, _log(rng, 1, max_len)]), empties=rng.random() < 0.5)
            if rows * max_len * kv * dim > 64 * 8191 * 8 * 128:  # what the plain form gathers
                continue
        elif op == "fork":
            c = dict(op=op, groups=_log(rng, 1, 32), beams=rng.randint(1, 8), layers=rng.randint(1, 32), kv=kv,
                     dim=dim, page=page, type=kind, max_len=_log(rng, 1, 1000), reserve=rng.randint(0, 3))
        elif op == "compact":
            c = dict(op=op, rows=_log(rng, 2, 64), layers=rng.randint(1, 32), kv=kv, dim=dim, page=page, type=kind,
                     max_len=_log(rng, 1, 1000), drop=rng.randint(2, 5))
        else:
            c = dict(op=op, groups=_log(rng, 1, 64), beams=rng.randint(1, 8), vocab=_log(rng, 64, 130000),
                     n_out=0)
            c["n_out"] = c["beams"] * rng.randint(1, 2)
        if op in ("fork", "compact") and _pool_bytes(c) > 3 << 30:
            continue
        if work(c)["bytes"] <= most[op]:
            return c


# ------------------------------------------------------------------ what a case holds, whatever the seed

def _lengths(case, n):
    """Lengths spread over 1 .. max_len; the first row has the largest."""
    top = case["max_len"]
    out = [top] + [1 + int((top - 1) * ((r * 0.6180339887498949) % 1.0)) for r in range(1, n)]
    if case.get("empties"):
        out = [0 if r % 7 == 6 else x for r, x in enumerate(out)]
    return out


def _blocks(n, page):
    return -(-n // page)


def _append_positions(case):
    """seq and pos of every appended row: the rows dealt over the sequences in runs, each at its own start."""
    rows, seqs = case["rows"], case["seqs"]
    seq, pos = [], []
    for s in range(seqs):
        n = rows // seqs + (1 if s < rows % seqs else 0)
        start = (case["far"] * (s + 1)) // seqs
        seq += [s] * n
        pos += list(range(start, start + n))
    return seq, pos


def _fork_plan(case):
    """Lengths of the beams (one length per group) and the parents the beams chose."""
    rng = random.Random(case["groups"] * 1009 + case["beams"])
    per = _lengths(case, case["groups"])
    lens = [per[g] for g in range(case["groups"]) for _ in range(case["beams"])]
    parent = []
    for g in range(case["groups"]):
        chosen = [min(int(rng.expovariate(1.2)), case["beams"] - 1) for _ in range(case["beams"])]
        parent += [g * case["beams"] + c for c in chosen]
    return lens, parent


def _fork_copies(case):
    """Valid positions copied into new pages: every child but the first of a parent whose last page is partly filled."""
    lens, parent = _fork_plan(case)
    seen, n = set(), 0
    for p in parent:
        if p in seen:
            n += lens[p] % case["page"]
        seen.add(p)
    return n


def _pool(case):
    """Pages of a fork or compact case: what the rows hold, and free ones."""
    if case["op"] == "fork":
        lens, _ = _fork_plan(case)
        used = sum(_blocks(n, case["page"]) for n in lens)
        return used + 2 * len(lens) * (1 + _blocks(case["reserve"], case["page"])) + 3
    return sum(_blocks(n, case["page"]) for n in _lengths(case, case["rows"])) + 5


def _pool_bytes(case):
    return 2 * _pool(case) * case["layers"] * case["kv"] * case["page"] * case["dim"] * SIZES[case["type"]]


def _compact_plan(case):
    """Page ids of every kept row (None: the row has ended), and how many pages move."""
    rng = random.Random(case["rows"] * 31 + case["drop"])
    ids = list(range(_pool(case)))
    rng.shuffle(ids)
    rows, at = [], 0
    for r, n in enumerate(_lengths(case, case["rows"])):
        b = _blocks(n, case["page"])
        rows.append(None if r % case["drop"] == case["drop"] - 1 else ids[at:at + b])
        at += b
    held = sorted(p for r in rows if r for p in r)
    return rows, sum(p >= len(held) for p in held)


def work(case):
    size = SIZES.get(case.get("type"), 4)
    if case["op"] == "rope":
        h, kv, d, n = case["heads"], case["kv"], case["dim"], case["rows"]
        return {"bytes": n * ((h + 2 * kv) * d * 4 + h * d * 4 + 2 * kv * d * size + 8) + case["rot"] * 4,
                "flops": 3 * n * (h + kv) * case["rot"]}
    if case["op"] == "attention":
        lens = [min(n, case["window"]) if case["window"] else n for n in _lengths(case, case["rows"])]
        total = sum(lens)
        return {"bytes": 2 * total * case["kv"] * case["dim"] * size + case["rows"] * case["heads"] * (case["dim"] * 8 + 4)
                + 4 * sum(_blocks(n, case["page"]) for n in lens) + 4 * case["rows"],
                "flops": 4 * total * case["heads"] * case["dim"]}
    if case["op"] == "fork":
        rows = case["groups"] * case["beams"]
        width = _blocks(case["max_len"] + case["reserve"], case["page"]) + 2
        return {"bytes": 4 * _fork_copies(case) * case["layers"] * case["kv"] * case["dim"] * size
                + 8 * rows * width + 8 * _pool(case) + 12 * rows, "flops": 0}
    if case["op"] == "compact":
        moved = _compact_plan(case)[1]
        width = _blocks(case["max_len"], case["page"]) + 1
        return {"bytes": 4 * moved * case["layers"] * case["kv"] * case["page"] * case["dim"] * size
                + 8 * case["rows"] * width + 8 * _pool(case), "flops": 0}
    rows = case["groups"] * case["beams"]
    return {"bytes": 4 * rows * case["vocab"] + 4 * rows + 12 * case["groups"] * case["n_out"],
            "flops": 4 * rows * case["vocab"]}


# ------------------------------------------------------------------ inputs

def _normal(shape, g, kind, scale=1.0):
    return (torch.randn(shape, generator=g, device="cuda", dtype=torch.float32) * scale).to(kind)


def _cache(layers, pages, case, g):
    """K and V pages; keys have a few strong channels, as keys of trained models do."""
    shape = (layers, pages, case["kv"], case["page"], case["dim"])
    kind = TYPES[case["type"]]
    k, v = torch.empty(shape, dtype=kind, device="cuda"), torch.empty(shape, dtype=kind, device="cuda")
    for layer in range(layers):
        k[layer] = _normal(shape[1:], g, kind)
        v[layer] = _normal(shape[1:], g, kind, 0.7)
    k[..., 3] *= 4
    k[..., case["dim"] // 2 + 1] *= 4
    return k, v


def _ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    st = dict(case=case)
    if case["op"] == "rope":
        seq, pos = _append_positions(case)
        page = case["page"]
        top = [0] * case["seqs"]
        low = [1 << 30] * case["seqs"]
        for s, p in zip(seq, pos):
            top[s], low[s] = max(top[s], p // page), min(low[s], p // page)
        width = max(top) + 2
        # the pages behind the appended positions are not part of this call's work: one page stands for them
        n = sum(t - b + 1 for t, b in zip(top, low)) + 1
        ids = torch.randperm(n, generator=g, device="cuda").to(torch.int32)
        table = torch.full((case["seqs"], width), -1, dtype=torch.int32, device="cuda")
        at = 1
        for s in range(case["seqs"]):
            table[s, :low[s]] = ids[0]
            table[s, low[s]:top[s] + 1] = ids[at:at + top[s] - low[s] + 1]
            at += top[s] - low[s] + 1
        st["k"], st["v"] = _cache(1, n, case, g)
        st["qkv"] = _normal((case["rows"], (case["heads"] + 2 * case["kv"]) * case["dim"]), g, torch.float32)
        half = torch.arange(case["rot"] // 2, dtype=torch.float64, device="cuda")
        st["freq"] = 10000.0 ** (-2.0 * half / case["rot"]) / case["stretch"]
        st["magnitude"] = 1.0 if case["stretch"] == 1.0 else 1.1
        st.update(seq=_ints(seq), pos=_ints(pos), table=table,
                  q_out=torch.zeros((case["rows"], case["heads"], case["dim"]), device="cuda"))
    elif case["op"] == "attention":
        lens = _lengths(case, case["rows"])
        blocks = [_blocks(n, case["page"]) for n in lens]
        ids = torch.randperm(sum(blocks) + 3, generator=g, device="cuda").to(torch.int32)
        table = torch.full((case["rows"], max(blocks) + 1), -1, dtype=torch.int32, device="cuda")
        at = 0
        for r, b in enumerate(blocks):
            table[r, :b] = ids[at:at + b]
            at += b
        st["k"], st["v"] = _cache(1, ids.numel(), case, g)
        st.update(q=_normal((case["rows"], case["heads"], case["dim"]), g, torch.float32, 1.5), table=table,
                  pos=_ints([n - 1 for n in lens]),
                  out=torch.empty((case["rows"], case["heads"], case["dim"]), device="cuda"),
                  lse=torch.empty((case["rows"], case["heads"]), device="cuda"))
    elif case["op"] == "fork":
        lens, parent = _fork_plan(case)
        n = _pool(case)
        width = _blocks(case["max_len"] + case["reserve"], case["page"]) + 2
        ids = torch.randperm(n, generator=g, device="cuda").to(torch.int32)
        table = torch.full((len(lens), width), -1, dtype=torch.int32, device="cuda")
        refs = torch.zeros(n, dtype=torch.int32, device="cuda")
        at = 0
        for grp in range(case["groups"]):
            full = lens[grp * case["beams"]] // case["page"]
            tail = _blocks(lens[grp * case["beams"]], case["page"]) - full
            shared = ids[at:at + full]  # the beams of a group share the pages they filled together
            at += full
            for b in range(case["beams"]):
                row = grp * case["beams"] + b
                table[row, :full] = shared
                table[row, full:full + tail] = ids[at:at + tail]
                at += tail
        held = table[table >= 0].long()
        refs.index_add_(0, held, torch.ones_like(held, dtype=torch.int32))
        st["k"], st["v"] = _cache(case["layers"], n, case, g)
        st.update(parent=_ints(parent), len_in=_ints(lens), table_in=table, refs_in=refs,
                  len_out=torch.empty_like(_ints(parent)), table_out=torch.empty_like(table),
                  refs_out=torch.empty_like(refs))
    elif case["op"] == "compact":
        rows, _ = _compact_plan(case)
        n = _pool(case)
        width = _blocks(case["max_len"], case["page"]) + 1
        table = _ints([(r or []) + [-1] * (width - len(r or [])) for r in rows])
        refs = torch.zeros(n, dtype=torch.int32, device="cuda")
        refs[table[table >= 0].long()] = 1
        st["k"], st["v"] = _cache(case["layers"], n, case, g)
        st.update(table_in=table, refs_in=refs, table_out=torch.empty_like(table), refs_out=torch.empty_like(refs),
                  n_used=torch.empty(1, dtype=torch.int32, device="cuda"))
    else:
        rows, n = case["groups"] * case["beams"], case["groups"] * case["n_out"]
        logits = _normal((rows, case["vocab"]), g, torch.float32, 2.0)
        likely = torch.randint(0, case["vocab"], (rows, 12), generator=g, device="cuda")
        logits.scatter_(1, likely, 9.0 + _normal((rows, 12), g, torch.float32, 1.5))
        st.update(logits=logits, scores=-10.0 * torch.rand(rows, generator=g, device="cuda"),
                  out_scores=torch.empty(n, device="cuda"), out_parent=torch.empty(n, dtype=torch.int32, device="cuda"),
                  out_token=torch.empty(n, dtype=torch.int32, device="cuda"))
    if own:
        _keep(st)
    return st


# ------------------------------------------------------------------ the library's calls

def _keep(st):
    """What a program that uses the library keeps: the pool's description, its rotation, a workspace."""
    from q8_quantized_llama_gb300 import binding as B
    case = st["case"]
    st["err"] = torch.zeros(1, dtype=torch.int32, device="cuda")
    if "k" in st:
        st["pages"] = B.make_pages(st["k"], st["v"])
    if case["op"] == "rope":
        st["rope"] = B.make_rope(st["freq"], case["style"], st["magnitude"])
        return
    if case["op"] == "attention":
        n = B.llama_q8_attention_paged_workspace_bytes(case["rows"], case["heads"], case["kv"], case["dim"])
    elif case["op"] == "fork":
        n = B.llama_q8_pages_fork_workspace_bytes(st["len_in"].numel(), st["parent"].numel(), st["table_in"].shape[1])
    elif case["op"] == "compact":
        n = B.llama_q8_pages_compact_workspace_bytes(st["refs_in"].numel())
    else:
        n = B.llama_q8_beam_select_workspace_bytes(case["groups"], case["beams"], case["vocab"], case["n_out"])
    st["ws"], st["ws_bytes"] = torch.zeros(n, dtype=torch.uint8, device="cuda"), n


def _run_own(st):
    from q8_quantized_llama_gb300 import binding as B
    case = st["case"]
    if case["op"] == "rope":
        qkv, table = st["qkv"], st["table"]
        B.llama_q8_rope_append(st["pages"], 0, qkv, qkv.shape[1], case["rows"], st["pos"], st["seq"], case["heads"],
                               st["rope"], table, table.shape[0], table.shape[1], st["q_out"], st["err"])
        return {"q": st["q_out"], "k": st["k"], "v": st["v"]}
    if case["op"] == "attention":
        table = st["table"]
        B.llama_q8_attention_paged(st["pages"], 0, st["q"], case["rows"], st["pos"], None, case["heads"], 0.0,
                                   case["window"], table, table.shape[0], table.shape[1], st["out"], st["lse"],
                                   st["ws"], st["ws_bytes"], st["err"])
        return {"out": st["out"], "lse": st["lse"]}
    if case["op"] == "fork":
        table = st["table_in"]
        B.llama_q8_pages_fork(st["pages"], table.shape[0], st["len_in"], table, table.shape[1], st["refs_in"],
                              st["parent"].numel(), st["parent"], case["reserve"], st["len_out"], st["table_out"],
                              st["refs_out"], st["ws"], st["ws_bytes"], st["err"])
        return {"len": st["len_out"], "table": st["table_out"], "refs": st["refs_out"], "k": st["k"], "v": st["v"]}
    if case["op"] == "compact":
        table = st["table_in"]
        B.llama_q8_pages_compact(st["pages"], table.shape[0], table, table.shape[1], st["refs_in"], st["table_out"],
                                 st["refs_out"], st["n_used"], st["ws"], st["ws_bytes"], st["err"])
        return {"table": st["table_out"], "refs": st["refs_out"], "used": st["n_used"], "k": st["k"], "v": st["v"]}
    logits = st["logits"]
    B.llama_q8_beam_select(logits, logits.shape[1], case["groups"], case["beams"], case["vocab"], st["scores"],
                           case["n_out"], st["out_scores"], st["out_parent"], st["out_token"], st["ws"],
                           st["ws_bytes"])
    return {"scores": st["out_scores"], "parent": st["out_parent"], "token": st["out_token"]}


# ------------------------------------------------------------------ the plain forms

def run(st):
    if own:
        return _run_own(st)
    return {"rope": _rope, "attention": _attention, "fork": _fork, "compact": _compact, "beam": _beam}[
        st["case"]["op"]](st)


def _rope(st):
    case = st["case"]
    h, kv, d, rot = case["heads"], case["kv"], case["dim"], case["rot"]
    x = st["qkv"].view(case["rows"], h + 2 * kv, d)
    # far positions: the angle in 64 bits
    a = st["pos"].double()[:, None] * st["freq"][None, :]
    c, s = (torch.cos(a) * st["magnitude"]).float()[:, None], (torch.sin(a) * st["magnitude"]).float()[:, None]
    qk = x[:, :h + kv].clone()
    if case["style"] == 0:
        one, two = x[:, :h + kv, 0:rot:2], x[:, :h + kv, 1:rot:2]
        qk[..., 0:rot:2], qk[..., 1:rot:2] = one * c - two * s, one * s + two * c
    else:
        one, two = x[:, :h + kv, :rot // 2], x[:, :h + kv, rot // 2:rot]
        qk[..., :rot // 2], qk[..., rot // 2:rot] = one * c - two * s, one * s + two * c
    pos = st["pos"].long()
    page, slot = st["table"][st["seq"].long(), pos // case["page"]].long(), pos % case["page"]
    st["k"][0, page, :, slot] = qk[:, h:].to(st["k"].dtype)
    st["v"][0, page, :, slot] = x[:, h + kv:].to(st["v"].dtype)
    return {"q": qk[:, :h].contiguous(), "k": st["k"], "v": st["v"]}


def _attention(st):
    case = st["case"]
    rows, h, kv, d = case["rows"], case["heads"], case["kv"], case["dim"]
    t = st["table"].clamp(min=0).long()
    span = t.shape[1] * case["page"]
    k = st["k"][0][t].transpose(1, 2).reshape(rows, kv, span, d).float()
    v = st["v"][0][t].transpose(1, 2).reshape(rows, kv, span, d).float()
    at, pos = torch.arange(span, device="cuda")[None, :], st["pos"].long()[:, None]
    see = at <= pos
    if case["window"]:
        see = see & (at > pos - case["window"])
    see = see[:, None, None, :]
    score = (st["q"].view(rows, kv, h // kv, d) @ k.transpose(-1, -2)) * d ** -0.5
    score = torch.where(see, score, float("-inf"))
    top = score.amax(-1, keepdim=True)
    top = torch.where(top == float("-inf"), 0.0, top)
    p = torch.exp(score - top)
    total = p.sum(-1, keepdim=True)
    v = torch.where(see[:, 0, 0, :][:, None, :, None], v, 0.0)
    out = (p @ v) / torch.where(total == 0, 1.0, total)
    return {"out": out.reshape(rows, h, d), "lse": (top + torch.log(total)).reshape(rows, h)}


def _fork(st):
    case = st["case"]
    parent, table, refs, page = st["parent"].long(), st["table_in"], st["refs_in"], case["page"]
    t, n = table[parent], st["len_in"][parent].long()[:, None]
    full, part, need = n // page, n % page, (n + case["reserve"] + page - 1) // page
    first = ~(parent[:, None] == parent[None, :]).tril(-1).any(1, keepdim=True)
    b = torch.arange(t.shape[1], device="cuda")[None, :]
    held = t >= 0
    kept = held & ((b < full) | (first & (refs[t.clamp(min=0).long()] == 1)))
    new = ~kept & (b >= full) & (b < need)
    free = torch.sort((refs != 0).to(torch.int32), stable=True).indices
    rank = (torch.cumsum(new.flatten().long(), 0) - 1).clamp(min=0).view(new.shape)
    out = torch.where(kept, t.long(), torch.where(new, free[rank], -1))
    refs_out = refs.clone()
    before, after = table[table >= 0].long(), out[out >= 0]
    refs_out.index_add_(0, before, torch.full_like(before, -1, dtype=torch.int32))
    refs_out.index_add_(0, after, torch.ones_like(after, dtype=torch.int32))
    copied = new & held & (b == full) & (part > 0)
    src, dst, valid = t[copied].long(), out[copied], part.expand(copied.shape)[copied]
    valid = (torch.arange(page, device="cuda")[None, :] < valid[:, None])[None, :, None, :, None]
    for x in (st["k"], st["v"]):
        x[:, dst] = torch.where(valid, x[:, src], x[:, dst])
    return {"len": n[:, 0].int(), "table": out.int(), "refs": refs_out, "k": st["k"], "v": st["v"]}


def _compact(st):
    table, refs = st["table_in"], st["refs_in"]
    ids, used = torch.arange(refs.numel(), device="cuda"), refs > 0
    n = used.sum()
    src, dst = ids[used & (ids >= n)], ids[~used & (ids < n)]
    to = ids.clone()
    to[src] = dst
    for x in (st["k"], st["v"]):
        x[:, dst] = x[:, src]
    refs_out = torch.zeros_like(refs)
    refs_out[to[used]] = refs[used]
    out = torch.where(table >= 0, to[table.clamp(min=0).long()].int(), -1)
    return {"table": out.int(), "refs": refs_out, "used": n.int().view(1), "k": st["k"], "v": st["v"]}


def _beam(st):
    case = st["case"]
    x = st["logits"]
    top = x.amax(1, keepdim=True)
    # totals of different beams lie next to each other: the long sum and the totals in 64 bits
    lse = top.double() + torch.log(torch.exp(x - top).sum(1, keepdim=True, dtype=torch.float64))
    total = (st["scores"].double()[:, None] + (x.double() - lse)).view(case["groups"], -1)
    val, at = torch.topk(total, min(case["n_out"] + 8, total.shape[1]), dim=1)
    at, order = torch.sort(at, dim=1)
    val, order = torch.sort(val.gather(1, order), dim=1, descending=True, stable=True)
    at = at.gather(1, order)[:, :case["n_out"]]
    base = torch.arange(case["groups"], device="cuda")[:, None] * case["beams"]
    return {"scores": val[:, :case["n_out"]].float().flatten(),
            "parent": (base + at // case["vocab"]).int().flatten(), "token": (at % case["vocab"]).int().flatten()}


# ------------------------------------------------------------------ the definitions, in 64 bits

def exact(case, seed):
    global own
    was, own = own, False
    try:
        st = prepare(case, seed)
    finally:
        own = was
    return {"rope": _exact_rope, "attention": _exact_attention, "fork": _exact_fork, "compact": _exact_compact,
            "beam": _exact_beam}[case["op"]](case, st)


def _exact_rope(case, st):
    # the rotation as a product of complex numbers
    h, kv, rot = case["heads"], case["kv"], case["rot"]
    x = st["qkv"].double().view(case["rows"], -1, case["dim"])
    turn = torch.polar(torch.full_like(st["freq"], st["magnitude"]).expand(case["rows"], -1),
                       torch.outer(st["pos"].double(), st["freq"]))
    head = x[:, :h + kv, :rot]
    if case["style"] == 0:
        z = torch.view_as_complex(head.reshape(case["rows"], h + kv, rot // 2, 2).contiguous())
        z = torch.view_as_real(z * turn[:, None]).reshape(case["rows"], h + kv, rot)
    else:
        z = torch.complex(head[..., :rot // 2], head[..., rot // 2:]) * turn[:, None]
        z = torch.cat([z.real, z.imag], -1)
    x = torch.cat([torch.cat([z, x[:, :h + kv, rot:]], -1), x[:, h + kv:]], 1)
    k, v = st["k"].double(), st["v"].double()
    page, slot = st["pos"].long() // case["page"], st["pos"].long() % case["page"]
    where = st["table"].long()[st["seq"].long(), page]
    for i in range(kv):
        k[0, where, i, slot] = x[:, h + i]
        v[0, where, i, slot] = x[:, h + kv + i]
    return {"q": x[:, :h].contiguous(), "k": k, "v": v}


def _exact_attention(case, st):
    h, kv, d = case["heads"], case["kv"], case["dim"]
    out = torch.zeros((case["rows"], h, d), dtype=torch.float64, device="cuda")
    lse = torch.full((case["rows"], h), float("-inf"), dtype=torch.float64, device="cuda")
    for r, n in enumerate(_lengths(case, case["rows"])):
        if n == 0:
            continue
        lo = max(0, n - case["window"]) if case["window"] else 0
        at = torch.arange(lo, n, device="cuda")
        page = st["table"][r].long()[at // case["page"]]
        k, v = (x[0][page, :, at % case["page"]].double() for x in (st["k"], st["v"]))
        q = st["q"][r].double().view(kv, h // kv, d)
        s = torch.einsum("ngd,tnd->ngt", q, k) / d ** 0.5
        z = torch.logsumexp(s, -1)
        lse[r] = z.reshape(h)
        out[r] = torch.einsum("ngt,tnd->ngd", torch.exp(s - z[..., None]), v).reshape(h, d)
    return {"out": out, "lse": lse}


def _exact_fork(case, st):
    page = case["page"]
    lens, table, refs = st["len_in"].tolist(), st["table_in"].tolist(), st["refs_in"].tolist()
    free = iter([p for p, n in enumerate(refs) if n == 0])
    count, seen, out, lens_out = list(refs), set(), [], []
    for row in table:
        for p in row:
            if p >= 0:
                count[p] -= 1
    for p in st["parent"].tolist():
        n, row = lens[p], []
        for b, old in enumerate(table[p]):
            if b < n // page or (old >= 0 and p not in seen and refs[old] == 1):
                row.append(old)
            elif b < _blocks(n + case["reserve"], page):
                row.append(next(free))
                if b == n // page and n % page:
                    for x in (st["k"], st["v"]):
                        x[:, row[-1], :, :n % page] = x[:, old, :, :n % page]
            else:
                row.append(-1)
        for x in row:
            if x >= 0:
                count[x] += 1
        seen.add(p)
        out.append(row)
        lens_out.append(n)
    return {"len": _ints(lens_out), "table": _ints(out), "refs": _ints(count), "k": st["k"], "v": st["v"]}


def _exact_compact(case, st):
    refs, table = st["refs_in"].tolist(), st["table_in"].tolist()
    n = sum(r > 0 for r in refs)
    holes = iter([p for p in range(n) if refs[p] == 0])
    to, count = {}, [0] * len(refs)
    for p, r in enumerate(refs):
        if r > 0:
            to[p] = p if p < n else next(holes)
            count[to[p]] = r
            if to[p] != p:
                for x in (st["k"], st["v"]):
                    x[:, to[p]] = x[:, p]
    return {"table": _ints([[to.get(p, -1) for p in row] for row in table]), "refs": _ints(count),
            "used": _ints([n]), "k": st["k"], "v": st["v"]}


def _exact_beam(case, st):
    scores, parent, token = [], [], []
    for g in range(case["groups"]):
        rows = slice(g * case["beams"], (g + 1) * case["beams"])
        total = st["scores"][rows, None].double() + torch.log_softmax(st["logits"][rows].double(), 1)
        val, at = torch.sort(total.flatten(), descending=True, stable=True)
        at = at[:case["n_out"]]
        scores.append(val[:case["n_out"]])
        parent.append(at // case["vocab"] + g * case["beams"])
        token.append(at % case["vocab"])
    return {"scores": torch.cat(scores), "parent": torch.cat(parent).int(), "token": torch.cat(token).int()}
