"""What is measured of the operators around many continuations of one prompt over the paged 8-bit cache: pages copied, sequences
forked, reordered and freed, the cache compacted, attention over a prefix that sequences share, and the next tokens drawn from logits.

The cache is that of perf/operators.py: codes of shape (pages, kv_heads, page, head_dim), one float32 scale for each (page, kv_head).
A sequence's pages are the leading entries of its row of `table`, -1 after them; `refs` counts the entries that hold each page (0: it is
free). Pages that a sequence has filled may be shared; the others ("open": the partly filled one and empty ones behind it) are its own.

The plain forms below are elementary torch operations: whole numbers exactly, attention in 32 bits, and weights, sums and borders of
the drawing in 64.
"""
import math
import random

import torch

own = False

STORE = {"e4m3": torch.float8_e4m3fn, "int8": torch.int8}
TYPE = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}


# ---------------------------------------------------------------- cases

def listed():
    return [
        # a beam search over one prompt: reordered by the parents of the step, an open page copied, room for the next token (latency)
        _fork("fork_beams", prompts=1, beams=4, longest=1023, mix=1),
        # many prompts with a beam each, long tables, reordered at once
        _fork("fork_batch_int8", prompts=32, beams=8, longest=8192, page=128, store="int8", mix=2),
        # a small pool with a few sequences in it (latency)
        _compact("compact_small", pages=301, batch=5, share=0.6, page=16, kv_heads=4, head_dim=64, store="int8", mix=3),
        # a pool of 2 GB that is a little over half full, with its holes all over it
        _compact("compact_pool", pages=16384, batch=64, share=0.55, mix=4),
        # a few pages handed to another cache (latency)
        _copy("copy_few", pages=7, pool=64, page=16, kv_heads=4, head_dim=64),
        # the pages of long sequences handed to another cache, in any order
        _copy("copy_sequences", pages=5003, pool=8192, store="int8"),
        # eight answers to one prompt, a token each (latency)
        _attend("attend_answers", sizes="8", prefix=1000, tail=70, mix=5),
        # a decode step of a full batch behind one long instruction, own parts of several lengths, two slots idle
        _attend("attend_instruction", sizes="64", prefix=8192, tail=2000, idle=2, lse=True, mix=6),
        # documents with several questions each and a few drafted tokens, seven query heads a key head, heads of 64, small pages
        _attend("attend_documents", sizes="9,17,2,12", prefix=30011, tail=517, most=5, heads=28, kv_heads=4, head_dim=64, page=16,
                store="int8", dtype="bf16", mix=7),
        # one sequence's next token (latency)
        _sample("sample_one", rows=1, vocab=32000, how="nucleus", dtype="fp16"),
        # a decode step's batch, every row with settings of its own, a few of them greedy, an odd vocabulary
        _sample("sample_mixed", rows=64, vocab=131071, how="mixed", dtype="bf16", mix=8),
        # a large batch of logits in 32 bits, cut by their mass alone
        _sample("sample_nucleus", rows=256, vocab=131072, how="nucleus", dtype="fp32"),
    ]


def draw(rng):
    kind = rng.choice(["fork", "fork", "compact", "copy", "attend", "attend", "attend", "sample", "sample", "sample"])
    store, page, dim, kv = rng.choice(["e4m3", "int8"]), rng.choice([16, 32, 64, 128]), rng.choice([64, 128, 128]), rng.choice([1, 2, 4, 8])
    mix = rng.randrange(1 << 20)
    if kind == "fork":
        prompts = _log(rng, 1, 32)
        case = _fork(None, prompts=prompts, beams=rng.randint(1, 8), longest=_log(rng, 1, 262144 // prompts // 8), room=rng.choice([0, 1, 1, 5, 300]), page=page,
                     kv_heads=kv, head_dim=dim, store=store, mix=mix)
    elif kind == "compact":
        pool = _log(rng, 16, (1 << 31) // (2 * kv * page * dim))
        case = _compact(None, pages=min(pool, 16384), batch=_log(rng, 1, 64), share=rng.uniform(0.05, 0.95), page=page, kv_heads=kv, head_dim=dim, store=store, mix=mix)
    elif kind == "copy":
        pool = min(8192, _log(rng, 16, (1 << 30) // (2 * kv * page * dim)))
        case = _copy(None, pages=_log(rng, 1, pool * 5 // 8), pool=pool, page=page, kv_heads=kv, head_dim=dim, store=store)
    elif kind == "attend":
        groups = _log(rng, 1, 4)
        sizes = [_log(rng, 1, 64 // groups) for _ in range(groups)]
        most = 1 if rng.random() < 0.6 else rng.randint(2, 6)
        case = _attend(None, sizes=",".join(map(str, sizes)), prefix=_log(rng, 1, 524288 // sum(sizes) // 2 if sum(sizes) > 16 else 16384), tail=most + _log(rng, 1, 2000), most=most,
                       heads=kv * rng.choice([1, 2, 3, 4, 7, 8]), kv_heads=kv, head_dim=dim, page=page, store=store, dtype=rng.choice(["fp16", "bf16"]),
                       idle=1 if sum(sizes) > 4 and rng.random() < 0.3 else 0, lse=rng.random() < 0.4, mix=mix)
    else:
        rows = _log(rng, 1, 256)
        case = _sample(None, rows=rows, vocab=_log(rng, 2, 131072), how=rng.choice(["plain", "nucleus", "mixed", "mixed"]), dtype=rng.choice(["fp16", "bf16", "fp32"]),
                       spread=rng.uniform(0.5, 4.0), mix=mix)
    case.pop("name")
    return case


def _log(rng, low, high):
    return min(high, max(low, int(round(math.exp(rng.uniform(math.log(low), math.log(high + 0.49)))))))


def _fork(name, prompts, beams, longest, room=1, page=64, kv_heads=8, head_dim=128, store="e4m3", mix=0):
    return {"name": name, "op": "fork", "prompts": prompts, "beams": beams, "longest": longest, "room": room, "page": page, "kv_heads": kv_heads,
            "head_dim": head_dim, "store": store, "mix": mix}


def _compact(name, pages, batch, share, page=64, kv_heads=8, head_dim=128, store="e4m3", mix=0):
    return {"name": name, "op": "compact", "pages": pages, "batch": batch, "share": share, "page": page, "kv_heads": kv_heads, "head_dim": head_dim,
            "store": store, "mix": mix}


def _copy(name, pages, pool, page=64, kv_heads=8, head_dim=128, store="e4m3"):
    return {"name": name, "op": "copy", "pages": pages, "pool": pool, "page": page, "kv_heads": kv_heads, "head_dim": head_dim, "store": store}


def _attend(name, sizes, prefix, tail, most=1, heads=32, kv_heads=8, head_dim=128, page=64, store="e4m3", dtype="fp16", idle=0, lse=False, mix=0):
    return {"name": name, "op": "attend", "sizes": sizes, "prefix": prefix, "tail": tail, "most": most, "heads": heads, "kv_heads": kv_heads,
            "head_dim": head_dim, "page": page, "store": store, "dtype": dtype, "idle": idle, "lse": lse, "mix": mix}


def _sample(name, rows, vocab, how, dtype, spread=2.5, mix=0):
    return {"name": name, "op": "sample", "rows": rows, "vocab": vocab, "how": how, "dtype": dtype, "spread": spread, "mix": mix}


def _trees(case):
    """For each prompt its length and its beams' common length, and each new sequence's parent (one in sixteen ends and is replaced by nothing)."""
    r = random.Random(case["mix"])
    longest, beams = case["longest"], case["beams"]
    shapes, parents = [], []
    for i in range(case["prompts"]):
        whole = longest if i == 0 else r.randint(max(1, longest // 4), longest)
        shapes.append((r.randint(0, whole), whole))
        parents += [-1 if beams > 1 and r.random() < 1 / 16 else i * beams + r.randrange(beams) for _ in range(beams)]
    return shapes, parents


def _groups(case):
    """Sequences of each group, its shared tokens, and new and total tokens of each sequence; the last `idle` ones have none in the cache."""
    r = random.Random(case["mix"])
    sizes = [int(n) for n in case["sizes"].split(",")]
    prefix = [case["prefix"]] + [r.randint(max(1, case["prefix"] // 3), case["prefix"]) for _ in sizes[1:]]
    new, total = [], []
    for n, p in zip(sizes, prefix):
        for _ in range(n):
            k = case["most"] if not new else r.randint(1, case["most"])
            new.append(k)
            total.append(p + r.randint(k, case["tail"]))
    for i in range(case["idle"]):
        total[-1 - i] = 0
    return sizes, prefix, new, total


def _page_bytes(case):
    return 2 * case["kv_heads"] * case["page"] * case["head_dim"] + 8 * case["kv_heads"]


def work(case):
    if case["op"] == "fork":
        shapes, parents = _trees(case)
        page, seen, held, tokens, copies = case["page"], set(), 0, 0, 0
        for p in parents:
            whole = shapes[p // case["beams"]][1] if p >= 0 else 0
            held += -(-(whole + case["room"]) // page)
            if p in seen and whole % page:
                copies, tokens = copies + 1, tokens + whole % page
            seen.add(p)
        nbytes = 2 * (copies * 8 * case["kv_heads"] + tokens * 2 * case["kv_heads"] * case["head_dim"])
        return {"bytes": nbytes + 8 * held + 8 * _pool(case) + 12 * len(parents), "flops": held}
    if case["op"] == "compact":
        used = _used(case)
        moved = int(used * (1 - used / case["pages"]))  # of places drawn at random
        return {"bytes": 2 * moved * _page_bytes(case) + 8 * used + 12 * case["pages"], "flops": case["pages"]}
    if case["op"] == "copy":
        return {"bytes": 2 * case["pages"] * _page_bytes(case) + 8 * case["pages"], "flops": case["pages"]}
    if case["op"] == "sample":
        n = case["rows"] * case["vocab"]
        return {"bytes": n * TYPE[case["dtype"]].itemsize + 24 * case["rows"], "flops": 4 * n}
    sizes, prefix, new, total = _groups(case)
    alive = [t > 0 for t in total]
    row, heads, first = case["kv_heads"] * case["head_dim"], case["heads"] * case["head_dim"], 0
    keys = 0
    for n, p in zip(sizes, prefix):
        keys += p if any(alive[first:first + n]) else 0
        keys += sum(t - p for t in total[first:first + n] if t)
        first += n
    pairs = sum(sum(range(t - k + 1, t + 1)) for k, t in zip(new, total) if t)
    nbytes = keys * row * 2 + -(-keys // case["page"]) * (case["kv_heads"] * 8 + 4) + sum(new) * heads * 4
    return {"bytes": nbytes + (sum(new) * case["heads"] * 4 if case["lse"] else 0), "flops": 4 * pairs * heads}


# ---------------------------------------------------------------- inputs

def _pool(case):
    """Pages of a fork's pool: what the sequences hold, and room for what the step takes, an eighth over."""
    shapes, parents = _trees(case)
    page = case["page"]
    held = sum(a // page + case["beams"] * (-(-b // page) - a // page) for a, b in shapes)
    return (held + len(parents) * (2 + case["room"] // page)) * 9 // 8 + 8


def _used(case):
    return max(1, int(case["pages"] * case["share"]))


def _codes(case, pages, g, dev):
    kv, page, dim = case["kv_heads"], case["page"], case["head_dim"]
    if case["store"] == "int8":
        return torch.randint(-127, 128, (pages, kv, page, dim), generator=g, device=dev, dtype=torch.int8)
    return torch.cat([(torch.randn(n, kv, page, dim, generator=g, device=dev, dtype=torch.float16) * 110).clamp(-448, 448).to(torch.float8_e4m3fn)
                      .view(torch.uint8) for n in [2048] * (pages // 2048) + [pages % 2048]]).view(torch.float8_e4m3fn)


def _scales(case, pages, g, dev):  # of values whose root mean square is near 1, from block to block up to a factor of 2 apart
    mid = 1 / 73.6 if case["store"] == "int8" else 1 / 110
    return torch.rand(pages, case["kv_heads"], generator=g, device=dev).mul(2).sub(1).exp2().mul(mid)


def _cache(s, case, pages, g, dev, names=("k", "v", "ks", "vs")):
    for name in names:
        s[name] = _codes(case, pages, g, dev) if len(name) == 1 else _scales(case, pages, g, dev)


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)
    s = {"case": case}
    if case["op"] == "copy":
        _cache(s, case, case["pool"], g, dev)
        s["to"] = [torch.zeros_like(s[n].view(torch.uint8)).view(s[n].dtype) for n in ("k", "v", "ks", "vs")]
        s["src"], s["dst"] = (torch.randperm(case["pool"], generator=g, device=dev)[:case["pages"]].to(torch.int32) for _ in range(2))
        return s
    if case["op"] == "sample":
        rows, vocab = case["rows"], case["vocab"]
        x = torch.randn(rows, vocab, generator=g, device=dev) * case["spread"]
        some = torch.randint(0, vocab, (rows, 24), generator=g, device=dev)  # the tokens that the context speaks for
        x.scatter_add_(1, some, torch.randn(rows, 24, generator=g, device=dev).abs() * 3 * case["spread"])
        s["x"] = x.to(TYPE[case["dtype"]])
        s["u"] = torch.rand(rows, generator=g, device=dev)
        pick = lambda *v: torch.tensor(v, device=dev)[torch.randint(0, len(v), (rows,), generator=g, device=dev)]  # noqa: E731
        s["temperature"] = s["top_k"] = s["top_p"] = s["min_p"] = None
        if case["how"] == "nucleus":
            s["temperature"], s["top_p"] = pick(0.7, 0.8, 1.0), pick(0.8, 0.9, 0.95)
        elif case["how"] == "mixed":
            s["temperature"], s["top_p"] = pick(0.0, 0.3, 0.6, 0.8, 1.0, 1.0, 1.3), pick(0.5, 0.9, 0.95, 1.0)
            s["top_k"], s["min_p"] = pick(0, 0, 1, 20, 50, 1000).to(torch.int32), pick(0.0, 0.0, 0.02, 0.1)
        return s
    if case["op"] == "fork":
        shapes, parents = _trees(case)
        page, beams, pages = case["page"], case["beams"], _pool(case)
        width = -(-(case["longest"] + case["room"]) // page)
        r = random.Random(seed)
        order = list(range(pages))
        r.shuffle(order)
        table = torch.full((len(parents), width), -1, dtype=torch.int32)
        refs, lens, at = torch.zeros(pages, dtype=torch.int32), [], 0
        for i, (prompt, whole) in enumerate(shapes):
            n, m = prompt // page, -(-whole // page)
            for j in range(beams):
                table[i * beams + j, :n] = torch.tensor(order[at:at + n], dtype=torch.int32)
            refs[order[at:at + n]] = beams
            at += n
            for j in range(beams):
                table[i * beams + j, n:m] = torch.tensor(order[at:at + m - n], dtype=torch.int32)
                refs[order[at:at + m - n]] = 1
                at += m - n
                lens.append(whole)
        s["refs"], s["table"], s["lens"] = refs.to(dev), table.to(dev), torch.tensor(lens, dtype=torch.int32, device=dev)
        s["parents"] = torch.tensor(parents, dtype=torch.int32, device=dev)
        _cache(s, case, pages, g, dev)
        return s
    if case["op"] == "compact":
        pages, used, batch = case["pages"], _used(case), case["batch"]
        order = torch.randperm(pages, generator=g, device=dev)[:used].to(torch.int32)
        each = -(-used // batch)  # pages of a sequence of its own; one of the next sequence's is shared with it
        at = torch.arange(batch, device=dev)[:, None] * each + torch.arange(each, device=dev)
        rows = torch.where(at < used, order[at.clamp(max=used - 1)], -1)
        first = torch.where(rows[:, 0] >= 0, rows[:, 0].roll(-1), -1)
        s["table"] = torch.cat([first[:, None], rows], 1)
        s["refs"] = torch.zeros(pages + 1, dtype=torch.int32, device=dev)
        s["refs"].scatter_add_(0, torch.where(s["table"] < 0, pages, s["table"]).long().reshape(-1), torch.ones(s["table"].numel(), dtype=torch.int32, device=dev))
        s["refs"] = s["refs"][:pages].clone()
        _cache(s, case, pages, g, dev)
        return s
    sizes, prefix, new, total = _groups(case)
    page, r = case["page"], random.Random(seed)
    rows, pages = [], 0
    for n, p in zip(sizes, prefix):
        common = list(range(pages, pages + p // page))  # a page that the prefix ends in is each sequence's own
        pages += len(common)
        for t in total[len(rows):len(rows) + n]:
            more = max(0, -(-t // page) - len(common))
            rows.append((common if t else []) + list(range(pages, pages + more)))
            pages += more
    order = torch.randperm(pages + 8, generator=g, device=dev).to(torch.int32)
    width = max(map(len, rows))
    flat = torch.tensor([row + [-1] * (width - len(row)) for row in rows], device=dev)
    s["table"] = torch.where(flat >= 0, order[flat.clamp(min=0)], -1)
    s["groups"] = torch.tensor([0] + sizes, device=dev).cumsum(0).to(torch.int32)
    s["shared"] = torch.tensor([p // page * page for p in prefix], device=dev, dtype=torch.int32)
    s["cu"] = torch.tensor([0] + new, device=dev).cumsum(0).to(torch.int32)
    s["lens"] = torch.tensor(total, device=dev, dtype=torch.int32)
    s["most"], s["longest"] = case["most"], max(total)
    s["rows"] = max(sum(new[a:a + n]) for a, n in zip([sum(sizes[:i]) for i in range(len(sizes))], sizes))
    s["q"] = torch.randn(sum(new), case["heads"], case["head_dim"], generator=g, device=dev, dtype=TYPE[case["dtype"]]) * 1.5
    _cache(s, case, pages + 8, g, dev)
    return s


# ---------------------------------------------------------------- one pass

def run(s):
    case = s["case"]
    if own:
        import tiled_tensor_core_tcgen05_gb300 as tg
        if case["op"] == "sample":
            return tg.sample(s["x"], s["u"], temperature=s["temperature"], top_k=s["top_k"], top_p=s["top_p"], min_p=s["min_p"])
        cache = tg.KvCache(s["k"], s["v"], s["ks"], s["vs"])
        if case["op"] == "fork":
            refs, table, lens, spare = tg.kv_fork(cache, s["refs"], s["table"], s["lens"], s["parents"], room=case["room"])
            return [refs, table, lens, spare, s["k"], s["v"], s["ks"], s["vs"]]
        if case["op"] == "compact":
            refs, table, moved, used = tg.kv_compact(cache, s["refs"], s["table"])
            return [refs, table, moved, used, s["k"], s["v"], s["ks"], s["vs"]]
        if case["op"] == "copy":
            tg.kv_copy(cache, s["src"], s["dst"], to=tg.KvCache(*s["to"]))
            return s["to"]
        return tg.attention_kv_shared(s["q"], cache, s["table"], s["lens"], s["groups"], s["shared"], s["cu"], max_new=s["most"], max_rows=s["rows"],
                                      max_len=s["longest"], return_lse=case["lse"])
    return {"sample": _draw, "fork": _branch, "compact": _gather, "copy": _hand, "attend": _attention}[case["op"]](s)


def _bytes(codes):
    return codes.view(torch.uint8)


def _hand(s):
    src, dst = s["src"].long(), s["dst"].long()
    for name, to in zip(("k", "v", "ks", "vs"), s["to"]):
        if to.dtype is torch.float32:
            to[dst] = s[name][src]
        else:
            _bytes(to)[dst] = _bytes(s[name])[src]
    return s["to"]


def _count(pages, entries, mask):
    """How many of the `entries` where `mask` is set name each page."""
    return torch.zeros(pages + 1, dtype=torch.int32, device=entries.device).scatter_add_(
        0, torch.where(mask, entries, pages).reshape(-1).long(), torch.ones(entries.numel(), dtype=torch.int32, device=entries.device))[:pages]


def _branch(s):
    case, table, lens, refs, parents = s["case"], s["table"], s["lens"], s["refs"], s["parents"]
    page, room, (batch, width), pages = case["page"], case["room"], s["table"].shape, s["refs"].numel()
    dev, n = table.device, parents.numel()
    at, i = torch.arange(width, device=dev), torch.arange(n, device=dev)
    full = lens // page
    held = (table >= 0).int().cumprod(1).sum(1)
    kept = ((at < full[:, None]) | ((refs[table.clamp(min=0).long()] == 1) & (at < held[:, None]))).int().cumprod(1).sum(1)
    # a sequence's first child takes over its open pages where no other sequence holds them
    live, p = parents >= 0, parents.clamp(min=0).long()
    first = torch.full((batch + 1,), n, device=dev).scatter_reduce_(0, torch.where(live, p, batch), i, "amin")
    heir = live & (first[p] == i)
    length = torch.where(live, lens[p], 0)
    start = torch.where(live, torch.where(heir, kept[p], full[p]), 0)
    end = torch.maximum(start, (length + room + page - 1) // page)
    new = torch.where(at < start[:, None], table[p], -1)
    source = torch.where((length % page > 0) & (start == full[p]), table[p, full[p].clamp(max=width - 1).long()], -1)
    left = refs + _count(pages, new, new >= 0) - _count(pages, table, at < held[:, None])
    free = (left == 0) & (_count(pages, source, source >= 0) == 0)
    order = torch.argsort((~free).int(), stable=True).int()
    count = end - start
    place = (count.cumsum(0) - count)[:, None] + at - start[:, None]
    wanted = (at >= start[:, None]) & (at < end[:, None])
    got = torch.where(wanted & (place < free.sum()), order[place.clamp(0, pages - 1).long()], -1)
    new = torch.where(wanted, got, new)
    spare = (free.sum() - count.sum()).to(torch.int32).view(1)
    target = new.gather(1, (length // page).clamp(max=width - 1)[:, None].long())[:, 0]
    some = (source >= 0) & (target >= 0)
    a, b = source[some].long(), target[some].long()
    here = (torch.arange(page, device=dev) < (length % page)[some][:, None])[:, None, :, None]
    for name in ("k", "v"):
        codes = _bytes(s[name])
        codes[b] = torch.where(here, codes[a], codes[b])
    for name in ("ks", "vs"):
        s[name][b] = s[name][a]
    return [left + _count(pages, got, got >= 0), new, length, spare, s["k"], s["v"], s["ks"], s["vs"]]


def _gather(s):
    refs, table, pages = s["refs"], s["table"], s["refs"].numel()
    held = refs > 0
    used = held.sum()
    at = torch.arange(pages, device=refs.device)
    holes, movers = (~held & (at < used)), held & (at >= used)
    b, a = holes.nonzero()[:, 0], movers.nonzero()[:, 0]  # the lowest page that has to move goes to the lowest hole, and so on
    moved = torch.where(held, at, -1).to(torch.int32)
    moved[a] = b.to(torch.int32)
    new = refs.clone()
    new[b], new[a] = refs[a], 0
    for name in ("k", "v"):
        _bytes(s[name])[b] = _bytes(s[name])[a]
    for name in ("ks", "vs"):
        s[name][b] = s[name][a]
    return [new, torch.where(table >= 0, moved[table.clamp(min=0).long()], -1), moved, used.to(torch.int32).view(1), s["k"], s["v"], s["ks"], s["vs"]]


def _dense(codes, scales, at, kv, dim):
    """(batch, kv, tokens, dim) in 32 bits of the pages `at` (batch, n)."""
    x = _bytes(codes)[at].view(codes.dtype).float() * scales[at][..., None, None]
    return x.transpose(1, 2).reshape(at.shape[0], kv, -1, dim)


def _attention(s):
    case = s["case"]
    kv, dim, share, most, batch = case["kv_heads"], case["head_dim"], case["heads"] // case["kv_heads"], s["most"], s["lens"].numel()
    dev = s["q"].device
    at = s["table"].long().clamp(min=0)
    new = (s["cu"][1:] - s["cu"][:-1]).long()
    rows = (s["cu"][:-1].long()[:, None] + torch.arange(most, device=dev)).clamp(max=s["q"].shape[0] - 1)
    q = s["q"].float()[rows].view(batch, most, kv, share, dim).permute(0, 2, 3, 1, 4).reshape(batch, kv, share * most, dim)
    k = _dense(s["k"], s["ks"], at, kv, dim)
    score = q @ k.transpose(-1, -2) / math.sqrt(dim)
    del k
    here = (s["lens"].long() - new)[:, None] + torch.arange(most, device=dev)
    key = torch.arange(score.shape[-1], device=dev)
    seen = (key <= here[..., None]) & (key < s["lens"][:, None, None])
    score = score.view(batch, kv, share, most, -1).masked_fill_(~seen[:, None, None], -math.inf)
    top = score.amax(-1, keepdim=True)
    p = (score - torch.where(top == -math.inf, 0.0, top)).exp_()
    total = p.sum(-1, keepdim=True)
    v = _dense(s["v"], s["vs"], at, kv, dim)
    v = v.masked_fill_((key >= s["lens"][:, None])[:, None, :, None], 0.0)
    o = (p.view(batch, kv, share * most, -1) @ v).view(batch, kv, share, most, dim) / torch.where(total == 0, 1.0, total)
    t = torch.arange(s["q"].shape[0], device=dev)
    b = torch.searchsorted(s["cu"][1:].contiguous(), t.to(torch.int32), right=True)
    j = t - s["cu"][b]
    out = o[b, :, :, j].reshape(-1, case["heads"], dim).to(s["q"].dtype)
    if not case["lse"]:
        return out
    return [out, (top + total.log())[b, :, :, j].reshape(-1, case["heads"])]


def _draw(s):
    x, rows = s["x"].double(), s["x"].shape[0]
    t = torch.ones(rows, device=x.device, dtype=torch.float64) if s["temperature"] is None else s["temperature"].double()
    greedy = t <= 0
    y = (x - x.amax(1, keepdim=True)) / torch.where(greedy, 1.0, t)[:, None]
    y, at = y.sort(dim=1, descending=True, stable=True)  # ties: the lowest index first
    rank = torch.arange(x.shape[1], device=x.device)
    keep = torch.ones_like(y, dtype=torch.bool)
    if s["top_k"] is not None:
        keep &= (rank < s["top_k"][:, None]) | (s["top_k"][:, None] <= 0)
    if s["min_p"] is not None:
        keep &= y >= s["min_p"].double().log()[:, None]
    w = y.exp() * keep
    if s["top_p"] is not None:
        total = w.cumsum(1)
        p = s["top_p"].double()[:, None]
        keep &= (total - w < p * total[:, -1:]) | (p >= 1) | (rank == 0)
        w = w * keep
    c = torch.zeros_like(w).scatter_(1, at, w).cumsum(1)
    token = torch.searchsorted(c, s["u"].double()[:, None] * c[:, -1:], right=True)[:, 0]
    return torch.where(greedy, at[:, 0], token).to(torch.int32)


# ---------------------------------------------------------------- the definitions, in 64 bits

def exact(case, seed):
    if case["op"] != "attend":
        return None  # whole numbers, and codes and scales that are moved, not computed
    s = prepare(case, seed)
    _, _, new, total = _groups(case)
    kv, dim, page, share = case["kv_heads"], case["head_dim"], case["page"], case["heads"] // case["kv_heads"]
    if sum(total) * kv * dim > 1 << 31:
        return None
    out = torch.zeros(sum(new), case["heads"], dim, dtype=torch.float64, device=s["q"].device)
    lse = torch.full((sum(new), case["heads"]), -math.inf, dtype=torch.float64, device=s["q"].device)
    done = 0
    for i, (n, t) in enumerate(zip(new, total)):
        if t:
            at = s["table"][i, :-(-t // page)].long()
            k, v = ((_bytes(c)[at].view(c.dtype).double() * f.double()[at][..., None, None]).transpose(0, 1).reshape(kv, -1, dim)[:, :t]
                    for c, f in ((s["k"], s["ks"]), (s["v"], s["vs"])))
            for r in range(n):
                see = t - n + r + 1
                q = s["q"][done + r].double().view(kv, share, dim)
                score = torch.einsum("gsd,gkd->gsk", q, k[:, :see]) / math.sqrt(dim)
                lse[done + r] = torch.logsumexp(score, -1).reshape(-1)
                out[done + r] = torch.einsum("gsk,gkd->gsd", torch.softmax(score, -1), v[:, :see]).reshape(-1, dim)
        done += n
    return [out, lse] if case["lse"] else out
