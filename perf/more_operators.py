"""What a server does to and around the paged key/value cache, as cases to measure: positions
turned into rotations of queries and keys, pages shared, copied and moved, and attention of
requests that share a long prefix.

    rotary   (a, b) -> (a cos t - b sin t, a sin t + b cos t) for pairs of channels, t = position
             times the pair's frequency; of a tensor, or of the queries and keys of new tokens
             while the keys and values enter the cache
    pages    the page tables of the next step from those of this one (requests go on, fork, end
             and begin), pages copied, moved together, states of requests copied
    attend   softmax(scale q K^T) V where the requests of a group have their first tokens in
             common

Where `own` is true, `run` calls the library; otherwise it evaluates the formulas with plain
torch operations in 32 bits (angles in 64).
"""
import math
import random

import torch

own = False

D = 128             # channels of a head
BLOCK = 32          # tokens that the cache keeps together
BASE = 10000.0      # of the rotary frequencies
TRAINED = 8192      # context that the scaled frequencies are derived from
FACTOR = 8.0        # and how far they are stretched


# ---------------------------------------------------------------- cases

def listed():
    return [
        # one token's queries: launch and latency
        {"name": "rotary one", "op": "rotary", "cached": False, "tokens": 1, "heads": 8, "channels": 128, "layout": "half",
         "scaling": "plain", "far": 4096, "dtype": "float32"},
        # the queries of a long prompt, part of each head turned
        {"name": "rotary prompt", "op": "rotary", "cached": False, "tokens": 16385, "heads": 32, "channels": 64, "layout": "pairs",
         "scaling": "linear", "far": 65536, "dtype": "bfloat16"},
        # a decode step: a new token of each request, far into its context
        {"name": "rotary cache step", "op": "rotary", "cached": True, "n": 64, "tokens": 64, "q_heads": 32, "heads": 8, "channels": 128,
         "layout": "half", "scaling": "turns", "far": 60000, "page": 64, "kind": 8},
        # prompts of unlike lengths enter the cache
        {"name": "rotary cache prompt", "op": "rotary", "cached": True, "n": 5, "tokens": 16391, "q_heads": 32, "heads": 8, "channels": 128,
         "layout": "half", "scaling": "index", "far": 300, "page": 64, "kind": 16},
        # a decode step's tables: most requests go on, some end, others begin
        {"name": "pages step", "op": "pages", "what": "step", "n": 64, "tokens": 4000, "page": 32, "heads": 1, "ragged": 1},
        # samples are drawn from each of a few prompts
        {"name": "pages fork", "op": "pages", "what": "fork", "n": 32, "rows": 256, "tokens": 3000, "page": 64, "heads": 4, "ragged": 2},
        # a cache in pieces is moved together
        {"name": "pages compact", "op": "pages", "what": "compact", "pages": 3001, "n": 40, "page": 64, "heads": 4, "ragged": 3},
        # requests move to another cache
        {"name": "pages copy", "op": "pages", "what": "copy", "pages": 1500, "n": 1200, "page": 64, "heads": 4, "ragged": 4},
        # the recurrent layers' states of requests that fork
        {"name": "pages slots", "op": "pages", "what": "slots", "n": 40, "heads": 48, "ragged": 5},
        # two samples of one short prompt
        {"name": "attend pair", "op": "attend", "groups": 1, "members": 2, "prefix": 300, "tail": 40, "new": 1, "q_heads": 8, "heads": 2,
         "page": 32, "kind": 16, "ragged": 0},
        # a batch behind one long instruction, 8-bit
        {"name": "attend samples", "op": "attend", "groups": 1, "members": 64, "prefix": 16384, "tail": 700, "new": 1, "q_heads": 32,
         "heads": 8, "page": 64, "kind": 8, "ragged": 6},
        # several conversations' requests bring a question each
        {"name": "attend tails", "op": "attend", "groups": 4, "members": 8, "prefix": 4100, "tail": 200, "new": 100, "q_heads": 32,
         "heads": 8, "page": 64, "kind": 16, "ragged": 7},
    ]


def _between(rng, lo, hi):
    """An integer whose logarithm is spread evenly over [lo, hi]."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("rotary", "rotary", "pages", "pages", "pages", "attend", "attend", "attend"))
    if op == "rotary":
        turn = {"op": op, "channels": 16 * rng.randrange(1, 9), "layout": rng.choice(("half", "pairs")),
                "scaling": rng.choice(("plain", "linear", "turns", "index")), "far": _between(rng, 16, 65536)}
        if rng.random() < 0.4:
            return {**turn, "cached": False, "tokens": _between(rng, 1, 16384), "heads": rng.randrange(1, 33),
                    "dtype": rng.choice(("float32", "bfloat16"))}
        tokens, heads = _between(rng, 1, 16384), rng.choice((1, 2, 3, 4, 8))
        return {**turn, "cached": True, "n": _between(rng, 1, min(tokens, 64)), "tokens": tokens, "q_heads": heads * rng.choice((1, 2, 3, 4)),
                "heads": heads, "page": rng.choice((32, 64, 128, 256)), "kind": rng.choice((8, 16))}
    if op == "pages":
        what = rng.choice(("step", "fork", "compact", "copy", "slots"))
        page, heads = rng.choice((32, 64, 128)), rng.randrange(1, 5)
        most = (384 << 20) // (page * heads * 512)  # pages of 384 MiB
        ragged = rng.randrange(1, 1000)
        if what == "slots":
            return {"op": op, "what": what, "n": _between(rng, 1, 40), "heads": rng.randrange(1, 49), "ragged": ragged}
        if what in ("compact", "copy"):
            pages = _between(rng, 8, most)
            return {"op": op, "what": what, "pages": pages, "n": _between(rng, 1, min(pages // 2, 1200)), "page": page, "heads": heads, "ragged": ragged}
        n = _between(rng, 1, 64)
        tokens = _between(rng, 1, min(4000, most * page // (2 * n + 8)))
        case = {"op": op, "what": what, "n": n, "tokens": tokens, "page": page, "heads": heads, "ragged": ragged}
        return case if what == "step" else {**case, "rows": _between(rng, n, 256)}
    heads = rng.choice((1, 2, 4, 8))
    group = rng.choice((1, 2, 3, 4, 7, 8))
    groups, members = _between(rng, 1, 8), _between(rng, 1, 64)
    members = min(members, max(1, 96 // groups))
    new = 1 if rng.random() < 0.6 else _between(rng, 2, max(2, min(128, 2048 // (groups * members))))
    tail = _between(rng, new, 1000)
    most = 130 * 10 ** 9 // (groups * members * new * heads * group * 4 * D) - tail  # 130 GFLOP
    return {"op": op, "groups": groups, "members": members, "prefix": _between(rng, 1, max(1, min(16384, most))), "tail": tail,
            "new": new, "q_heads": heads * group, "heads": heads, "page": rng.choice((32, 64, 128, 256)), "kind": rng.choice((8, 16)),
            "ragged": rng.randrange(0, 1000)}


def _rows(case):
    """(new tokens, tokens in the cache with the new ones among them) of each request that turns and writes its tokens."""
    n, t, r = case["n"], case["tokens"], random.Random(case["tokens"])
    new = [t // n + (i < t % n) for i in range(n)]
    if t > 4 * n:  # unlike lengths
        for i in range(0, n - 1, 2):
            d = r.randrange(0, new[i] // 2 + 1)
            new[i], new[i + 1] = new[i] - d, new[i + 1] + d
    return [(m, m + r.randrange(0, case["far"])) for m in new]


def _tails(case):
    """(new tokens, tokens behind the prefix with the new ones among them) of each request."""
    r = random.Random(case["ragged"])
    got = []
    for _ in range(case["groups"] * case["members"]):
        new, tail = case["new"], case["tail"]
        if case["ragged"] and got:
            new = r.randrange(max(1, new // 2), new + 1)
            tail = r.randrange(max(new, tail // 2), tail + 1)
        got.append((new, tail))
    return got


def _prefixes(case):
    r = random.Random(case["ragged"] + 1)
    return [case["prefix"] if not case["ragged"] or not i else r.randrange((case["prefix"] + 1) // 2, case["prefix"] + 1)
            for i in range(case["groups"])]


def _code(case):
    """Bytes of a token's key or value of one head."""
    return D * case["kind"] // 8 + (4 if case["kind"] == 8 else 0)


def work(case):
    op = case["op"]
    if op == "rotary":
        t = case["tokens"]
        if not case["cached"]:
            return {"bytes": t * (case["heads"] * D * 2 * (4 if case["dtype"] == "float32" else 2) + 4), "flops": t * case["heads"] * case["channels"] * 3}
        h = case["heads"] * 2  # written, and read back
        return {"bytes": t * (case["q_heads"] * D * 4 + h * (2 * D * 2 + 2 * _code(case))), "flops": t * (case["q_heads"] + case["heads"]) * case["channels"] * 3}
    if op == "pages":
        what = case["what"]
        if what == "slots":
            return {"bytes": case["n"] * case["heads"] * D * D * 4 * 2, "flops": 0}
        page = case["page"] * case["heads"] * 512
        if what == "copy":
            return {"bytes": case["n"] * page * 2, "flops": 0}
        b = _book(case)
        if what == "compact":
            live = sum(x != 0 for x in b["refs"])
            return {"bytes": sum(x != 0 for x in b["refs"][live:]) * page * 2 + len(b["refs"]) * 12 + sum(len(r) for r in b["rows"]) * 8, "flops": 0}
        after = _assign_by_hand(case, b)
        blocks = sum(x[2] for x in after["copies"]) * case["heads"] * BLOCK * 512
        entries = sum(len(r) for r in b["rows"]) + sum(x >= 0 for r in after["pages"] for x in r)
        return {"bytes": blocks * 2 + entries * 4 + len(b["refs"]) * 8, "flops": 0}
    tails, prefixes, m = _tails(case), _prefixes(case), case["members"]
    seen = sum(new * (prefixes[i // m] + tail - new) + new * (new + 1) // 2 for i, (new, tail) in enumerate(tails))
    return {"bytes": (sum(prefixes) + sum(t for _, t in tails)) * case["heads"] * 2 * _code(case) + sum(a for a, _ in tails) * case["q_heads"] * 2 * D * 2,
            "flops": seen * case["q_heads"] * 4 * D}


# ---------------------------------------------------------------- page tables on the host

def _book(case):
    """Page tables, contexts and reference counts of a cache in use; for a step also what the
    rows of the next one continue and how many tokens each brings."""
    r = random.Random(case["ragged"])
    page, n = case.get("page"), case["n"]
    if case["what"] == "compact":
        total = case["pages"]
        held = r.sample(range(total), max(1, total // 2))
        refs, rows, at = [0] * total, [], 0
        for b in range(n):
            take = held[at:at + max(1, len(held) // n)]
            at += len(take)
            # every row also holds the first row's first pages
            rows.append((rows[0][:2] if rows else []) + take)
            for p in rows[-1]:
                refs[p] += 1
        for p in held[at:]:  # held by the program itself
            refs[p] += 1
        return {"refs": refs, "rows": rows}
    context = [max(1, case["tokens"] - (r.randrange(0, case["tokens"] // 2 + 1) if b else 0)) for b in range(n)]
    if case["what"] == "step":
        parent, add = list(range(n)), [1] * n
        for j in range(n):
            if r.random() < 1 / 16:  # one has ended, and another takes its place
                parent[j], add[j] = -1, r.randrange(1, case["tokens"] + 1)
    else:
        parent = sorted(r.randrange(n) for _ in range(case["rows"]))
        add = [r.choice((0, 1, 1, 1, 5)) for _ in parent]
    common = min(context) // 4 // page
    need = [-(-c // page) for c in context]
    ahead = sum(-(-a // page) + 1 for a in add)
    total = sum(need) + ahead + 5
    order = list(range(total))
    r.shuffle(order)
    refs, rows = [0] * total, []
    for b in range(n):
        row = (rows[0][:common] if b else []) + [order.pop() for _ in range(need[b] - (common if b else 0))]
        rows.append(row)
        for p in row:
            refs[p] += 1
    return {"refs": refs, "rows": rows, "context": context, "parent": parent, "add": add,
            "width": -(-max(max(context), max((context[a] if a >= 0 else 0) + x for a, x in zip(parent, add))) // page) + 1}


def _assign_by_hand(case, b):
    """The next step's tables, one row after the other."""
    page, hold, full = case["page"], list(b["refs"]), []
    for row in b["rows"]:
        for p in row:
            hold[p] -= 1
    for a in b["parent"]:
        kept = b["context"][a] if a >= 0 else 0
        full.append(kept // page)
        for p in (b["rows"][a] if a >= 0 else [])[:kept // page]:
            hold[p] += 1
    free = iter([p for p, x in enumerate(b["refs"]) if x == 0])
    refs, taken, pages, context, copies = list(hold), set(), [], [], []
    for a, x, f in zip(b["parent"], b["add"], full):
        old = b["rows"][a] if a >= 0 else []
        kept = b["context"][a] if a >= 0 else 0
        row = old[:f]
        if kept % page:
            last = old[f]
            if hold[last] == 0 and last not in taken:  # nobody else has it
                taken.add(last)
                row = row + [last]
                refs[last] = 1
            else:
                row = row + [next(free)]
                refs[row[-1]] = 1
                copies.append((last, row[-1], -(-(kept % page) // BLOCK)))
        while len(row) < -(-(kept + x) // page):
            row = row + [next(free)]
            refs[row[-1]] = 1
        pages.append(row + [-1] * (b["width"] - len(row)))
        context.append(kept + x)
    return {"pages": pages, "context": context, "refs": refs, "copies": copies}


# ---------------------------------------------------------------- inputs

def _normal(g, *shape):
    return torch.randn(shape, generator=g, device="cuda")


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _counts(lens):
    return torch.tensor([0] + list(lens), device="cuda").cumsum(0).to(torch.int32)


def _vectors(g, t, h):
    """Keys and values with unlike tokens and a few strong channels."""
    x = _normal(g, t, h, D) * torch.exp2(2 * torch.rand((t, h, 1), generator=g, device="cuda"))
    x[:, :, ::37] *= 3
    return x.to(torch.bfloat16)


def _inputs(case, seed):
    """Inputs of a case, made from the seed alone."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    op, bf16 = case["op"], torch.bfloat16
    if op == "rotary":
        t, h = case["tokens"], case["heads"]
        if not case["cached"]:
            dt = getattr(torch, case["dtype"])
            return {"x": _normal(g, t, h, D).to(dt), "y": torch.empty((t, h, D), dtype=dt, device="cuda"),
                    "positions": torch.randint(0, case["far"], (t,), generator=g, device="cuda").to(torch.int32)}
        # the rows of one projection: queries, keys and values of a token together
        both, hq, page = _rows(case), case["q_heads"], case["page"]
        qkv = torch.cat([_normal(g, t, hq, D).to(bf16), _vectors(g, t, h), _vectors(g, t, h)], 1)
        # only the pages that the new tokens go to are there
        width = max(-(-c // page) for _, c in both)
        spans = [((c - m) // page, -(-c // page)) for m, c in both]
        pages = sum(b - a for a, b in spans) + 3
        order, at = torch.randperm(pages, generator=g, device="cuda").to(torch.int32), 0
        table = torch.full((case["n"], width), -1, dtype=torch.int32, device="cuda")
        for i, (a, b) in enumerate(spans):
            table[i, a:b] = order[at:at + b - a]
            at += b - a
        return {"both": both, "pages": pages, "table": table, "cu": _counts(m for m, _ in both), "context": _i32([c for _, c in both]),
                "q": qkv[:, :hq], "k": qkv[:, hq:hq + h], "v": qkv[:, hq + h:],
                "q_out": torch.empty((t, hq, D), dtype=bf16, device="cuda"),
                "k_out": torch.empty((t, h, D), dtype=bf16, device="cuda"), "v_out": torch.empty((t, h, D), dtype=bf16, device="cuda")}
    if op == "pages":
        what, n = case["what"], case["n"]
        r = random.Random(case["ragged"] * 1000003 + seed)
        if what == "slots":
            pick = r.sample(range(2 * n), 2 * n)
            return {"memory": _normal(g, 2 * n, case["heads"], D * D), "src": _i32(pick[:n]), "dst": _i32(pick[n:])}
        shape = (case["heads"], case["page"] // BLOCK, BLOCK * 2 * D)
        if what == "copy":
            src, dst = r.sample(range(case["pages"]), n), r.sample(range(case["pages"]), n)
            return {"memory": _normal(g, case["pages"], *shape).to(bf16), "to": torch.zeros((case["pages"], *shape), dtype=bf16, device="cuda"),
                    "src": _i32(src), "dst": _i32(dst)}
        b = _book(case)
        total = len(b["refs"])
        width = b["width"] if "width" in b else max(map(len, b["rows"]))
        # the same tables over other pages
        other = r.sample(range(total), total)
        b["rows"] = [[other[p] for p in row] for row in b["rows"]]
        refs = [0] * total
        for p, x in enumerate(b["refs"]):
            refs[other[p]] = x
        b["refs"] = refs
        s = {"book": b, "memory": _normal(g, total, *shape).to(bf16), "refs": _i32(refs), "new_refs": torch.empty(total, dtype=torch.int32, device="cuda"),
             "pages": _i32([row + [-1] * (width - len(row)) for row in b["rows"]])}
        if what == "compact":
            return {**s, "moved": torch.empty_like(s["refs"]), "new_pages": torch.empty_like(s["pages"])}
        return {**s, "context": _i32(b["context"]), "parent": _i32(b["parent"]), "add": _i32(b["add"]),
                "new_context": torch.empty(len(b["parent"]), dtype=torch.int32, device="cuda"),
                "new_pages": torch.empty((len(b["parent"]), width), dtype=torch.int32, device="cuda")}
    page, h, m = case["page"], case["heads"], case["members"]
    tails, prefixes = _tails(case), _prefixes(case)
    whole = [p // page * page for p in prefixes]  # the tokens whose pages are shared
    contexts = [prefixes[i // m] + tail for i, (_, tail) in enumerate(tails)]
    width = max(-(-c // page) for c in contexts)
    need = [x // page for x in whole] + [-(-c // page) - whole[i // m] // page for i, c in enumerate(contexts)]
    pages = sum(need) + 3
    order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    table, at = torch.full((len(tails), width), -1, dtype=torch.int32, device="cuda"), 0
    for i, x in enumerate(whole):
        table[i * m:(i + 1) * m, :x // page] = order[at:at + x // page]
        at += x // page
    for i, x in enumerate(need[case["groups"]:]):
        table[i, whole[i // m] // page:whole[i // m] // page + x] = order[at:at + x]
        at += x
    t = sum(new for new, _ in tails)
    return {"tails": tails, "prefixes": prefixes, "whole": whole, "pages": pages, "table": table, "context": _i32(contexts),
            "cu": _counts(new for new, _ in tails), "group_cu": _i32([i * m for i in range(case["groups"] + 1)]), "shared": _i32(prefixes),
            # keys and values: of the prefixes, then of each request's own tokens
            "prefix": [_vectors(g, sum(prefixes), h) for _ in range(2)], "tail": [_vectors(g, sum(x for _, x in tails), h) for _ in range(2)],
            "q": _normal(g, t, case["q_heads"], D).to(bf16), "o": torch.empty((t, case["q_heads"], D), dtype=bf16, device="cuda"),
            "scale": 1 / math.sqrt(D)}


def _frequencies(case):
    """Angle of each pair of channels from one position to the next, and what the rotated values are multiplied by."""
    c, rule = case["channels"], case["scaling"]
    i = torch.arange(c // 2, dtype=torch.float64, device="cuda")
    f = torch.exp(-2 * i / c * math.log(BASE))
    if rule == "linear":
        return f / FACTOR, 1.0
    if rule == "turns":  # fast pairs as they are, slow ones stretched
        keep = ((TRAINED * f / (2 * math.pi) - 1) / (4 - 1)).clamp(0, 1)
        return f * (keep + (1 - keep) / FACTOR), 1.0
    if rule == "index":
        lo, hi = (c * math.log(TRAINED / (2 * math.pi * x)) / (2 * math.log(BASE)) for x in (32, 1))
        lo, hi = max(math.floor(lo), 0), min(math.ceil(hi), c - 1)
        keep = 1 - ((i - lo) / max(hi - lo, 0.001)).clamp(0, 1)
        return f * (keep + (1 - keep) / FACTOR), 0.1 * math.log(FACTOR) + 1
    return f, 1.0


def prepare(case, seed):
    s = _inputs(case, seed)
    s["case"] = case
    op = case["op"]
    if own:
        from quantized_delta_rule_decode_amd import qdr
    if op == "rotary":
        if own:
            rules = {"plain": qdr.ROTARY_PLAIN, "linear": qdr.ROTARY_LINEAR, "turns": qdr.ROTARY_TURNS, "index": qdr.ROTARY_INDEX}
            freq, amplitude = qdr.qdr_rotary_frequencies(rules[case["scaling"]], case["channels"], BASE, factor=FACTOR, context=TRAINED, low=1.0,
                                                         high=32.0 if case["scaling"] == "index" else 4.0)
            s["rotary"] = qdr.Rotary(freq, qdr.ROTARY_HALF if case["layout"] == "half" else qdr.ROTARY_PAIRS, amplitude)
            if case["cached"]:
                s["cache"] = qdr.KVCache(s["pages"], case["page"], case["heads"], case["kind"])
        else:
            s["freq"], s["amplitude"] = _frequencies(case)
            if case["cached"]:
                _empty_store(s)
        return s
    if op == "pages":
        if own and case["what"] == "slots":
            memory = torch.empty_like(s["memory"])
            s["pool"] = qdr.Pool(2 * case["n"], case["heads"], [qdr.K_FP32] * case["heads"], None, scale_mode=qdr.SCALE_ROW_ABSMAX, dev_mem=memory)
            s["memory"] = memory.copy_(s["memory"])
        elif own:
            for name, x in [("cache", "memory")] + ([("other", "to")] if case["what"] == "copy" else []):
                memory = torch.empty_like(s[x])
                s[name] = qdr.KVCache(memory.shape[0], case["page"], case["heads"], qdr.KV_BF16, dev_mem=memory)
                s[x] = memory.copy_(s[x])
            if case["what"] == "compact":
                s["workspace"] = torch.empty(s["cache"].qdr_kv_compact_workspace(), dtype=torch.uint8, device="cuda")
            elif case["what"] != "copy":
                s["workspace"] = torch.empty(s["cache"].qdr_kv_assign_workspace(s["parent"].shape[0]), dtype=torch.uint8, device="cuda")
        return s
    if own:
        s["cache"] = qdr.KVCache(s["pages"], case["page"], case["heads"], case["kind"])
        k, v, cu, context, first = _cached(s)
        s["cache"].qdr_kv_write(s["table"][first].contiguous(), cu, context, k, v)
        s["workspace"] = torch.empty(s["cache"].qdr_kv_attend_shared_workspace(len(s["tails"]), s["q"].shape[0], case["groups"], case["q_heads"], s["table"].shape[1]),
                                     dtype=torch.uint8, device="cuda")
    else:
        _empty_store(s)
        k, v, cu, context, first = _cached(s)
        _store(s, _places(case, s["table"][first], cu, context, k.shape[0]), k, v)
    for x in ("prefix", "tail"):
        del s[x]
    return s


def _cached(s):
    """Keys and values as they enter the cache: the shared pages' once, and each request's from
    there on; with their counts, contexts and rows of the table."""
    m, parts, lens, contexts, first = s["case"]["members"], [[], []], [], [], []
    at = 0
    for i, (p, w) in enumerate(zip(s["prefixes"], s["whole"])):
        for x in range(2):
            parts[x].append(s["prefix"][x][at:at + w])
        at += p
        lens.append(w)
        contexts.append(w)
        first.append(i * m)
    starts = [sum(s["prefixes"][:i]) for i in range(len(s["prefixes"]))]
    at = 0
    for i, (_, tail) in enumerate(s["tails"]):
        g = i // m
        for x in range(2):
            parts[x] += [s["prefix"][x][starts[g] + s["whole"][g]:starts[g] + s["prefixes"][g]], s["tail"][x][at:at + tail]]
        at += tail
        contexts.append(s["prefixes"][g] + tail)
        lens.append(contexts[-1] - s["whole"][g])
        first.append(i)
    return torch.cat(parts[0]), torch.cat(parts[1]), _counts(lens), _i32(contexts), torch.tensor(first, device="cuda")


# ---------------------------------------------------------------- one pass

def run(state):
    case = state["case"]
    op = case["op"]
    if op == "rotary":
        if not case["cached"]:
            if own:
                turn = state["rotary"].qdr_rotate if case["dtype"] == "float32" else state["rotary"].qdr_rotate_bf16
                turn(state["positions"], state["x"], state["y"])
                return {"y": state["y"]}
            return {"y": _turned(state, state["x"], state["positions"]).to(state["x"].dtype)}
        if own:
            state["cache"].qdr_kv_write_rotary(state["rotary"], state["table"], state["cu"], state["context"], state["k"], state["v"],
                                               q=state["q"], q_out=state["q_out"])
            state["cache"].qdr_kv_read(state["table"], state["cu"], state["context"], state["k_out"], state["v_out"])
            return {"q": state["q_out"], "k": state["k_out"], "v": state["v_out"]}
        return _plain_write(state)
    if op == "pages":
        what = case["what"]
        if what == "slots":
            if own:
                state["pool"].qdr_slot_copy(state["src"], state["dst"])
            else:
                state["memory"][state["dst"].long()] = state["memory"][state["src"].long()]
            return {"memory": state["memory"]}
        if what == "copy":
            if own:
                state["cache"].qdr_kv_copy(state["src"], state["dst"], to=state["other"])
            else:
                state["to"][state["dst"].long()] = state["memory"][state["src"].long()]
            return {"memory": state["to"]}
        if what == "compact":
            if own:
                state["cache"].qdr_kv_compact(state["refs"], state["pages"], state["moved"], state["new_refs"], state["new_pages"],
                                              workspace=state["workspace"])
                return {x: state[x] for x in ("moved", "new_refs", "new_pages", "memory")}
            return _plain_compact(state)
        if own:
            state["cache"].qdr_kv_assign(state["pages"], state["context"], state["parent"], state["add"], state["refs"], state["new_pages"],
                                         state["new_context"], state["new_refs"], workspace=state["workspace"])
            return {x: state[x] for x in ("new_pages", "new_context", "new_refs", "memory")}
        return _plain_assign(state)
    if own:
        state["cache"].qdr_kv_attend_shared(state["table"], state["cu"], state["context"], state["group_cu"], state["shared"], state["q"],
                                            state["o"], scale=state["scale"], workspace=state["workspace"])
        return {"o": state["o"]}
    return _plain_attend(state)


# ---------------------------------------------------------------- plain forms

def _turned(s, x, positions):
    """x in 32 bits with its first channels turned."""
    c, layout = s["case"]["channels"], s["case"]["layout"]
    angle = positions.double()[:, None] * s["freq"]
    cos, sin = ((f * s["amplitude"]).float()[:, None] for f in (angle.cos(), angle.sin()))
    y = x.float().clone()
    z = y[..., :c].clone()
    if layout == "half":
        a, b = z[..., :c // 2], z[..., c // 2:]
        y[..., :c // 2], y[..., c // 2:c] = a * cos - b * sin, a * sin + b * cos
    else:
        a, b = z[..., 0::2], z[..., 1::2]
        y[..., 0:c:2], y[..., 1:c:2] = a * cos - b * sin, a * sin + b * cos
    return y


def _empty_store(s):
    case = s["case"]
    shape = (s["pages"] * case["page"], case["heads"])
    if case["kind"] == 8:
        s["codes"] = [torch.zeros(shape + (D,), dtype=torch.int8, device="cuda") for _ in range(2)]
        s["scales"] = [torch.zeros(shape, device="cuda") for _ in range(2)]
    else:
        s["values"] = [torch.zeros(shape + (D,), dtype=torch.bfloat16, device="cuda") for _ in range(2)]


def _positions(cu, context, tokens):
    """Request and position of every token that `cu` counts."""
    cu, token = cu.long(), torch.arange(tokens, device="cuda")
    row = torch.searchsorted(cu[1:].contiguous(), token, right=True)
    return row, context.long()[row] - cu[row + 1] + token


def _places(case, table, cu, context, tokens):
    """Where those tokens are in the cache."""
    row, pos = _positions(cu, context, tokens)
    return table.long()[row, pos // case["page"]] * case["page"] + pos % case["page"]


def _store(s, at, k, v):
    for i, x in enumerate((k, v)):
        if s["case"]["kind"] == 16:
            s["values"][i][at] = x.to(torch.bfloat16)
            continue
        x = x.float()
        most = x.abs().amax(-1)
        most = torch.where(most < 2.0 ** -126, 1.0, most)
        s["scales"][i][at] = most / 127
        s["codes"][i][at] = torch.round(x * 127 / most[..., None]).to(torch.int8)


def _load(s, at):
    if s["case"]["kind"] == 16:
        return [x[at].float() for x in s["values"]]
    return [c[at].float() * f[at][..., None] for c, f in zip(s["codes"], s["scales"])]


def _plain_write(s):
    t = s["q"].shape[0]
    _, pos = _positions(s["cu"], s["context"], t)
    at = _places(s["case"], s["table"], s["cu"], s["context"], t)
    _store(s, at, _turned(s, s["k"], pos), s["v"])
    k, v = _load(s, at)
    return {"q": _turned(s, s["q"], pos).to(torch.bfloat16), "k": k.to(torch.bfloat16), "v": v.to(torch.bfloat16)}


def _plain_assign(s):
    page, total = s["case"]["page"], s["refs"].shape[0]
    pages, context, parent, refs = (s[x].long() for x in ("pages", "context", "parent", "refs"))
    rows, width = parent.shape[0], pages.shape[1]
    col, j = torch.arange(width, device="cuda"), torch.arange(rows, device="cuda")
    one = torch.ones((), dtype=torch.int64, device="cuda")
    kept = torch.where(parent >= 0, context[parent.clamp_min(0)], 0)
    after = kept + s["add"].long()
    full, part, most = kept // page, kept % page, -(-after // page)
    old = pages[parent.clamp_min(0)]
    # who holds a page besides the rows that only begin to fill it (one place more takes what has no page)
    hold = torch.cat([refs, one[None] * 0])
    hold.scatter_add_(0, torch.where(col < -(-context // page)[:, None], pages, total).flatten(), (-one).expand(pages.numel()))
    hold.scatter_add_(0, torch.where(col < full[:, None], old, total).flatten(), one.expand(old.numel()))
    last = torch.where(part > 0, old.gather(1, full.clamp_max(width - 1)[:, None])[:, 0], total)
    first = torch.full((total + 1,), rows, device="cuda").scatter_reduce_(0, last, j, "amin")
    stays = (part > 0) & (hold[last] == 0) & (first[last] == j)
    begin = full + stays.long()
    need = most - begin
    free = torch.argsort((refs != 0).long(), stable=True)
    take = free[((need.cumsum(0) - need - begin)[:, None] + col).clamp(0, total - 1)]
    new = torch.where(col < begin[:, None], old, torch.where(col < most[:, None], take, -1))
    fresh = (col >= full[:, None]) & (col < most[:, None])
    hold[torch.where(fresh, new, total).flatten()] = 1
    copy = ((part > 0) & ~stays).nonzero()[:, 0]
    src, dst = last[copy], new[copy, full[copy]]
    block = torch.arange(page // BLOCK, device="cuda") < (-(-part[copy] // BLOCK))[:, None]
    s["memory"][dst] = torch.where(block[:, None, :, None], s["memory"][src], s["memory"][dst])
    return {"new_pages": new.to(torch.int32), "new_context": after.to(torch.int32), "new_refs": hold[:total].to(torch.int32), "memory": s["memory"]}


def _plain_compact(s):
    refs, pages = s["refs"].long(), s["pages"].long()
    total = refs.shape[0]
    p = torch.arange(total, device="cuda")
    live = refs != 0
    count = live.sum()
    free = torch.argsort(live.long(), stable=True)
    behind = live & (p >= count)
    moved = torch.where(live, torch.where(behind, free[(behind.long().cumsum(0) - 1).clamp_min(0)], p), -1)
    src = behind.nonzero()[:, 0]
    s["memory"][moved[src]] = s["memory"][src]
    new_refs = torch.zeros(total + 1, dtype=torch.int64, device="cuda").scatter_(0, torch.where(live, moved, total), refs)
    new_pages = torch.where(pages >= 0, moved[pages.clamp_min(0)], -1)
    return {"moved": moved.to(torch.int32), "new_refs": new_refs[:total].to(torch.int32), "new_pages": new_pages.to(torch.int32), "memory": s["memory"]}


def _plain_attend(s):
    """Scores of a group's rows and its prefix as one product, each request's own tokens padded."""
    case, page, m, h = s["case"], s["case"]["page"], s["case"]["members"], s["case"]["heads"]
    group, context = case["q_heads"] // case["heads"], s["context"].long()
    new = s["cu"].diff().long()
    out, at = torch.empty_like(s["o"]), 0
    for i, p in enumerate(s["prefixes"]):
        here = s["tails"][i * m:(i + 1) * m]
        most, tail, t = max(a for a, _ in here), max(b for _, b in here), sum(a for a, _ in here)
        table, rows = s["table"][i * m:(i + 1) * m].long(), torch.arange(most, device="cuda")
        inside = rows < new[i * m:(i + 1) * m, None]
        q = s["q"].float()[torch.where(inside, s["cu"][i * m:(i + 1) * m].long()[:, None] + rows, 0)]
        q = q.view(m, most, h, group, D).permute(2, 0, 3, 1, 4)  # [head][request][query head of it][row]
        key = torch.arange(p, device="cuda")
        pk, pv = (x.transpose(0, 1) for x in _load(s, table[0, key // page] * page + key % page))
        key = p + torch.arange(tail, device="cuda")
        where = table.gather(1, (key // page).clamp_max(table.shape[1] - 1)[None].expand(m, -1)).clamp_min(0) * page + key % page
        tk, tv = (x.permute(2, 0, 1, 3) for x in _load(s, where))
        ends = context[i * m:(i + 1) * m]
        tv = torch.where((key < ends[:, None])[None, :, :, None], tv, 0)
        flat = q.reshape(h, m * group * most, D)
        sp = (flat @ pk.transpose(-1, -2)).view(h, m, group * most, p) * s["scale"]
        st = (q.reshape(h, m, group * most, D) @ tk.transpose(-1, -2)).view(h, m, group, most, tail) * s["scale"]
        seen = key <= (ends - new[i * m:(i + 1) * m])[:, None, None] + rows[:, None]
        st = st.masked_fill(~seen[None, :, None], -math.inf).view(h, m, group * most, tail)
        top = torch.maximum(sp.amax(-1, keepdim=True), st.amax(-1, keepdim=True))
        sp, st = (sp - top).exp_(), (st - top).exp_()
        o = (sp.view(h, m * group * most, p) @ pv).view(h, m, group * most, D) + st @ tv
        o = o / (sp.sum(-1, keepdim=True) + st.sum(-1, keepdim=True))
        o = o.view(h, m, group, most, D).permute(1, 3, 0, 2, 4).reshape(m, most, case["q_heads"], D)
        out[at:at + t] = o[inside].to(torch.bfloat16)
        at += t
    return {"o": out}


# ---------------------------------------------------------------- in 64 bits

def exact(case, seed):
    s = _inputs(case, seed)
    op = case["op"]

    def held(x):
        if case["kind"] == 16:
            return x
        most = x.abs().amax(-1, keepdim=True)
        most = torch.where(most < 2.0 ** -126, torch.ones_like(most), most)
        return torch.round(x * 127 / most) * most / 127

    if op == "rotary":
        c = case["channels"]
        freq, amplitude = [], 1.0
        for i in range(c // 2):
            f, keep = BASE ** (-2.0 * i / c), 1.0
            if case["scaling"] == "linear":
                keep = 0.0
            elif case["scaling"] == "turns":
                keep = min(max((f * TRAINED / math.tau - 1.0) / 3.0, 0.0), 1.0)
            elif case["scaling"] == "index":
                lo, hi = [0.5 * c * math.log(TRAINED / math.tau / x, BASE) for x in (32.0, 1.0)]
                lo, hi = max(int(math.floor(lo)), 0), min(int(math.ceil(hi)), c - 1)
                keep, amplitude = 1.0 - min(max((i - lo) / max(hi - lo, 0.001), 0.0), 1.0), 1.0 + 0.1 * math.log(FACTOR)
            freq.append(f * keep + f / FACTOR * (1.0 - keep))
        freq = torch.tensor(freq, dtype=torch.float64, device="cuda")

        def turned(x, pos):
            z, half = x.double(), case["layout"] == "half"
            i = torch.arange(c, device="cuda")
            pair, second = (i % (c // 2), i >= c // 2) if half else (i // 2, i % 2 == 1)
            other = torch.where(second, i - (c // 2 if half else 1), i + (c // 2 if half else 1))
            angle = pos.double()[:, None] * freq[pair]
            y = z[..., :c] * (amplitude * angle.cos())[:, None] + z[..., other] * (amplitude * torch.where(second, 1.0, -1.0) * angle.sin())[:, None]
            return torch.cat([y, z[..., c:]], -1)

        if not case["cached"]:
            return {"y": turned(s["x"], s["positions"])}
        pos = torch.cat([torch.arange(b - a, b, device="cuda") for a, b in s["both"]])
        return {"q": turned(s["q"], pos), "k": held(turned(s["k"], pos)), "v": held(s["v"].double())}

    if op == "pages":
        what = case["what"]
        if what in ("slots", "copy"):
            to = s["memory"] if what == "slots" else s["to"]
            for a, b in zip(s["src"].tolist(), s["dst"].tolist()):
                to[b] = s["memory"][a]
            return {"memory": to.double()}
        book = s["book"]
        if what == "compact":
            live = [p for p, x in enumerate(book["refs"]) if x]
            room = iter([p for p, x in enumerate(book["refs"]) if not x])
            moved, refs = [-1] * len(book["refs"]), [0] * len(book["refs"])
            for p in live:
                moved[p] = p if p < len(live) else next(room)
                refs[moved[p]] = book["refs"][p]
                if moved[p] != p:
                    s["memory"][moved[p]] = s["memory"][p]
            width = s["pages"].shape[1]
            pages = [[moved[p] for p in row] + [-1] * (width - len(row)) for row in book["rows"]]
            return {"moved": _i32(moved), "new_refs": _i32(refs), "new_pages": _i32(pages), "memory": s["memory"].double()}
        after = _assign_by_hand(case, book)
        for a, b, blocks in after["copies"]:
            s["memory"][b, :, :blocks] = s["memory"][a, :, :blocks]
        return {"new_pages": _i32(after["pages"]), "new_context": _i32(after["context"]), "new_refs": _i32(after["refs"]), "memory": s["memory"].double()}

    out, m, group = [], case["members"], case["q_heads"] // case["heads"]
    (pk, pv), (tk, tv) = ([held(x.double()) for x in s[part]] for part in ("prefix", "tail"))
    at, first = 0, 0
    for i, (new, tail) in enumerate(s["tails"]):
        g = i // m
        a = sum(s["prefixes"][:g])
        k = torch.cat([pk[a:a + s["prefixes"][g]], tk[at:at + tail]])
        v = torch.cat([pv[a:a + s["prefixes"][g]], tv[at:at + tail]])
        q = s["q"][first:first + new].double().view(new, case["heads"], group, D)
        last = torch.arange(k.shape[0] - new, k.shape[0], device="cuda")
        hidden = torch.arange(k.shape[0], device="cuda")[None, :] > last[:, None]
        heads = []
        for x in range(case["heads"]):
            sc = q[:, x].reshape(new * group, D) @ k[:, x].t().contiguous() * s["scale"]
            sc = sc.view(new, group, -1).masked_fill_(hidden[:, None], -math.inf)
            heads.append((torch.softmax(sc, -1).view(new * group, -1) @ v[:, x].contiguous()).view(new, group, D))
        out.append(torch.cat(heads, 1))
        at, first = at + tail, first + new
    return {"o": torch.cat(out)}
