"""The token mixers beside the quantised decode step, as cases to measure: the prompt form of
the recurrences, the single-token form of the additive one, the paged key/value cache, and the
attention that reads it.

    prompt   S_t = a_t S_{t-1} + k_t u_t^T,  o_t = S_t^T q_t  over whole prompts, where
             u_t = v_t ("sum") or u_t = beta_t (v_t - a_t S_{t-1}^T k_t) ("delta")
    step     the same recurrence ("sum") for one token of each request, in place
    cache    8-bit codes of new keys and values, one scale per token and head, and back
    attend   softmax(scale q K^T) V of a chunk of new tokens over their pages

Where `own` is true, `run` calls the library; otherwise it evaluates the formulas with plain
torch operations in 32 bits (the decays' logarithms in 64).
"""
import math
import random

import torch

own = False

D = 128            # key and value channels of a head
CHUNK = 64         # tokens the plain prompt form takes at a time
LOG_ZERO = -2000.0  # stands for log2(0): 2^-2000 is zero in 32 and in 64 bits


# ---------------------------------------------------------------- cases

def listed():
    return [
        # one short prompt of a small model: launches and latency
        {"name": "prompt delta short", "op": "prompt", "rule": "delta", "n": 1, "tokens": 37, "heads": 4, "carry": False, "ragged": 0},
        # a serving batch of prompts of unlike lengths
        {"name": "prompt delta batch", "op": "prompt", "rule": "delta", "n": 32, "tokens": 16411, "heads": 32, "carry": False, "ragged": 1},
        # one long document, continued from the state of its first part
        {"name": "prompt delta long", "op": "prompt", "rule": "delta", "n": 1, "tokens": 32768, "heads": 48, "carry": True, "ragged": 0},
        # the additive rule: a batch whose requests continue
        {"name": "prompt sum batch", "op": "prompt", "rule": "sum", "n": 8, "tokens": 16000, "heads": 48, "carry": True, "ragged": 2},
        # and one long prompt with few heads, where only the columns of the states run side by side
        {"name": "prompt sum long", "op": "prompt", "rule": "sum", "n": 1, "tokens": 16385, "heads": 16, "carry": False, "ragged": 0},
        # one request's next token
        {"name": "step one", "op": "step", "n": 1, "heads": 32, "dtype": "float32"},
        # a full batch's next tokens
        {"name": "step batch", "op": "step", "n": 256, "heads": 48, "dtype": "bfloat16"},
        # the new tokens of one decode step enter the cache
        {"name": "cache step", "op": "cache", "n": 64, "tokens": 64, "heads": 8, "page": 64, "kind": 8},
        # the tokens of a batch of prompts enter the cache
        {"name": "cache prompt", "op": "cache", "n": 5, "tokens": 16391, "heads": 8, "page": 64, "kind": 8},
        # one request's next token over a short context
        {"name": "attend one", "op": "attend", "n": 1, "new": 1, "context": 777, "q_heads": 8, "heads": 2, "page": 32, "kind": 16, "ragged": 0},
        # a batch's next tokens over 8-bit caches
        {"name": "attend decode", "op": "attend", "n": 64, "new": 1, "context": 8192, "q_heads": 32, "heads": 8, "page": 64, "kind": 8, "ragged": 3},
        # chunks of prompts over what is cached of them
        {"name": "attend chunk", "op": "attend", "n": 4, "new": 1024, "context": 8192, "q_heads": 32, "heads": 8, "page": 64, "kind": 16, "ragged": 4},
    ]


def _between(rng, lo, hi):
    """An integer whose logarithm is spread evenly over [lo, hi]."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("prompt", "prompt", "step", "cache", "attend", "attend"))
    if op == "prompt":
        n = _between(rng, 1, 32)
        heads = _between(rng, 1, 48)
        tokens = _between(rng, n, max(n, min(32768, 700000 // heads)))
        return {"op": op, "rule": rng.choice(("delta", "sum")), "n": n, "tokens": tokens, "heads": heads,
                "carry": rng.random() < 0.5, "ragged": rng.randrange(1, 1000)}
    if op == "step":
        return {"op": op, "n": _between(rng, 1, 256), "heads": _between(rng, 1, 48), "dtype": rng.choice(("float32", "bfloat16"))}
    if op == "cache":
        tokens = _between(rng, 1, 16384)
        return {"op": op, "n": _between(rng, 1, min(tokens, 64)), "tokens": tokens, "heads": _between(rng, 1, 16),
                "page": rng.choice((32, 64, 128, 256)), "kind": rng.choice((8, 16))}
    heads = rng.choice((1, 2, 4, 8))
    group = rng.choice((1, 2, 3, 4, 7, 8, 16))
    if heads * group > 64:
        group = 8
    new = 1 if rng.random() < 0.5 else _between(rng, 2, 1024)
    n = _between(rng, 1, 64 if new == 1 else max(1, min(32, 4096 // new)))
    context = _between(rng, new, 8192)
    return {"op": op, "n": n, "new": new, "context": context, "q_heads": heads * group, "heads": heads,
            "page": rng.choice((32, 64, 128, 256)), "kind": rng.choice((8, 16)), "ragged": rng.randrange(0, 1000)}


def _lengths(case):
    """Tokens of each prompt: they add up to the case's count; a ragged batch has short, long and (rarely) empty ones."""
    n, tokens = case["n"], case["tokens"]
    if n == 1 or not case["ragged"]:
        return [tokens // n + (i < tokens % n) for i in range(n)]
    r = random.Random(case["ragged"])
    cut = [0] + sorted(r.randrange(0, tokens + 1) for _ in range(n - 1)) + [tokens]
    return [b - a for a, b in zip(cut, cut[1:])]


def _contexts(case):
    """(new tokens, cached tokens with the new ones among them) of each request; the first has the case's counts."""
    r = random.Random(case["ragged"])
    got = [(case["new"], case["context"])]
    for _ in range(case["n"] - 1):
        new = case["new"] if not case["ragged"] else r.randrange(max(1, case["new"] // 2), case["new"] + 1)
        got.append((new, case["context"] if not case["ragged"] else r.randrange(max(new, case["context"] // 2), case["context"] + 1)))
    return got


def work(case):
    op = case["op"]
    if op == "prompt":
        t, states = case["tokens"] * case["heads"], case["n"] * case["heads"]
        delta = case["rule"] == "delta"
        return {"bytes": t * (4 * D * 2 + (8 if delta else 4)) + states * D * D * 4 * (2 if case["carry"] else 1),
                "flops": t * 2 * D * D * (3 if delta else 2)}
    if op == "step":
        s = case["n"] * case["heads"]
        return {"bytes": s * (2 * D * D * 4 + 4 * D * (4 if case["dtype"] == "float32" else 2) + 4), "flops": s * 5 * D * D}
    if op == "cache":
        t = case["tokens"] * case["heads"] * 2
        code = D * case["kind"] // 8 + (4 if case["kind"] == 8 else 0)
        return {"bytes": t * (2 * D * 2 + 2 * code), "flops": t * 4 * D}
    both = _contexts(case)
    code = D * case["kind"] // 8 + (4 if case["kind"] == 8 else 0)
    seen = sum(new * (context - new) + new * (new + 1) // 2 for new, context in both)
    return {"bytes": sum(c for _, c in both) * case["heads"] * 2 * code + sum(m for m, _ in both) * case["q_heads"] * 2 * D * 2,
            "flops": seen * case["q_heads"] * 4 * D}


# ---------------------------------------------------------------- inputs

def _normal(g, *shape):
    return torch.randn(shape, generator=g, device="cuda")


def _unit(x):
    return x / x.norm(dim=-1, keepdim=True)


def _inputs(case, seed):
    """Inputs of a case, made from the seed alone."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    op, bf16 = case["op"], torch.bfloat16
    if op == "prompt":
        n, t, h = case["n"], case["tokens"], case["heads"]
        lens = _lengths(case)
        s = {"lens": lens,
             "cu": torch.tensor([0] + lens, device="cuda").cumsum(0).to(torch.int32),
             "slots": torch.randperm(n, generator=g, device="cuda").to(torch.int32),
             # queries and keys of unit length and gates exp(-g), as the decode step has them
             "q": (_unit(_normal(g, t, h, D)) / math.sqrt(D)).to(bf16), "k": _unit(_normal(g, t, h, D)).to(bf16),
             "v": _normal(g, t, h, D).to(bf16),
             "gate": torch.exp2(-torch.exp2(-12 * torch.rand((t, h), generator=g, device="cuda"))),
             "beta": torch.rand((t, h), generator=g, device="cuda") if case["rule"] == "delta" else None,
             "o": torch.empty((t, h, D), dtype=bf16, device="cuda")}
        s["S"] = _normal(g, n, h, D, D) if case["carry"] else torch.zeros((n, h, D, D), device="cuda")
        return s
    if op == "step":
        n, h, dt = case["n"], case["heads"], getattr(torch, case["dtype"])
        return {"slots": torch.randperm(n, generator=g, device="cuda").to(torch.int32),
                "q": (_unit(_normal(g, n, h, D)) / math.sqrt(D)).to(dt), "k": _unit(_normal(g, n, h, D)).to(dt),
                "v": _normal(g, n, h, D).to(dt), "gate": torch.exp2(-torch.exp2(-12 * torch.rand((n, h), generator=g, device="cuda"))),
                "o": torch.empty((n, h, D), dtype=dt, device="cuda"), "S": _normal(g, n, h, D, D)}
    # keys and values with unlike tokens and a few strong channels
    def vectors(t, h):
        x = _normal(g, t, h, D) * torch.exp2(2 * torch.rand((t, h, 1), generator=g, device="cuda"))
        x[:, :, ::37] *= 3
        return x.to(bf16)
    page, h = case["page"], case["heads"]
    if op == "cache":  # each request writes behind what it has cached before
        n, t, r = case["n"], case["tokens"], random.Random(case["tokens"])
        new = [t // n + (i < t % n) for i in range(n)]
        both = [(m, m + r.randrange(0, 300)) for m in new]
    else:
        both = _contexts(case)
    need = [-(-c // page) for _, c in both]
    pages, most = sum(need) + 3, max(need)
    order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    table = torch.full((case["n"], most), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, m in enumerate(need):
        table[b, :m] = order[at:at + m]
        at += m
    t = sum(new for new, _ in both)
    s = {"both": both, "pages": pages, "table": table, "context": torch.tensor([c for _, c in both], dtype=torch.int32, device="cuda"),
         "cu": torch.tensor([0] + [new for new, _ in both], device="cuda").cumsum(0).to(torch.int32)}
    if op == "cache":
        return {**s, "k": vectors(t, h), "v": vectors(t, h), "k_out": torch.empty((t, h, D), dtype=bf16, device="cuda"),
                "v_out": torch.empty((t, h, D), dtype=bf16, device="cuda")}
    kv = sum(c for _, c in both)
    return {**s, "k": vectors(kv, h), "v": vectors(kv, h), "q": _normal(g, t, case["q_heads"], D).to(bf16),
            "whole": torch.tensor([0] + [c for _, c in both], device="cuda").cumsum(0).to(torch.int32),
            "o": torch.empty((t, case["q_heads"], D), dtype=bf16, device="cuda"), "scale": 1 / math.sqrt(D)}


def prepare(case, seed):
    s = _inputs(case, seed)
    s["case"] = case
    op = case["op"]
    if op in ("prompt", "step"):
        n, h = case["n"], case["heads"]
        if own:  # the pool that keeps the states, uncompressed
            from quantized_delta_rule_decode_amd import qdr
            s["memory"] = torch.empty(n * h * D * D, dtype=torch.float32, device="cuda")
            s["pool"] = qdr.Pool(n, h, [qdr.K_FP32] * h, None, scale_mode=qdr.SCALE_ROW_ABSMAX, dev_mem=s["memory"])
            s["pool"].qdr_pack(torch.arange(n, dtype=torch.int32, device="cuda"), s.pop("S"))
            if op == "prompt":
                s["rule"] = qdr.RULE_DELTA if case["rule"] == "delta" else qdr.RULE_SUM
                s["carry"] = torch.ones(n, dtype=torch.int32, device="cuda") if case["carry"] else None
                s["workspace"] = torch.empty(s["pool"].qdr_prompt_workspace(n, case["tokens"]), dtype=torch.uint8, device="cuda")
        return s
    if own:
        from quantized_delta_rule_decode_amd import qdr
        s["cache"] = qdr.KVCache(s["pages"], case["page"], case["heads"], case["kind"])
        if op == "attend":
            s["cache"].qdr_kv_write(s["table"], s["whole"], s["context"], s.pop("k"), s.pop("v"))
            s["workspace"] = torch.empty(s["cache"].qdr_kv_attend_workspace(case["n"], s["q"].shape[0], case["q_heads"], s["table"].shape[1]), dtype=torch.uint8, device="cuda")
        return s
    shape = (s["pages"] * case["page"], case["heads"])
    if case["kind"] == 8:
        s["codes"] = [torch.zeros(shape + (D,), dtype=torch.int8, device="cuda") for _ in range(2)]
        s["scales"] = [torch.zeros(shape, device="cuda") for _ in range(2)]
    else:
        s["values"] = [torch.zeros(shape + (D,), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    if op == "attend":
        _store(s, _places(s, s["whole"]), s.pop("k"), s.pop("v"))
    return s


# ---------------------------------------------------------------- one pass

def run(state):
    case = state["case"]
    op = case["op"]
    if op == "prompt":
        if own:
            state["pool"].qdr_prompt(state["rule"], state["slots"], state["cu"], state["q"], state["k"], state["v"], state["beta"],
                                     state["gate"], state["o"], carry=state["carry"], workspace=state["workspace"])
            return {"o": state["o"], "S": _rows(state)}
        return _plain_prompt(state)
    if op == "step":
        if own:
            step = state["pool"].qdr_linear_step if case["dtype"] == "float32" else state["pool"].qdr_linear_step_bf16
            step(state["slots"], state["q"], state["k"], state["v"], state["gate"], state["o"])
            return {"o": state["o"], "S": _rows(state)}
        return _plain_step(state)
    if op == "cache":
        if own:
            state["cache"].qdr_kv_write(state["table"], state["cu"], state["context"], state["k"], state["v"])
            state["cache"].qdr_kv_read(state["table"], state["cu"], state["context"], state["k_out"], state["v_out"])
            return {"k": state["k_out"], "v": state["v_out"]}
        at = _places(state, state["cu"])
        _store(state, at, state["k"], state["v"])
        k, v = _load(state, at)
        return {"k": k.to(torch.bfloat16), "v": v.to(torch.bfloat16)}
    if own:
        state["cache"].qdr_kv_attend(state["table"], state["cu"], state["context"], state["q"], state["o"], scale=state["scale"],
                                     workspace=state["workspace"])
        return {"o": state["o"]}
    return _plain_attend(state)


def _rows(state):
    """The states as [request, head, 32, 4, 128] rows: an uncompressed pool keeps four rows of a column together."""
    case = state["case"]
    return state["memory"].view(case["n"], case["heads"], D // 4, D, 4).permute(0, 1, 2, 4, 3)


# ---------------------------------------------------------------- plain forms

def _padded(x, at, inside):
    """Tokens laid out [request, head, chunk, CHUNK, ...], zero behind a prompt's end."""
    y = x.float()[at] * inside.view(inside.shape + (1,) * (x.dim() - 1))
    n, length = at.shape
    return y.view(n, length // CHUNK, CHUNK, *x.shape[1:]).movedim(3, 1)


def _plain_prompt(s):
    lens = torch.tensor(s["lens"], device="cuda")
    length = max(1, -(-max(s["lens"]) // CHUNK)) * CHUNK
    pos = torch.arange(length, device="cuda")
    inside = pos < lens[:, None]
    at = torch.where(inside, s["cu"][:-1].long()[:, None] + pos, 0)
    q, k, v = (_padded(s[x], at, inside) for x in ("q", "k", "v"))
    lg = torch.log2(s["gate"].double()).clamp_min(LOG_ZERO)[at] * inside[..., None]
    lg = lg.view(at.shape[0], -1, CHUNK, lg.shape[-1]).movedim(3, 1).cumsum(-1)
    step = torch.arange(CHUNK, device="cuda")
    lower = step[:, None] >= step[None, :]
    decay = torch.where(lower, torch.exp2(torch.where(lower, lg[..., :, None] - lg[..., None, :], 0)).float(), 0)
    first, last = torch.exp2(lg).float()[..., None], torch.exp2(lg[..., -1:] - lg).float()[..., None]
    kt = (k * last).transpose(-1, -2)
    scores = q @ k.transpose(-1, -2) * decay
    solve = None
    if s["beta"] is not None:
        beta = _padded(s["beta"], at, inside)
        low = torch.where(step[:, None] > step[None, :], k @ k.transpose(-1, -2) * decay, 0) * beta[..., None]
        eye = torch.eye(CHUNK, device="cuda")
        solve, power = eye - low, low @ low
        for _ in range(5):  # (1 + L)^-1 = (1 - L)(1 + L^2)(1 + L^4)... of a strictly lower L
            solve, power = solve + solve @ power, power @ power
        solve = solve * beta[..., None, :]
    S = s["S"][s["slots"].long()] * (1.0 if s["case"]["carry"] else 0.0)
    out = torch.empty_like(v)
    for c in range(v.shape[2]):
        u = v[:, :, c]
        if solve is not None:
            u = solve[:, :, c] @ (u - first[:, :, c] * (k[:, :, c] @ S))
        out[:, :, c] = first[:, :, c] * (q[:, :, c] @ S) + scores[:, :, c] @ u
        S = first[:, :, c, -1:] * S + kt[:, :, c] @ u
    s["S"][s["slots"].long()] = S
    o = out.movedim(1, 3).reshape(at.shape[0], length, -1, D)[inside].to(torch.bfloat16)
    return {"o": o, "S": s["S"].view(*S.shape[:2], D // 4, 4, D)}


def _plain_step(s):
    q, k, v = (s[x].float() for x in ("q", "k", "v"))
    at = s["slots"].long()
    S = s["gate"][..., None, None] * s["S"][at] + k[..., :, None] * v[..., None, :]
    s["S"][at] = S
    return {"o": (q[..., :, None] * S).sum(-2).to(s["q"].dtype), "S": s["S"].view(*S.shape[:2], D // 4, 4, D)}


def _places(s, cu):
    """Where the last tokens of each request are in the cache: page and row of every token that `cu` counts."""
    cu, page = cu.long(), s["case"]["page"]
    token = torch.arange(s["k"].shape[0], device="cuda")
    row = torch.searchsorted(cu[1:].contiguous(), token, right=True)
    pos = s["context"].long()[row] - cu[row + 1] + token
    return s["table"].long()[row, pos // page] * page + pos % page


def _store(s, at, k, v):
    for i, x in enumerate((k, v)):
        if s["case"]["kind"] == 16:
            s["values"][i][at] = x
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


def _plain_attend(s):
    case, page = s["case"], s["case"]["page"]
    new, context = s["cu"].diff().long(), s["context"].long()
    m, length = max(a for a, _ in s["both"]), max(b for _, b in s["both"])
    key = torch.arange(length, device="cuda")
    at = s["table"].long().clamp_min(0)[:, key // page] * page + key % page
    k, v = (x.transpose(1, 2) for x in _load(s, at))
    row = torch.arange(m, device="cuda")
    inside = row < new[:, None]
    q = s["q"].float()[torch.where(inside, s["cu"][:-1].long()[:, None] + row, 0)]
    n, h, group = case["n"], case["heads"], case["q_heads"] // case["heads"]
    q = q.view(n, m, h, group, D).permute(0, 2, 3, 1, 4).reshape(n, h, group * m, D)
    seen = key <= (context - new)[:, None, None] + row[:, None]
    scores = (q @ k.transpose(-1, -2)).view(n, h, group, m, length) * s["scale"]
    scores.masked_fill_(~seen[:, None, None], -math.inf)
    scores -= scores.amax(-1, keepdim=True)
    p = scores.exp_()
    total = p.sum(-1, keepdim=True)
    o = (p.view(n, h, group * m, length) @ torch.where((key < context[:, None])[:, None, :, None], v, 0)).view(n, h, group, m, D) / total
    return {"o": o.permute(0, 3, 1, 2, 4).reshape(n, m, case["q_heads"], D)[inside].to(torch.bfloat16)}


# ---------------------------------------------------------------- in 64 bits

def exact(case, seed):
    s = _inputs(case, seed)
    op = case["op"]
    if op == "step":
        k, v, S = s["k"].double(), s["v"].double(), s["S"].double()
        at = s["slots"].long()
        S[at] = s["gate"].double()[..., None, None] * S[at] + torch.einsum("bhi,bhj->bhij", k, v)
        return {"o": torch.einsum("bhij,bhi->bhj", S[at], s["q"].double()), "S": S.view(*S.shape[:2], D // 4, 4, D)}
    if op == "prompt":
        # token by token, every prompt at once; one that has ended keeps its state
        n, h = case["n"], case["heads"]
        lens = torch.tensor(s["lens"], device="cuda")
        S = s["S"].double()[s["slots"].long()]
        o = torch.zeros((case["tokens"], h, D), dtype=torch.float64, device="cuda")
        order = sorted(range(n), key=lambda b: -s["lens"][b])
        S, start = S[order], s["cu"][:-1].long()[order]
        for t in range(max(s["lens"])):
            live = sum(x > t for x in s["lens"])
            at = start[:live] + t
            q, k, u = (s[x][at].double() for x in ("q", "k", "v"))
            M = S[:live].mul_(s["gate"][at].double()[..., None, None])
            if s["beta"] is not None:
                u = s["beta"][at].double()[..., None] * (u - (k[..., None, :] @ M)[..., 0, :])
            M.addcmul_(k[..., :, None], u[..., None, :])
            o[at] = (q[..., None, :] @ M)[..., 0, :]
        out = torch.empty_like(S)
        out[s["slots"].long()[order]] = S
        return {"o": o, "S": out.view(n, h, D // 4, 4, D)}

    def held(x):
        x = x.double()
        if case["kind"] == 16:
            return x
        most = x.abs().amax(-1, keepdim=True)
        most = torch.where(most < 2.0 ** -126, torch.ones_like(most), most)
        return torch.round(x * 127 / most) * most / 127

    k, v = held(s["k"]), held(s["v"])
    if op == "cache":
        return {"k": k, "v": v}
    out, first, at = [], 0, 0
    group = case["q_heads"] // case["heads"]
    for new, context in s["both"]:
        K, V = k[at:at + context], v[at:at + context]
        q = s["q"][first:first + new].double()
        future = torch.arange(context, device="cuda")[None, :] > torch.arange(context - new, context, device="cuda")[:, None]
        heads = []
        for j in range(case["q_heads"]):
            z = (q[:, j] @ K[:, j // group].T) * s["scale"]
            heads.append(torch.softmax(z.masked_fill(future, -math.inf), -1) @ V[:, j // group])
        out.append(torch.stack(heads, 1))
        first, at = first + new, at + context
    return {"o": torch.cat(out)}
