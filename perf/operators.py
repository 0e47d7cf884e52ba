"""The operators of a decode step around its weight-streaming GEMMs, as measured cases.

    append     write new keys and values into a paged cache        wsm.paged_cache_append
    attention  one new token of each sequence over a paged cache   wsm.paged_attention
    experts    matrix products grouped by expert, ragged rows      wsm.expert_gemm
    logprobs   log probability of given tokens, with the entropy
               of the distribution and its top alternatives        wsm.token_logprobs

A step of a model with experts runs them in this order: qkv projection, append, attention, o projection,
router, experts (gate and up, then down), and after the last layer the vocabulary projection and logprobs.
Head counts and widths are those of the repository's decode workload (32 query and 8 key-value heads of 128,
width 4096) and neighbours of them; page sizes, expert counts and vocabularies are generic.
"""
import math
import random

import torch

own = False

DEVICE = "cuda"
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32, "e4m3": torch.float8_e4m3fn}
WIDTH = {"bf16": 2, "fp16": 2, "fp32": 4, "e4m3": 1}


# ------------------------------------------------------------------ cases

def _attention(name, batch, heads, kv_heads, dim, page, short, length, window=0, query="bf16", cache="bf16",
               layout="token"):
    case = {"op": "attention", "batch": batch, "heads": heads, "kv_heads": kv_heads, "dim": dim, "page": page,
            "short": short, "length": length, "window": window, "query": query, "cache": cache, "layout": layout}
    return {"name": name, **case} if name else case


def _append(name, tokens, kv_heads, dim, page, dtype="bf16", layout="token", padded=0):
    case = {"op": "append", "tokens": tokens, "kv_heads": kv_heads, "dim": dim, "page": page, "dtype": dtype,
            "layout": layout, "padded": padded}
    return {"name": name, **case} if name else case


def _experts(name, rows, experts, inner, outer, silu, scaled=False, skew=0.5, dtype="bf16"):
    case = {"op": "experts", "rows": rows, "experts": experts, "inner": inner, "outer": outer, "silu": silu,
            "scaled": scaled, "skew": skew, "dtype": dtype}
    return {"name": name, **case} if name else case


def _logprobs(name, rows, vocab, top, dtype="fp32", masked=0.0, pad=0):
    case = {"op": "logprobs", "rows": rows, "vocab": vocab, "top": top, "dtype": dtype, "masked": masked, "pad": pad}
    return {"name": name, **case} if name else case


def listed():
    return [
        # a single chat at its start: nothing but latency
        _attention("attention_1x37", 1, 32, 8, 128, 16, 37, 37),
        # a server's ordinary batch, ragged, with an idle slot
        _attention("attention_64_ragged", 64, 32, 8, 128, 16, 1, 4096),
        # one long document: few rows, so the length itself is split
        _attention("attention_1x131041", 1, 32, 8, 128, 64, 131041, 131041),
        # a full batch over an 8-bit cache, seven query heads to a key-value head, fp16 queries
        _attention("attention_96_e4m3", 96, 28, 4, 128, 32, 200, 8192, query="fp16", cache="e4m3", layout="head"),
        # the new token of every sequence of a batch, with idle slots
        _append("append_64", 64, 8, 128, 16, padded=5),
        # a prompt's keys and values
        _append("append_prompt_16001", 16001, 8, 128, 16),
        # eight tokens, each to two experts: gate and up with their activation
        _experts("experts_decode_16", 16, 32, 4096, 4096, True),
        # a server's batch, 8 experts to a token: the down projection, each row times its router weight
        _experts("experts_batch_1000", 1000, 64, 1280, 4096, False, scaled=True, skew=1.0),
        # a prompt of 4096 tokens to two experts each
        _experts("experts_prompt_8192", 8192, 16, 4096, 6144, True),
        # a few chats: fp32 logits as the vocabulary projection leaves them
        _logprobs("logprobs_4", 4, 131072, 8),
        # a batch under a grammar that leaves one token in ten
        _logprobs("logprobs_128_masked", 128, 128000, 20, dtype="bf16", masked=0.9),
        # scoring a prompt: the rows of an odd vocabulary, no alternatives asked
        _logprobs("logprobs_2049_odd", 2049, 100003, 0),
    ]


def _spread(rng, low, high):
    """A whole number, spread evenly over its logarithm."""
    return max(low, min(high, round(math.exp(rng.uniform(math.log(low), math.log(high))))))


def draw(rng):
    op = rng.choice(["attention", "attention", "append", "experts", "experts", "logprobs"])
    if op == "attention":
        kv_heads, group = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 4, 5, 7, 8, 16])
        dim, batch = rng.choice([64, 128, 128, 256]), _spread(rng, 1, 160)
        most = max(64, min(131072, (1 << 29) // (batch * kv_heads * dim)))
        length = _spread(rng, 16, most)
        query = rng.choice(["bf16", "fp16"])
        return _attention(None, batch, kv_heads * group, kv_heads, dim, rng.choice([16, 32, 64, 128]),
                          _spread(rng, 1, length), length, rng.choice([0, 0, 0, 1000]), query,
                          rng.choice([query, query, "e4m3"]), rng.choice(["token", "head"]))
    if op == "append":
        tokens = _spread(rng, 1, 16001)
        return _append(None, tokens, rng.choice([1, 2, 4, 8]), rng.choice([64, 128]), rng.choice([16, 32, 64]),
                       rng.choice(["bf16", "fp16"]), rng.choice(["token", "head"]), rng.randrange(0, 1 + tokens // 4))
    if op == "experts":
        experts = _spread(rng, 2, 128)
        inner = 8 * _spread(rng, 32, 640)
        silu = rng.random() < 0.5
        outer = 16 * _spread(rng, 8, max(8, min(384, (1 << 30) // (experts * inner * 16))))
        if not silu:
            outer -= rng.randrange(0, 16)
        return _experts(None, _spread(rng, 1, 8192), experts, inner, outer, silu, rng.random() < 0.5,
                        rng.choice([0.0, 0.5, 1.5]), rng.choice(["bf16", "fp16"]))
    vocab = _spread(rng, 1000, 200000)
    return _logprobs(None, _spread(rng, 1, max(1, min(2049, 200_000_000 // vocab))), vocab,
                     rng.choice([0, 1, 5, 20, 32]), rng.choice(["fp32", "bf16", "fp16"]), rng.choice([0.0, 0.0, 0.5]),
                     rng.choice([0, 0, 8]))


# ------------------------------------------------------------------ inputs

def _normal(gen, *shape, dtype=torch.bfloat16, scale=1.0):
    """Normal values of the given type, drawn in pieces so that the 32-bit draw stays small."""
    out = torch.empty(shape, dtype=dtype, device=DEVICE)
    flat, step = out.view(-1), 1 << 26
    for at in range(0, flat.numel(), step):
        part = flat[at:at + step]
        part.copy_(torch.randn(part.numel(), generator=gen, device=DEVICE) * scale)
    return out


def _caches(gen, pages, case, dtype):
    """Key and value caches [pages, page, kv_heads, dim], laid out token by token or head by head."""
    page, kv_heads, dim = case["page"], case["kv_heads"], case["dim"]
    if case["layout"] == "token":
        return [_normal(gen, pages, page, kv_heads, dim, dtype=dtype) for _ in range(2)]
    return [_normal(gen, pages, kv_heads, page, dim, dtype=dtype).transpose(1, 2) for _ in range(2)]


def _lengths(case, rng):
    """Tokens of each sequence; a batch of eight or more holds one slot without any."""
    lengths = [_spread(rng, case["short"], case["length"]) for _ in range(case["batch"])]
    lengths[rng.randrange(len(lengths))] = case["length"]
    if len(lengths) >= 8:
        lengths[rng.randrange(len(lengths))] = 0
    return lengths


def prepare(case, seed):
    gen, rng = torch.Generator(DEVICE).manual_seed(seed), random.Random(seed)
    state = {"case": case}
    if case["op"] == "attention":
        batch, heads, kv_heads, dim, page = (case[k] for k in ("batch", "heads", "kv_heads", "dim", "page"))
        lengths = _lengths(case, rng)
        need = [-(-n // page) for n in lengths]
        wide = max(1, max(need))
        # the pool's pages, handed out in no order; entries past a sequence's last page are not read
        order = torch.randperm(sum(need) + 3, generator=gen, device=DEVICE).int()
        held = torch.arange(wide, device=DEVICE)[None, :] < torch.tensor(need, device=DEVICE)[:, None]
        table = torch.full((batch, wide), -1, dtype=torch.int32, device=DEVICE)
        table[held] = order[:sum(need)]
        k_cache, v_cache = _caches(gen, sum(need) + 3, case, TYPES[case["cache"]])
        # the queries as the fused projection leaves them, scores of a spread as trained heads have it
        qkv = _normal(gen, batch, (heads + 2 * kv_heads) * dim, dtype=TYPES[case["query"]], scale=2.0)
        state.update(q=qkv[:, :heads * dim].view(batch, heads, dim), k_cache=k_cache, v_cache=v_cache, table=table,
                     lengths=torch.tensor(lengths, dtype=torch.int32, device=DEVICE), scale=dim ** -0.5,
                     lse=torch.empty(batch, heads, dtype=torch.float32, device=DEVICE))
        # what one number of an 8-bit cache stands for
        state.update(k_scale=0.75 if case["cache"] == "e4m3" else 1.0, v_scale=1.5 if case["cache"] == "e4m3" else 1.0)
    elif case["op"] == "append":
        tokens, kv_heads, dim, page = (case[k] for k in ("tokens", "kv_heads", "dim", "page"))
        dtype = TYPES[case["dtype"]]
        pages = -(-tokens // page) + 2
        qkv = _normal(gen, tokens, 6 * kv_heads * dim, dtype=dtype)
        k, v = (qkv[:, n * kv_heads * dim:(n + 1) * kv_heads * dim].view(tokens, kv_heads, dim) for n in (4, 5))
        slots = torch.randperm(pages * page, generator=gen, device=DEVICE)[:tokens]
        if case["padded"]:
            slots[torch.randperm(tokens, generator=gen, device=DEVICE)[:case["padded"]]] = -1
        k_cache, v_cache = _caches(gen, pages, case, dtype)
        state.update(k=k, v=v, slots=slots, k_cache=k_cache, v_cache=v_cache)
    elif case["op"] == "experts":
        rows, experts, inner, outer = (case[k] for k in ("rows", "experts", "inner", "outer"))
        dtype = TYPES[case["dtype"]]
        # some experts are liked more than others, and some get no row
        liking = (torch.randn(experts, generator=gen, device=DEVICE) * case["skew"]).exp()
        chosen = torch.multinomial(liking, rows, replacement=True, generator=gen)
        counts = torch.bincount(chosen, minlength=experts)
        offsets = torch.zeros(experts + 1, dtype=torch.int32, device=DEVICE)
        offsets[1:] = counts.cumsum(0)
        state.update(x=_normal(gen, rows, inner, dtype=dtype),
                     w=_normal(gen, experts, outer, inner, dtype=dtype, scale=inner ** -0.5),
                     offsets=offsets, bounds=offsets.tolist(),
                     row_scale=torch.rand(rows, generator=gen, device=DEVICE) if case["scaled"] else None)
    else:
        rows, vocab, dtype = case["rows"], case["vocab"], TYPES[case["dtype"]]
        logits = _normal(gen, rows, vocab + case["pad"], dtype=dtype, scale=2.5)[:, :vocab]
        # a few likely tokens in each row, and the one that was taken mostly among them
        likely = torch.randint(vocab, (rows, 1), generator=gen, device=DEVICE)
        likely = (likely + torch.arange(12, device=DEVICE) * (vocab // 12)) % vocab
        lift = torch.rand(rows, 12, generator=gen, device=DEVICE) * 12
        logits.scatter_(1, likely, (logits.gather(1, likely).float() + lift).to(dtype))
        if case["masked"]:
            out = torch.rand(rows, vocab, generator=gen, device=DEVICE) < case["masked"]
            out.scatter_(1, likely[:, :1], False)
            logits.masked_fill_(out, -math.inf)
        tokens = likely[:, 0].clone()
        if rows >= 8:
            tokens[rng.randrange(rows)] = -1  # a row of padding
        state.update(logits=logits, tokens=tokens)
    return state


# ------------------------------------------------------------------ the plain forms

def _plain_attention(s):
    case, q, table, lengths = s["case"], s["q"].float(), s["table"].long().clamp(min=0), s["lengths"].long()
    batch, heads, dim = q.shape
    kv_heads, span = case["kv_heads"], table.shape[1] * case["page"]
    k = s["k_cache"][table].float().reshape(batch, span, kv_heads, dim).permute(0, 2, 3, 1)
    v = s["v_cache"][table].float().reshape(batch, span, kv_heads, dim).transpose(1, 2)
    scores = q.view(batch, kv_heads, heads // kv_heads, dim) @ k * (s["scale"] * s["k_scale"])
    at = torch.arange(span, device=q.device)
    seen = at < lengths[:, None]
    if case["window"]:
        seen &= at >= lengths[:, None] - case["window"]
    scores = scores.masked_fill(~seen[:, None, None, :], -math.inf)
    top = scores.amax(-1, keepdim=True)
    top = top.masked_fill(top == -math.inf, 0.0)
    p = (scores - top).exp()
    total = p.sum(-1, keepdim=True)
    out = (p @ v) * s["v_scale"] / total.masked_fill(total == 0, 1.0)
    lse = (top + total.log()).view(batch, heads)
    return out.reshape(batch, heads, dim).to(s["q"].dtype), lse


def _plain_append(s):
    page, slots = s["case"]["page"], s["slots"]
    kept = (slots >= 0).nonzero().view(-1)
    at = slots[kept]
    s["k_cache"][at // page, at % page] = s["k"][kept]
    s["v_cache"][at // page, at % page] = s["v"][kept]
    return s["k_cache"], s["v_cache"]


def _plain_experts(s):
    x, w, bounds = s["x"], s["w"], s["bounds"]
    # one 32-bit product for each expert that has rows: a batched one over all experts would read them all
    y = torch.cat([x[a:b].float() @ w[e].float().T for e, (a, b) in enumerate(zip(bounds, bounds[1:])) if b > a])
    if s["case"]["silu"]:
        # gate and up rows lie in alternating blocks of eight
        y = y.view(len(y), -1, 2, 8)
        gate, up = y[:, :, 0], y[:, :, 1]
        y = (gate / (1 + (-gate).exp()) * up).reshape(len(y), -1)
    if s["row_scale"] is not None:
        y = y * s["row_scale"][:, None]
    return y.to(x.dtype)


def _plain_logprobs(s):
    x, tokens, k = s["logits"].float(), s["tokens"], s["case"]["top"]
    top = x.amax(1, keepdim=True)
    away = x - top
    e = away.exp()
    total = e.sum(1)
    rest = top.view(-1) + total.log()
    logprob = (x.gather(1, tokens.clamp(min=0)[:, None]).view(-1) - rest).masked_fill(tokens < 0, 0.0)
    entropy = total.log() - (e * away.masked_fill(away == -math.inf, 0.0)).sum(1) / total
    if not k:
        return logprob, entropy
    # one whole number for value and place, so that equal values go to the lowest index
    bits = (x + 0.0).view(torch.int32).long()
    bits = torch.where(bits < 0, -(bits & 0x7FFFFFFF), bits)
    place = torch.arange(x.shape[1], device=x.device)
    ids = (x.shape[1] - 1) - (bits * (1 << 20) + (x.shape[1] - 1 - place)).topk(k, 1).values.remainder(1 << 20)
    best = x.gather(1, ids)
    return logprob, entropy, ids.masked_fill(best == -math.inf, -1), best - rest[:, None]


# ------------------------------------------------------------------ one pass

def run(state):
    s, op = state, state["case"]["op"]
    if own:
        import weight_streaming_megakernel_b200 as wsm
        if op == "attention":
            out = wsm.paged_attention(s["q"], s["k_cache"], s["v_cache"], s["table"], s["lengths"], scale=s["scale"],
                                      window=s["case"]["window"], k_scale=s["k_scale"], v_scale=s["v_scale"],
                                      lse=s["lse"])
            return out, s["lse"]
        if op == "append":
            wsm.paged_cache_append(s["k"], s["v"], s["k_cache"], s["v_cache"], s["slots"])
            return s["k_cache"], s["v_cache"]
        if op == "experts":
            return wsm.expert_gemm(s["x"], s["w"], s["offsets"], row_scale=s["row_scale"],
                                   epilogue=wsm.EPI_SILU_MUL if s["case"]["silu"] else wsm.EPI_NONE)
        got = wsm.token_logprobs(s["logits"], s["tokens"], top=s["case"]["top"])
        return got if s["case"]["top"] else got[:2]
    return {"attention": _plain_attention, "append": _plain_append, "experts": _plain_experts,
            "logprobs": _plain_logprobs}[op](s)


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    """Bytes and operations; for what the seed decides, the middle of its range."""
    if case["op"] == "attention":
        # lengths are spread evenly over their logarithm, one of them is the longest
        low, high, batch = case["short"], case["length"], case["batch"]
        mean = (high - low) / math.log(high / low) if high > low else high
        seen = min(case["window"] or mean, mean)
        tokens = min(case["window"] or high, high) + seen * (batch - 1 - (batch >= 8))
        kv, q = case["kv_heads"] * case["dim"] * WIDTH[case["cache"]], case["heads"] * case["dim"] * 2
        return {"bytes": int(2 * tokens * kv + batch * (2 * q + 4 * case["heads"] + 4) + 4 * tokens / case["page"]),
                "flops": int(4 * tokens * case["heads"] * case["dim"])}
    if case["op"] == "append":
        row = 2 * case["kv_heads"] * case["dim"] * WIDTH[case["dtype"]]
        return {"bytes": 2 * (case["tokens"] - case["padded"]) * row + 8 * case["tokens"], "flops": 0}
    if case["op"] == "experts":
        rows, experts, inner, outer = (case[k] for k in ("rows", "experts", "inner", "outer"))
        # experts that get a row when all are liked alike
        used = experts * (1 - (1 - 1 / experts) ** rows)
        out = outer // 2 if case["silu"] else outer
        return {"bytes": int(2 * (used * inner * outer + rows * (inner + out)) + 4 * (experts + 1)
                             + (4 * rows if case["scaled"] else 0)),
                "flops": 2 * rows * inner * outer}
    rows, vocab, k = case["rows"], case["vocab"], case["top"]
    return {"bytes": rows * (vocab * WIDTH[case["dtype"]] + 8 + 8 + 12 * k), "flops": 4 * rows * vocab}


# ------------------------------------------------------------------ the definitions in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "attention":
        batch, heads, dim = s["q"].shape
        group, page = heads // case["kv_heads"], case["page"]
        out = torch.zeros(batch, heads, dim, dtype=torch.float64, device=DEVICE)
        lse = torch.full((batch, heads), -math.inf, dtype=torch.float64, device=DEVICE)
        for b, n in enumerate(s["lengths"].tolist()):
            first = max(0, n - case["window"]) if case["window"] else 0
            if n == first:
                continue
            at = torch.arange(first, n, device=DEVICE)
            pages = s["table"][b].long()[at // page]
            for h in range(case["kv_heads"]):
                k = s["k_cache"][pages, at % page, h].double() * s["k_scale"]
                v = s["v_cache"][pages, at % page, h].double() * s["v_scale"]
                mine = slice(h * group, (h + 1) * group)
                scores = s["q"][b, mine].double() @ k.T * s["scale"]
                lse[b, mine] = torch.logsumexp(scores, 1)
                out[b, mine] = torch.softmax(scores, 1) @ v
        return out, lse
    if case["op"] == "append":
        k_cache, v_cache = s["k_cache"].double(), s["v_cache"].double()
        page = case["page"]
        at = s["slots"]
        keep = at >= 0
        k_cache.index_put_((at[keep] // page, at[keep] % page), s["k"][keep].double())
        v_cache.index_put_((at[keep] // page, at[keep] % page), s["v"][keep].double())
        return k_cache, v_cache
    if case["op"] == "experts":
        parts = []
        for e in range(case["experts"]):
            mine = s["x"][s["bounds"][e]:s["bounds"][e + 1]].double()
            y = torch.einsum("rk,nk->rn", mine, s["w"][e].double())
            if case["silu"]:
                rows = torch.arange(case["outer"], device=DEVICE)
                gate, up = y[:, rows % 16 < 8], y[:, rows % 16 >= 8]
                y = gate * torch.sigmoid(gate) * up
            parts.append(y)
        y = torch.cat(parts)
        return y * s["row_scale"].double()[:, None] if case["scaled"] else y
    logprob, entropy, ids, best = [], [], [], []
    for x, t in zip(s["logits"], s["tokens"].tolist()):
        lp = torch.log_softmax(x.double(), 0)
        logprob.append(lp[t] if t >= 0 else lp.new_zeros(()))
        p = lp.exp()
        entropy.append(-(p * lp.clamp(min=-1e300)).sum())
        if case["top"]:
            value, place = x.sort(descending=True, stable=True)
            place, value = place[:case["top"]], value[:case["top"]]
            ids.append(place.masked_fill(value == -math.inf, -1))
            best.append(lp[place])
    got = [torch.stack(logprob), torch.stack(entropy)]
    return got + [torch.stack(ids), torch.stack(best)] if case["top"] else got
