"""Plain 64-bit forms of the decode-step operators, and how far a kernel may be from them.

Nothing here uses the library.  Tolerances count roundings: `half(t)` is half a step of a type relative to the
value (bf16 2^-8, fp16 2^-11), fp32 sums of n terms are off by at most n 2^-24 of the sum of their magnitudes.
"""
import math

import torch

U32 = 2.0 ** -24


def half(dtype):
    return torch.finfo(dtype).eps / 2


def attention(q, k_cache, v_cache, table, lengths, scale, window=0, k_scale=1.0, v_scale=1.0, cap=None):
    """(out, lse, sum of weight * |v|, bound on a score's error) in 64 bits, sequence by sequence; tokens on pages
    outside the cache are left out."""
    q, kc, vc = q.double().cpu(), k_cache.double().cpu(), v_cache.double().cpu()
    table, lengths = table.cpu().long(), lengths.cpu().tolist()
    batch, heads, dim = q.shape
    pages, page, kv_heads, _ = kc.shape
    group = heads // kv_heads
    out = torch.zeros(batch, heads, dim, dtype=torch.float64)
    mag = torch.zeros(batch, heads, dim, dtype=torch.float64)
    lse = torch.full((batch, heads), -math.inf, dtype=torch.float64)
    err = torch.zeros(batch, heads, 1, dtype=torch.float64)
    for b in range(batch):
        n = min(max(lengths[b], 0), table.shape[1] * page)
        at = torch.arange(max(0, n - window) if window else 0, n)
        pg = table[b][at // page] if n else at
        ok = (pg >= 0) & (pg < pages)
        at, pg = at[ok], pg[ok]
        if len(at) == 0:
            continue
        for h in range(heads):
            k = kc[pg, at % page, h // group] * k_scale
            v = vc[pg, at % page, h // group] * v_scale
            s = (k @ q[b, h]) * scale
            lse[b, h] = torch.logsumexp(s, 0)
            if lse[b, h] == -math.inf:
                continue
            w = torch.softmax(s, 0)
            out[b, h] = w @ v
            mag[b, h] = w @ v.abs()
            # a score: dim products and sums, then the factor; the weights' sum over n tokens
            reach = float((k.abs() @ q[b, h].abs()).max() * abs(scale))
            err[b, h] = (dim + 8) * U32 * reach + (n + 64) * U32 + 2.0 ** -21
    return out, lse, mag, err


def check_attention(got, lse, ref, weight_type, what=""):
    """Off by the output's rounding, the weights' rounding to 16 bits, and the scores' and sums' errors."""
    out, lse_ref, mag, err = ref
    g = got.double().cpu()
    bound = half(got.dtype) * (out.abs() + (half(weight_type) + 2 * err) * mag) + (half(weight_type) + 2 * err) * mag
    # (outputs below the type's normal range are off by half its smallest step instead)
    bound = bound + torch.finfo(got.dtype).smallest_normal * torch.finfo(got.dtype).eps / 2
    bad = ~((g - out).abs() <= bound)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} off, first at {bad.nonzero()[0].tolist()}: " \
                          f"{g[bad][0]} for {out[bad][0]} +- {bound[bad][0]}"
    if lse is not None:
        l = lse.double().cpu()
        fine = torch.isfinite(lse_ref)
        assert torch.equal(torch.isfinite(l), fine) and torch.equal(l[~fine], lse_ref[~fine]), f"{what}: lse"
        off = (l - lse_ref)[fine].abs()
        assert (off <= (2 * err[..., 0] + 4 * U32 * lse_ref.abs())[fine]).all(), f"{what}: lse off by {off.max()}"


def experts(x, w, offsets, silu, row_scale=None):
    """(y, sum of |x w| behind each product of g and u, ...): y and the bound of its error in 64 bits; rows of no
    expert are NaN.  Offsets are taken into [0, rows] and never falling."""
    x, w = x.double().cpu(), w.double().cpu()
    rows, kk = x.shape
    n = w.shape[1]
    y = torch.full((rows, n // 2 if silu else n), math.nan, dtype=torch.float64)
    bound = torch.zeros_like(y)
    at = 0
    marks = []
    for o in offsets.cpu().tolist():
        at = min(max(o, at, 0), rows)
        marks.append(at)
    # tensor-core sums: kk terms, each partial sum kept to 2^-22 of the magnitudes at least
    per = kk * 2.0 ** -22
    for e in range(w.shape[0]):
        a, b = marks[e], marks[e + 1]
        if a == b:
            continue
        p, s = x[a:b] @ w[e].T, (x[a:b].abs() @ w[e].abs().T) * per
        if silu:
            i = torch.arange(n)
            gate, up, bg, bu = p[:, i % 16 < 8], p[:, i % 16 >= 8], s[:, i % 16 < 8], s[:, i % 16 >= 8]
            act = gate * torch.sigmoid(gate)
            # |silu'| < 1.1; 2^-19 for the activation's evaluation in fp32
            p, s = act * up, 1.1 * bg * up.abs() + act.abs() * bu + 1.1 * bg * bu + 2.0 ** -19 * (act * up).abs()
        f = row_scale[a:b].double().cpu()[:, None] if row_scale is not None else 1.0
        y[a:b], bound[a:b] = p * f, s * abs(f) + 4 * U32 * (p * f).abs()
    return y, bound


def check_experts(got, ref, what=""):
    y, bound = ref
    g = got.double().cpu()
    mine = ~torch.isnan(y)
    tol = bound + half(got.dtype) * (y.abs() + bound) + torch.finfo(got.dtype).smallest_normal * torch.finfo(got.dtype).eps / 2
    bad = mine & ~((g - y).abs() <= tol)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {int(mine.sum())} off, first at {bad.nonzero()[0].tolist()}: " \
                          f"{g[bad][0]} for {y[bad][0]} +- {tol[bad][0]}"


def logprobs(logits, tokens, top):
    """(logprob, entropy, ids, logprobs of the alternatives) in 64 bits."""
    x = logits.double().cpu()
    rows, vocab = x.shape
    lp_out = torch.zeros(rows, dtype=torch.float64)
    ent = torch.zeros(rows, dtype=torch.float64)
    ids = torch.full((rows, top), -1, dtype=torch.int64)
    best = torch.full((rows, top), -math.inf, dtype=torch.float64)
    for r in range(rows):
        t = int(tokens[r]) if tokens is not None else -1
        if torch.isnan(x[r]).any() or (x[r] == math.inf).any():
            lp_out[r] = math.nan if t >= 0 else 0.0
            ent[r] = math.nan
            best[r] = math.nan
            continue
        none = bool((x[r] == -math.inf).all())
        lp = torch.full((vocab,), -math.inf, dtype=torch.float64) if none else torch.log_softmax(x[r], 0)
        lp_out[r] = math.nan if t >= vocab else lp[t] if t >= 0 else 0.0
        if not none:
            keep = lp > -math.inf
            ent[r] = -(lp[keep].exp() * lp[keep]).sum()
        order = sorted((i for i in range(vocab) if x[r, i] > -math.inf), key=lambda i: (-float(x[r, i]), i))[:top] \
            if vocab <= 4096 else [int(i) for i in torch.sort(x[r], descending=True, stable=True).indices[:top]
                                   if x[r, i] > -math.inf]
        for j, i in enumerate(order):
            ids[r, j], best[r, j] = i, lp[i]
    return lp_out, ent, ids, best


def check_logprobs(got, ref, logits, what=""):
    """A row's sum: chains of up to 96 + n / 2048 fp32 additions, 2^-22 for each power, and powers' arguments off by
    2^-24 of |y|, weighted by the weight: at most 2^-24 of the entropy's bits."""
    n = logits.shape[1]
    rel = (96 + n / 2048 + 2 * math.log2(n + 1)) * U32 + 2.0 ** -21
    lp, ent, ids, best = ref
    for name, g, e, tol in (("logprob", got.logprob, lp, rel + 8 * U32 * lp.abs()),
                            ("entropy", got.entropy, ent, rel * (4 + 2 * math.log2(n + 1))),
                            ("top_logprobs", got.top_logprobs, best, rel + 8 * U32 * best.abs())):
        g = g.double().cpu()
        fine = torch.isfinite(e)
        assert torch.equal(torch.isnan(g), torch.isnan(e)), f"{what}: {name} NaN places"
        assert torch.equal(g[~fine & ~torch.isnan(e)], e[~fine & ~torch.isnan(e)]), f"{what}: {name} infinities"
        tol = tol if isinstance(tol, float) else tol[fine]
        off = (g - e)[fine].abs()
        assert (off <= tol).all(), f"{what}: {name} off by {off.max()}"
    assert torch.equal(got.top_ids.cpu(), ids), f"{what}: alternatives"
