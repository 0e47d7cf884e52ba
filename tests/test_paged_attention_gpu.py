"""The paged cache: appending to it, and the attention of one new token over it, against 64-bit forms."""
import itertools
import math

import pytest
import torch

import operators_ref as ref
import weight_streaming_megakernel_b200 as wsm

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
E4M3 = torch.float8_e4m3fn


@pytest.fixture(autouse=True)
def _clean():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    torch.cuda.set_device(0)
    wsm.operator_status()
    yield
    torch.cuda.synchronize()


def make(lengths, heads, kv_heads, dim, page, dtype=torch.bfloat16, cache=None, layout="token", seed=0, spare=2,
         stale=math.nan, q_scale=2.0):
    """Inputs of an attention call.  Cache slots that no token has hold `stale`; table entries past a sequence's last
    page hold numbers outside the cache."""
    g = torch.Generator().manual_seed(seed)
    need = [-(-n // page) for n in lengths]
    wide = max(1, max(need))
    order = torch.randperm(sum(need) + spare, generator=g)
    table = torch.full((len(lengths), wide), 10 ** 9, dtype=torch.int32)
    at = 0
    shape = (sum(need) + spare, page, kv_heads, dim)
    cache = cache or dtype
    k = torch.randn(shape, generator=g)
    v = torch.randn(shape, generator=g)
    dead = torch.ones(shape[:2], dtype=torch.bool)
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n].int()
        for i in range(n):
            dead[order[at + i], :min(page, lengths[b] - i * page)] = False
        at += n
    k[dead], v[dead] = stale, stale
    k, v = k.to(cache), v.to(cache)
    if layout == "head":
        k, v = (t.transpose(1, 2).contiguous().to(DEV).transpose(1, 2) for t in (k, v))
    q = (torch.randn(len(lengths), heads, dim, generator=g) * q_scale).to(dtype)
    return (q.to(DEV), k.to(DEV), v.to(DEV), table.to(DEV),
            torch.tensor(lengths, dtype=torch.int32, device=DEV))


def run_and_check(args, window=0, k_scale=1.0, v_scale=1.0, scale=None, what=""):
    q, k, v, table, lengths = args
    lse = torch.full(q.shape[:2], 7.0, device=DEV)
    out = wsm.paged_attention(q, k, v, table, lengths, window=window, k_scale=k_scale, v_scale=v_scale, scale=scale, lse=lse)
    torch.cuda.synchronize()
    want = ref.attention(q, k, v, table, lengths, q.shape[-1] ** -0.5 if scale is None else scale, window, k_scale, v_scale)
    ref.check_attention(out, lse, want, torch.float16 if k.dtype == E4M3 else q.dtype, what)
    assert wsm.operator_status() == 0
    return out, lse


# ------------------------------------------------------------------ attention

@pytest.mark.parametrize("length", [1, 2, 15, 16, 17, 31, 33, 127, 128, 129, 130, 257, 1000])
def test_lengths(length):
    run_and_check(make([length], 8, 2, 128, 16, seed=length))


@pytest.mark.parametrize("dim", [64, 96, 128, 256])
@pytest.mark.parametrize("dtype,cache", [(torch.bfloat16, None), (torch.float16, None), (torch.bfloat16, E4M3),
                                         (torch.float16, E4M3)])
@pytest.mark.parametrize("layout", ["token", "head"])
def test_types_and_dims(dim, dtype, cache, layout):
    args = make([0, 1, 77, 300, 129, 16], 8, 2, dim, 16, dtype, cache, layout, seed=dim)
    scales = dict(k_scale=0.5, v_scale=1.75) if cache == E4M3 else {}
    run_and_check(args, **scales)


@pytest.mark.parametrize("heads,kv_heads", [(1, 1), (4, 4), (7, 1), (28, 4), (16, 1), (17, 1), (40, 2), (64, 1), (33, 3)])
def test_head_groups(heads, kv_heads):
    run_and_check(make([200, 3, 0, 513], heads, kv_heads, 64, 32, seed=heads))
    run_and_check(make([140, 9], heads, kv_heads, 64, 32, torch.bfloat16, E4M3, seed=heads))


@pytest.mark.parametrize("page", [1, 3, 16, 24, 100, 256])
def test_page_sizes(page):
    run_and_check(make([1, 99, 250, 400], 8, 2, 64, page, seed=page))


@pytest.mark.parametrize("window", [1, 5, 16, 100, 128, 400, 5000])
def test_window(window):
    run_and_check(make([0, 1, 90, 350, 700], 8, 2, 64, 16, seed=window), window=window)


def test_long_and_ragged():
    """Few long sequences are cut over the whole GPU and joined; short ones beside them are not."""
    run_and_check(make([9001, 3, 0, 4097, 128, 129, 1], 4, 1, 128, 64, seed=3), what="ragged")
    run_and_check(make([33333], 8, 2, 64, 16, torch.float16, seed=4), what="one")
    run_and_check(make([20011], 4, 2, 128, 32, torch.bfloat16, E4M3, seed=5), k_scale=2.0, v_scale=0.25, what="e4m3")


def test_many_sequences():
    lengths = [(37 * i * i + i) % 200 for i in range(700)]
    run_and_check(make(lengths, 2, 1, 64, 16, seed=8))


def test_most_sequences():
    """The largest batch; most rows idle."""
    lengths = [0 if i % 64 else 5 + i // 64 for i in range(4096)]
    run_and_check(make(lengths, 2, 2, 64, 16, seed=9))
    with pytest.raises(wsm.WsmError):
        q, k, v, table, lens = make([1], 2, 2, 64, 16)
        wsm.paged_attention(q.expand(4097, 2, 64).contiguous(), k, v, table.expand(4097, 1).contiguous(),
                            lens.expand(4097).contiguous())


def test_zero_sizes():
    q, k, v, table, lengths = make([5], 2, 2, 64, 16)
    assert wsm.paged_attention(q[:0], k, v, table[:0], lengths[:0]).shape == (0, 2, 64)
    # no pages at all: every sequence is empty
    lse = torch.zeros(1, 2, device=DEV)
    out = wsm.paged_attention(q, k, v, table[:, :0], lengths * 0, lse=lse)
    assert not out.any() and (lse == -math.inf).all()


def test_strided_queries_outputs_and_tables():
    """q a slice of a fused projection, out a slice of a wider buffer, the table a view: neighbours stay untouched."""
    q, k, v, table, lengths = make([70, 0, 300], 6, 2, 64, 16, seed=2)
    fused = torch.full((3, 6 + 4, 64), math.nan, dtype=q.dtype, device=DEV)
    fused[:, :6] = q
    wide = torch.full((3, 9, 64), 5.0, dtype=q.dtype, device=DEV)
    tab = torch.full((3, table.shape[1] + 3), -5, dtype=torch.int32, device=DEV)
    tab[:, :table.shape[1]] = table
    got = wsm.paged_attention(fused[:, :6], k, v, tab[:, :table.shape[1]], lengths, wide[:, 2:8])
    plain = wsm.paged_attention(q, k, v, table, lengths)
    assert torch.equal(got, plain) and (wide[:, :2] == 5).all() and (wide[:, 8:] == 5).all()
    # batch and heads swapped in memory
    qt = q.transpose(0, 1).contiguous().transpose(0, 1)
    assert torch.equal(wsm.paged_attention(qt, k, v, table, lengths), plain)


def test_interleaved_key_value_cache():
    """K and V in one buffer, page by page."""
    q, k, v, table, lengths = make([40, 200], 4, 2, 64, 16, seed=6)
    both = torch.stack([k, v], 1)
    assert torch.equal(wsm.paged_attention(q, both[:, 0], both[:, 1], table, lengths), wsm.paged_attention(q, k, v, table, lengths))


def test_bad_pages_are_left_out_and_recorded():
    q, k, v, table, lengths = make([100, 64], 4, 2, 64, 16, seed=1)
    for bad in (-1, k.shape[0], 2 ** 31 - 1, -2 ** 31):
        t = table.clone()
        t[0, 2] = bad
        lse = torch.zeros(2, 4, device=DEV)
        out = wsm.paged_attention(q, k, v, t, lengths, lse=lse)
        assert wsm.operator_status() == wsm.WSM_ERR_INVALID and "sequence" in wsm.last_error()
        assert wsm.operator_status() == 0
        ref.check_attention(out, lse, ref.attention(q, k, v, t, lengths, 64 ** -0.5), q.dtype, f"page {bad}")
    t = torch.full_like(table, -1)
    out = wsm.paged_attention(q, k, v, t, lengths)
    assert not out.any() and wsm.operator_status() == wsm.WSM_ERR_INVALID


def test_lengths_out_of_range():
    q, k, v, table, lengths = make([48, 20], 4, 2, 64, 16, stale=0.5, seed=1)
    bad = torch.tensor([10 ** 6, -3], dtype=torch.int32, device=DEV)
    t = table.clone()
    t[1] = t[0]
    out = wsm.paged_attention(q, k, v, t, bad)
    assert wsm.operator_status() == wsm.WSM_ERR_INVALID
    full = torch.tensor([48, 0], dtype=torch.int32, device=DEV)
    assert torch.equal(out, wsm.paged_attention(q, k, v, t, full)) and not out[1].any()


def test_infinities_and_nan():
    """Infinite scores and NaN spread as in the formula; a sequence with nothing but -infinity gives zeros."""
    q, k, v, table, lengths = make([50, 50, 50, 50], 2, 1, 64, 16, seed=4)
    q, k = q.abs(), k.clone()
    k[table[0].long(), :, :, 0] = -math.inf             # all scores -infinity
    k[table[1, 0].long(), 3, 0, 5] = math.inf           # one +infinity: NaN
    k[table[2, 0].long(), 3, 0, 5] = -math.inf          # one -infinity: that token has no weight
    v = v.clone()
    v[table[3, 1].long(), 2, 0, 7] = math.nan           # one NaN value: its column only
    lse = torch.zeros(4, 2, device=DEV)
    out = wsm.paged_attention(q, k, v, table, lengths, lse=lse)
    assert not out[0].any() and (lse[0] == -math.inf).all()
    assert torch.isnan(out[1]).all()
    assert torch.isfinite(out[2]).all() and torch.isfinite(lse[2]).all()
    assert torch.isnan(out[3, :, 7]).all() and torch.isfinite(out[3][:, torch.arange(64) != 7]).all()
    want = ref.attention(q[2:3], k, v, table[2:3], lengths[2:3], 64 ** -0.5)
    ref.check_attention(out[2:3], lse[2:3], want, q.dtype)


def test_wide_range_queries_on_an_8_bit_cache():
    """bf16 queries far outside fp16's range, and rows of zeros."""
    q, k, v, table, lengths = make([60, 60, 60, 60], 2, 1, 64, 16, torch.bfloat16, E4M3, seed=4)
    q = q * torch.tensor([1e30, 1e-30, 0.0, 1.0], device=DEV, dtype=q.dtype)[:, None, None]
    for b, scale in ((0, 1e-31), (1, 1e30), (2, 1.0), (3, 0.125)):
        run_and_check((q[b:b + 1], k, v, table[b:b + 1], lengths[b:b + 1]), scale=scale, what=str(b))


def test_offsets_past_32_bits():
    """Pages more than 2^31 elements apart."""
    far = (1 << 31) + 1024
    buf = torch.empty(2 * far + 16 * 64, dtype=torch.bfloat16, device=DEV)
    big = buf.as_strided((3, 16, 1, 64), (far, 64, 64, 1))
    q, k, v, table, lengths = make([48], 2, 1, 64, 16, spare=0, seed=7)
    big.copy_(k)
    assert torch.equal(wsm.paged_attention(q, big, big, table, lengths), wsm.paged_attention(q, k, k, table, lengths))
    out = torch.zeros_like(k)
    slots = torch.arange(48, device=DEV)
    rows = k.reshape(48, 1, 64)
    big.zero_()
    wsm.paged_cache_append(rows, rows, big, v, slots)
    assert torch.equal(big, k) and not out.any()


def test_runs_are_bitwise_alike():
    args = make([5000, 17, 2048], 8, 2, 128, 16, seed=11)
    first = wsm.paged_attention(*args)
    for _ in range(20):
        assert torch.equal(wsm.paged_attention(*args), first)


def test_graphs_and_streams():
    """Two graphs captured on one stream and replayed together, beside eager calls on a third stream."""
    cases = [make([3000, 40], 8, 2, 128, 16, seed=s) for s in (1, 2, 3)]
    want = [wsm.paged_attention(*c) for c in cases]
    outs, graphs = [], []
    side = torch.cuda.Stream()
    for c in cases[:2]:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            outs.append(wsm.paged_attention(*c))
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    eager = []
    for _ in range(30):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        eager.append(wsm.paged_attention(*cases[2], stream=streams[2]))
    torch.cuda.synchronize()
    assert torch.equal(outs[0], want[0]) and torch.equal(outs[1], want[1])
    assert all(torch.equal(e, want[2]) for e in eager)


# ------------------------------------------------------------------ append

@pytest.mark.parametrize("dtype,cache", [(torch.bfloat16, torch.bfloat16), (torch.float16, torch.float16),
                                         (torch.bfloat16, E4M3), (torch.float16, E4M3)])
@pytest.mark.parametrize("tokens,heads,dim,page", [(1, 1, 64, 16), (5, 8, 128, 16), (333, 2, 64, 7), (70, 16, 256, 32),
                                                   (1000, 3, 48, 64), (3, 1, 16, 1)])
@pytest.mark.parametrize("layout", ["token", "head"])
def test_append(dtype, cache, tokens, heads, dim, page, layout):
    g = torch.Generator().manual_seed(tokens)
    pages = -(-tokens // page) + 2
    fused = (torch.randn(tokens, 3 * heads * dim, generator=g) * 3).to(dtype).to(DEV)
    k, v = (fused[:, i * heads * dim:(i + 1) * heads * dim].view(tokens, heads, dim) for i in (1, 2))
    slots = torch.randperm(pages * page, generator=g)[:tokens]
    slots[::5] = -1 - slots[::5]
    shape = (pages, page, heads, dim)
    old = [torch.randn(shape, generator=g).to(cache) for _ in range(2)]
    caches = [t.to(DEV) if layout == "token" else t.transpose(1, 2).contiguous().to(DEV).transpose(1, 2) for t in old]
    scales = (0.25, 1.5) if cache == E4M3 else (1.0, 1.0)
    wsm.paged_cache_append(k, v, *caches, slots.to(DEV), k_scale=scales[0], v_scale=scales[1])
    assert wsm.operator_status() == 0
    for rows, before, got, scale in zip((k, v), old, caches, scales):
        want = before.float()
        for t, s in enumerate(slots.tolist()):
            if s >= 0:
                x = rows[t].float().cpu()
                want[s // page, s % page] = (x / scale).clamp(-448, 448).to(cache).float() if cache == E4M3 else x
        assert torch.equal(got.float().cpu(), want)


def test_append_saturates_and_keeps_nan():
    k = torch.tensor([1e4, -1e4, 448.0, 465.0, math.nan, 2.0 ** -9, 2.0 ** -11, -0.0] * 2, dtype=torch.bfloat16, device=DEV).view(1, 1, 16)
    cache = torch.zeros(1, 1, 1, 16, dtype=E4M3, device=DEV)
    wsm.paged_cache_append(k, k, cache, cache.clone(), torch.zeros(1, dtype=torch.int64, device=DEV))
    got = cache.float().view(-1)[:8].tolist()
    assert got[:4] == [448.0, -448.0, 448.0, 448.0] and math.isnan(got[4]) and got[5:7] == [2.0 ** -9, 0.0]


def test_append_bad_slots_are_skipped_and_recorded():
    k = torch.ones(3, 1, 64, dtype=torch.bfloat16, device=DEV)
    kc, vc = (torch.zeros(4, 16, 1, 64, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    wsm.paged_cache_append(k, k, kc, vc, torch.tensor([64, 2 ** 62, 5], device=DEV))
    assert wsm.operator_status() == wsm.WSM_ERR_INVALID
    assert (kc.view(64, 64)[5] == 1).all() and int(kc.count_nonzero()) == 64 and int(vc.count_nonzero()) == 64
    wsm.paged_cache_append(k[:0], k[:0], kc, vc, torch.empty(0, dtype=torch.int64, device=DEV))


def test_append_then_attention_in_a_graph():
    """A captured step: the new token of each sequence goes in and takes part at once; lengths and slots move between
    replays, as a decode loop moves them."""
    q, k, v, table, lengths = make([30, 47, 0], 4, 2, 64, 16, stale=0.0, seed=3)
    table = torch.cat([table, torch.tensor([[4], [5], [6]], dtype=torch.int32, device=DEV)], 1)
    pool = torch.zeros(7, 16, 2, 64, dtype=torch.bfloat16, device=DEV)
    pool[:k.shape[0]] = k
    vpool = torch.zeros_like(pool)
    vpool[:v.shape[0]] = v
    # the sequences' pages in order: 2, 3 and 0 pages before, one more each
    table = torch.tensor([[0, 1, 2], [3, 4, 5], [6, 6, 6]], dtype=torch.int32, device=DEV)
    new = torch.randn(3, 2, 64, device=DEV).to(torch.bfloat16)
    slots = torch.empty(3, dtype=torch.int64, device=DEV)

    def place(lens):
        for b, n in enumerate(lens.tolist()):
            slots[b] = int(table[b, (n - 1) // 16]) * 16 + (n - 1) % 16

    lens = torch.tensor([31, 48, 1], dtype=torch.int32, device=DEV)
    place(lens)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        wsm.paged_cache_append(new, new, pool, vpool, slots)
        out = wsm.paged_attention(q, pool, vpool, table, lens)
    for step in range(4):
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(pool.view(-1, 2, 64)[slots], new)
        ref.check_attention(out, None, ref.attention(q, pool, vpool, table, lens, 0.125), q.dtype, f"step {step}")
        lens.add_(torch.tensor([1, 0, 2], dtype=torch.int32, device=DEV))
        place(lens)
        new.normal_()
    assert wsm.operator_status() == 0
