"""Paged attention over scores of any finite size: where one token's score is far above all others the output is that
token's value, bit for bit, however large the scores are."""
import math

import pytest
import torch

import weight_streaming_megakernel_b200 as wsm

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
E4M3 = torch.float8_e4m3fn
TYPES = [(torch.bfloat16, None), (torch.float16, None), (torch.bfloat16, E4M3), (torch.float16, E4M3)]


@pytest.fixture(autouse=True)
def _clean():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    torch.cuda.set_device(0)
    wsm.operator_status()
    yield
    torch.cuda.synchronize()


def make(lengths, best, top, dtype, cache, seed, heads=6, kv_heads=2, dim=64, page=16):
    """Queries of one element, so that a token's raw score is that element of its key, a small whole number: at most
    `top` - 1, and `top` for the tokens in best[b], a fraction of the length each.  Every sum is exact in fp32."""
    g = torch.Generator().manual_seed(seed)
    n = max(lengths)
    pages = -(-n // page)
    k = torch.zeros(len(lengths), pages * page, kv_heads, dim)
    k[..., 0] = torch.randint(top - 8, top, k.shape[:3], generator=g).float()
    v = torch.randn(k.shape, generator=g)
    at = [[min(n - 1, int(f * n)) for f in best] for n in lengths]
    for b, tokens in enumerate(at):
        k[b, tokens, :, 0] = top
    k, v = (t.to(cache or dtype).view(-1, page, kv_heads, dim).to(DEV) for t in (k, v))
    q = torch.zeros(len(lengths), heads, dim, dtype=dtype, device=DEV)
    q[..., 0] = 1
    table = torch.arange(len(lengths) * pages, dtype=torch.int32, device=DEV).view(len(lengths), pages)
    picked = torch.stack([v.view(len(lengths), -1, kv_heads, dim)[b, t].double() for b, t in enumerate(at)])
    want = picked.mean(1).repeat_interleave(heads // kv_heads, 1)
    return q, k, v, table, torch.tensor(lengths, dtype=torch.int32, device=DEV), want


# The size of the scores in base 2, as a power of two: below and past the border of the exact form, where fp32 holds them
# to 1, to tens, to thousands, and up to the largest.  `unit`: the factor in base 2 is a power of two itself, so that the
# products are exact too, or has all its bits.
@pytest.mark.parametrize("power", [9, 10, 11, 16, 23, 24, 25, 27, 28, 29, 30, 33, 40, 64, 100, 126])
@pytest.mark.parametrize("dtype,cache", TYPES)
@pytest.mark.parametrize("top", [15, -1])
@pytest.mark.parametrize("unit", [math.log2(math.e), 1.0])
def test_one_token_has_all_the_weight(power, dtype, cache, top, unit):
    k_scale, v_scale = (0.5, 2.0) if cache else (1.0, 1.0)
    scale = 2.0 ** power / (16 * k_scale * unit)
    for sign in (1.0, -1.0):
        for best in ((0.0,), (0.37,), (1.0,)):
            q, k, v, table, lengths, want = make([37, 1, 5001, 300], best, top, dtype, cache, seed=power)
            lse = torch.zeros(q.shape[:2], device=DEV)
            out = wsm.paged_attention(q * sign, k, v, table, lengths, scale=scale * sign, k_scale=k_scale, v_scale=v_scale, lse=lse)
            # the other tokens, each e^-(scale * k_scale) of the best one's weight at most, together move the output by
            # their weights times twice the largest value (a value of 0 in an 8-bit cache shows it); the rounding of that
            # to 16 bits is the factor 2: 0 but for the smallest scores
            others = 2 * 5001 * math.exp(-scale * k_scale) * 2 * float(v.float().abs().max()) * v_scale
            assert ((out.double() - (want * v_scale).to(dtype).double()).abs() <= others).all(), f"best at {best}"
            # the factor, the score, the reference, the sum's logarithm and ln 2: a rounding each
            exact = scale * k_scale * top
            assert ((lse.double() - exact).abs() <= 8 * 2.0 ** -24 * abs(exact) + 2.0 ** -20).all()
    assert wsm.operator_status() == 0


@pytest.mark.parametrize("power", [12, 24, 28, 30, 40, 100])
@pytest.mark.parametrize("dtype,cache", TYPES)
@pytest.mark.parametrize("unit", [math.log2(math.e), 1.0])
def test_equal_scores_share(power, dtype, cache, unit):
    """Two tokens, far apart in the sequence, with the largest score: the mean of their values, rounded once."""
    scale = 2.0 ** power / (16 * unit)
    q, k, v, table, lengths, want = make([40, 5001, 300], (0.1, 0.9), 15, dtype, cache, seed=power)
    out = wsm.paged_attention(q, k, v, table, lengths, scale=scale)
    assert torch.equal(out, want.to(dtype))


@pytest.mark.parametrize("dtype,cache", TYPES)
def test_scores_that_grow_past_the_border(dtype, cache):
    """Scores that rise along the sequence from small ones to 2^30, and rows of heads far apart in size."""
    q, k, v, table, lengths, want = make([3000], (1.0,), 15, dtype, cache, seed=1)
    k = k.float()
    k.view(-1, 2, 64)[:2999, :, 0] = (torch.arange(2999, device=DEV) * 14 // 2999)[:, None]
    k = k.to(cache or dtype)
    q = q * torch.tensor([2.0 ** -14, 1.0, 2.0 ** -4, 1.0, 2.0 ** -7, 2.0 ** -14], dtype=dtype, device=DEV)[:, None]
    out = wsm.paged_attention(q, k, v, table, lengths, scale=2.0 ** 26)
    assert torch.equal(out, want.to(dtype))


@pytest.mark.parametrize("dtype,cache", TYPES)
@pytest.mark.parametrize("scale", [0.0, -0.0, 2.0 ** -149])
def test_a_scale_of_nothing_is_a_mean(dtype, cache, scale):
    """All scores vanish, whatever the queries and keys: every token has the same weight."""
    size = 2.0 ** 60 if dtype == torch.bfloat16 else 2.0 ** 12
    q, k, v, table, lengths, _ = make([300, 1, 20], (0.5,), 15, dtype, cache, seed=3)
    if cache is None:
        k = (k.double() * size).to(dtype)
    lse = torch.zeros(q.shape[:2], device=DEV)
    out = wsm.paged_attention((q.double() * size).to(dtype), k, v, table, lengths, scale=scale, lse=lse)
    values = v.view(3, -1, 2, 64).double()
    for b, n in enumerate(lengths.tolist()):
        want = values[b, :n].mean(0).repeat_interleave(3, 0)
        # equal weights, whole powers of two or off by the exponential's 2^-22, and n fp32 additions
        off = 2.0 ** -9 if dtype == torch.bfloat16 else 2.0 ** -12
        slack = (n + 8) * 2.0 ** -22 * values[b, :n].abs().mean(0).repeat_interleave(3, 0)
        assert ((out[b].double() - want).abs() <= 2 * off * want.abs() + slack + 2.0 ** -25).all()
        assert (lse[b].double() - math.log(n)).abs().max() <= 2.0 ** -20


def test_a_factor_past_fp32_is_refused():
    q, k, v, table, lengths, _ = make([20], (0.5,), 15, torch.float16, E4M3, seed=3)
    with pytest.raises(wsm.WsmError, match="past fp32"):
        wsm.paged_attention(q, k, v, table, lengths, scale=2.0 ** 127, k_scale=4.0)
