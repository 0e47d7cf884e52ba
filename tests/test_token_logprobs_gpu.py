"""Token log probabilities, entropies and alternatives against the 64-bit form."""
import math

import pytest
import torch

import operators_ref as ref
import weight_streaming_megakernel_b200 as wsm

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(autouse=True)
def _clean():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    torch.cuda.set_device(0)
    wsm.operator_status()
    yield
    torch.cuda.synchronize()


def make(rows, vocab, dtype=torch.float32, seed=0, spread=3.0):
    g = torch.Generator().manual_seed(seed)
    x = (torch.randn(rows, vocab, generator=g) * spread).to(dtype)
    return x.to(DEV), torch.randint(vocab, (rows,), generator=g).to(DEV)


def run_and_check(x, t, top, what=""):
    got = wsm.token_logprobs(x, t, top=top)
    torch.cuda.synchronize()
    ref.check_logprobs(got, ref.logprobs(x, t, top), x, what)
    return got


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("vocab", [1, 2, 3, 7, 8, 9, 31, 100, 1000, 1023, 4097, 33333])
def test_vocabularies(dtype, vocab):
    x, t = make(5, vocab, dtype, seed=vocab)
    for top in sorted({0, 1, min(5, vocab), min(32, vocab)}):
        run_and_check(x, t, top, f"top {top}")
    assert wsm.operator_status() == 0


@pytest.mark.parametrize("rows", [1, 3, 40, 100, 200, 700])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_rows(rows, dtype):
    """From a cluster of blocks to a row, to one block to each."""
    run_and_check(*make(rows, 20011, dtype, seed=rows), top=10)


def test_wide_rows():
    run_and_check(*make(2, 200003, seed=1), top=32)
    run_and_check(*make(2, 1_000_003, torch.bfloat16, seed=2), top=20)


def test_ties_go_to_the_lower_index():
    x, t = make(6, 5000, torch.bfloat16, seed=3, spread=0.5)
    x[0] = 1.0                                          # all alike
    x[1] = (torch.arange(5000) % 3).to(x.dtype)
    x[2] = -torch.arange(5000).div(1000).floor().to(x.dtype)
    x[3, ::2], x[3, 1::2] = 0.0, -0.0                   # equal values of two signs
    x[4] = torch.arange(5000).to(x.dtype)               # rising: every element enters the list
    run_and_check(x, t, 32)
    run_and_check(x.float(), t, 7)


def test_adversarial_orders():
    n = 30000
    base = torch.linspace(-30, 30, n)
    x = torch.stack([base, base.flip(0), base.roll(n // 2), torch.cat([base[::2], base[1::2]])]).to(DEV)
    run_and_check(x, torch.tensor([0, 1, n - 1, n // 2], device=DEV), 32)


def test_masked_rows():
    x, t = make(9, 3000, seed=4)
    x[0] = -math.inf                                    # nothing left
    x[1, :] = -math.inf
    x[1, 1234] = 2.5                                    # one left
    t[1] = 1234
    x[2, 100:] = -math.inf
    t[2] = 2000                                         # a masked token
    x[3, :2990] = -math.inf
    x[4, ::2] = -math.inf
    x[5] = torch.finfo(torch.float32).min               # the type's lowest value is not -infinity
    x[6, 10:] = torch.finfo(torch.float32).min
    x[7] *= 1e30
    x[8] = x[8] * 1e-30 + 5e4
    run_and_check(x, t, 12)
    y = x[:5].to(torch.bfloat16)
    run_and_check(y, t[:5], 12)


def test_large_offsets_and_certain_tokens():
    """Rows far from zero, and rows whose one token has all but the last bits of the probability."""
    x, t = make(4, 2000, seed=4)
    x[0] += 1000
    x[1] -= 1000
    x[2, 77] = 60.0
    t[2] = 77
    x[3, 5] = 300.0
    t[3] = 6
    run_and_check(x, t, 5)


def test_nan_and_infinity():
    x, t = make(5, 900, seed=5)
    x[0, 17] = math.nan
    x[1, 800] = math.inf
    x[2] = math.nan
    x[3, 3], x[3, 4] = math.inf, -math.inf
    t[2] = -1
    run_and_check(x, t, 6)


def test_padding_and_bad_tokens():
    x, t = make(4, 500, seed=6)
    t[1] = -100
    got = run_and_check(x, t, 3)
    assert got.logprob[1] == 0 and wsm.operator_status() == 0
    t[2] = 500
    run_and_check(x, t, 3)
    assert wsm.operator_status() == wsm.WSM_ERR_INVALID and wsm.operator_status() == 0
    t[2] = 2 ** 62
    run_and_check(x, t, 0)
    assert wsm.operator_status() == wsm.WSM_ERR_INVALID
    got = wsm.token_logprobs(x, top=2)
    assert not got.logprob.any()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("vocab", [9, 1003, 9001])
def test_many_rows(dtype, vocab):
    """More rows than the GPU takes at once, hard ones among them."""
    x, t = make(400, vocab, dtype, seed=vocab)
    x[::50] = 1.0                                       # all alike
    x[1::50] = -math.inf                                # nothing left
    x[2::50, vocab // 3:] = -math.inf
    x[3::50] = torch.arange(vocab).to(dtype)            # rising
    x[4::50, vocab // 2:] = torch.finfo(dtype).min
    x[5::50, vocab // 2] = math.nan
    t[6::50] = -1
    for top in sorted({0, min(3, vocab), min(32, vocab)}):
        run_and_check(x, t, top, f"top {top}")
    wide = torch.full((400, vocab + 5), math.nan, dtype=dtype, device=DEV)
    wide[:, 3:3 + vocab] = x
    run_and_check(wide[:, 3:3 + vocab], t, min(3, vocab), "a wider buffer")


def test_strides_and_alignment():
    """Rows of a wider buffer, at every distance from a 16-byte boundary."""
    for dtype in (torch.float32, torch.bfloat16):
        x, t = make(6, 1003, dtype, seed=7)
        for at in range(9):
            wide = torch.full((6, 1021), math.nan, dtype=dtype, device=DEV)
            wide[:, at:at + 1003] = x
            run_and_check(wide[:, at:at + 1003], t, 4, f"at {at}")
        run_and_check(x[:1].expand(6, 1003), t, 4, "one row six times")


def test_no_rows():
    x, t = make(3, 50)
    got = wsm.token_logprobs(x[:0], t[:0], top=3)
    assert got.logprob.shape == (0,) and got.top_ids.shape == (0, 3)


def test_offsets_past_32_bits():
    buf = torch.empty((1 << 31) + 70000, dtype=torch.bfloat16, device=DEV)
    x, t = make(2, 60000, torch.bfloat16, seed=8)
    far = buf.as_strided((2, 60000), ((1 << 31) + 1001, 1))
    far.copy_(x)
    run_and_check(far, t, 5)


def test_skinny_gemm_logits_graph_and_streams():
    """The vocabulary projection's fp32 result straight into the operator, captured; replays beside another stream."""
    g0 = torch.Generator().manual_seed(1)
    h = torch.randn(4, 512, generator=g0).to(torch.bfloat16).to(DEV)
    w = (torch.randn(10000, 512, generator=g0) * 0.2).to(torch.bfloat16).to(DEV)
    t = torch.tensor([1, 22, 333, 4444], device=DEV)
    y, yf = torch.empty(4, 10000, dtype=torch.bfloat16, device=DEV), torch.empty(4, 10000, device=DEV)
    wsm.skinny_gemm(h, w, y, yf32=yf)
    want = run_and_check(yf, t, 8)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        wsm.skinny_gemm(h, w, y, yf32=yf)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        wsm.skinny_gemm(h, w, y, yf32=yf)
        got = wsm.token_logprobs(yf, t, top=8)
    other = torch.cuda.Stream()
    x2, t2 = make(300, 5000, seed=9)
    torch.cuda.synchronize()
    want2 = wsm.token_logprobs(x2, t2, top=8)
    torch.cuda.synchronize()
    for _ in range(20):
        yf.zero_()
        torch.cuda.synchronize()
        graph.replay()
        got2 = wsm.token_logprobs(x2, t2, top=8, stream=other)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        assert all(torch.equal(a, b) for a, b in zip(got2, want2))
