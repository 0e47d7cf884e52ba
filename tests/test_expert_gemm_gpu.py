"""Products grouped by expert against the 64-bit form."""
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
    wsm.debug_stall(0)
    torch.cuda.synchronize()


def make(counts, n, k, dtype=torch.bfloat16, seed=0, lead=0, behind=0):
    g = torch.Generator().manual_seed(seed)
    rows = lead + sum(counts) + behind
    x = torch.randn(rows, k, generator=g).to(dtype)
    w = (torch.randn(len(counts), n, k, generator=g) * k ** -0.5).to(dtype)
    offsets = torch.tensor([lead] + [lead + sum(counts[:i + 1]) for i in range(len(counts))], dtype=torch.int32)
    return x.to(DEV), w.to(DEV), offsets.to(DEV)


def run_and_check(x, w, offsets, silu=False, scaled=False, what=""):
    rows, n = x.shape[0], w.shape[1]
    f = (torch.arange(rows) % 7 * 0.3 - 0.6).to(DEV) if scaled else None
    y = torch.full((rows, n // 2 if silu else n), 3.0, dtype=x.dtype, device=DEV)
    got = wsm.expert_gemm(x, w, offsets, y, epilogue=wsm.EPI_SILU_MUL if silu else wsm.EPI_NONE, row_scale=f)
    torch.cuda.synchronize()
    want = ref.experts(x, w, offsets, silu, f)
    ref.check_experts(got, want, what)
    assert (got.cpu()[torch.isnan(want[0])] == 3.0).all(), f"{what}: rows of no expert"
    assert wsm.operator_status() == 0, what
    return got


@pytest.mark.parametrize("m", [1, 2, 15, 16, 17, 31, 33, 48, 64, 65, 80, 127, 129, 176, 255, 256, 257, 300, 513])
def test_row_counts(m):
    """Every tile height: one expert with m rows beside others with few."""
    run_and_check(*make([3, m, 0, 1], 200, 264, seed=m))


@pytest.mark.parametrize("n", [1, 7, 8, 127, 128, 129, 500])
@pytest.mark.parametrize("k", [8, 56, 64, 72, 128, 200])
def test_outputs_and_depths(n, k):
    run_and_check(*make([5, 0, 40], n, k, seed=n + k), scaled=True)


@pytest.mark.parametrize("n", [16, 112, 128, 144, 544])
def test_silu_mul(n):
    run_and_check(*make([2, 70, 0, 19], n, 328, seed=n), silu=True)
    run_and_check(*make([2, 70, 0, 19], n, 328, torch.float16, seed=n), silu=True, scaled=True)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_cut_along_k(dtype):
    """Few tiles and a long K: every tile is cut into units whose partials are joined."""
    run_and_check(*make([1, 0, 9], 130, 4104, dtype, seed=1), scaled=True)
    run_and_check(*make([100], 256, 6000, dtype, seed=2))
    run_and_check(*make([300, 7], 256, 4096, dtype, seed=3), silu=True)


@pytest.mark.parametrize("m", [64, 65, 80, 127, 129, 176, 240, 241, 255, 256, 257, 300])
def test_row_counts_of_high_tiles(m):
    """Enough tiles for the highest ones: up to 256 rows each."""
    run_and_check(*make([3, m, 0, 1], 6300, 72, seed=m), scaled=m % 2 == 0)
    run_and_check(*make([0, m], 6304, 200, torch.float16, seed=m), silu=True, scaled=m % 2 == 1)


def test_high_tiles_cut_along_k():
    """A tile of up to 256 rows whose units are joined; and one of 128 rows, and of 64."""
    run_and_check(*make([200], 6300, 4104, seed=1), scaled=True)
    run_and_check(*make([5, 100], 3200, 4104, seed=2), silu=True, scaled=True)
    run_and_check(*make([190], 640, 4104, torch.float16, seed=3), silu=True)


@pytest.mark.parametrize("counts", [[0] * 40 + [1], [1] + [0] * 40, [0] * 8, [5] * 33, [0, 700, 0, 0, 3],
                                    [i % 3 for i in range(1024)]])
def test_ragged(counts):
    run_and_check(*make(counts, 136, 128, seed=len(counts)), what=str(counts[:8]))


def test_many_tiles():
    """More tiles than the GPU takes at once, the last ones cut in two."""
    run_and_check(*make([33, 270, 0, 511, 1, 64], 8192, 1088, seed=5))
    run_and_check(*make([33, 270, 0, 511, 1, 64], 8192, 1088, torch.float16, seed=6), silu=True, scaled=True)


def test_rows_outside_all_experts_stay():
    run_and_check(*make([3, 20], 72, 64, lead=5, behind=9))
    run_and_check(*make([0, 0], 72, 64, lead=5, behind=9))


def test_bad_offsets_are_mended_and_recorded():
    x, w, offsets = make([10, 10, 10], 40, 64)
    for bad in ([0, 10, 5, 30], [-4, 10, 20, 30], [0, 10, 20, 10 ** 9], [40, 50, 60, 70], [0, 31, -2 ** 31, 2 ** 31 - 1]):
        o = torch.tensor(bad, dtype=torch.int32, device=DEV)
        y = torch.full((30, 40), 3.0, dtype=x.dtype, device=DEV)
        wsm.expert_gemm(x, w, o, y)
        assert wsm.operator_status() == wsm.WSM_ERR_INVALID, bad
        want = ref.experts(x, w, o, False)
        ref.check_experts(y, want, str(bad))
        assert (y.cpu()[torch.isnan(want[0])] == 3.0).all()


def test_strides():
    """Rows of x and y in wider buffers, w a slice of a larger one."""
    x, w, offsets = make([7, 0, 25], 48, 72, seed=4)
    plain = run_and_check(x, w, offsets)
    wx = torch.full((32, 200), math.nan, dtype=x.dtype, device=DEV)
    wx[:, 64:136] = x
    ww = torch.full((3, 60, 96), math.nan, dtype=w.dtype, device=DEV)
    ww[:, :48, 8:80] = w
    wy = torch.full((32, 61), 9.0, dtype=x.dtype, device=DEV)
    got = wsm.expert_gemm(wx[:, 64:136], ww[:, :48, 8:80], offsets, wy[:, 5:53])
    assert torch.equal(got, plain) and (wy[:, :5] == 9).all() and (wy[:, 53:] == 9).all()


def test_infinities_stay_in_their_rows():
    x, w, offsets = make([20, 20], 40, 72, seed=4)
    plain = run_and_check(x, w, offsets)
    x[19, 3], x[20, 5] = math.inf, math.nan
    got = wsm.expert_gemm(x, w, offsets)
    keep = torch.ones(40, dtype=torch.bool)
    keep[19:21] = False
    assert torch.equal(got[keep.to(DEV)], plain[keep.to(DEV)])
    assert not torch.isfinite(got[19:21]).any()


def test_runs_are_bitwise_alike():
    x, w, offsets = make([1, 60, 3, 0, 130], 384, 2048, seed=9)
    first = wsm.expert_gemm(x, w, offsets)
    for _ in range(20):
        assert torch.equal(wsm.expert_gemm(x, w, offsets), first)


def test_zero_rows():
    x, w, offsets = make([0, 0], 40, 64)
    assert wsm.expert_gemm(x, w, offsets).shape == (0, 40)


def test_graphs_and_streams():
    """Two graphs captured on one stream and replayed together, with other row counts than at capture, beside eager
    calls on a third stream."""
    cases = [list(make(c, 640, 1024, seed=s)) for s, c in enumerate(([3, 40, 0], [20, 0, 23], [1, 1, 41]))]
    want = [wsm.expert_gemm(*c) for c in cases]
    side, graphs, outs = torch.cuda.Stream(), [], []
    moved = [c[2].clone() for c in cases]
    for c, o in zip(cases[:2], moved):
        now = o.clone()
        o.zero_()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            outs.append(wsm.expert_gemm(c[0], c[1], o))
        graphs.append(g)
        o.copy_(now)
    streams = [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    eager = []
    for _ in range(30):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        eager.append(wsm.expert_gemm(*cases[2], stream=streams[2]))
    torch.cuda.synchronize()
    assert torch.equal(outs[0], want[0]) and torch.equal(outs[1], want[1])
    assert all(torch.equal(e, want[2]) for e in eager)


def test_stalled_call_is_reported_and_the_next_is_right():
    """A device-side wait that runs out (on a flag nothing sets) ends the call with an error status."""
    x, w, offsets = make([30, 5], 300, 2048, seed=2)
    want = wsm.expert_gemm(x, w, offsets)
    wsm.debug_stall(1, 20_000_000)
    wsm.expert_gemm(x, w, offsets)
    assert wsm.operator_status() == wsm.WSM_ERR_TIMEOUT
    assert wsm.operator_status() == 0
    assert torch.equal(wsm.expert_gemm(x, w, offsets), want)


def test_agrees_with_skinny_gemm():
    """One expert with up to 64 rows is the decode GEMM."""
    x, w, offsets = make([16], 512, 1024, seed=2)
    a, b = wsm.expert_gemm(x, w, offsets), wsm.skinny_gemm(x, w[0].contiguous())
    want = ref.experts(x, w, offsets, False)
    ref.check_experts(a, want)
    ref.check_experts(b, want)
