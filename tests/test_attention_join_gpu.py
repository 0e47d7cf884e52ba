"""Where paged attention's second kernel finds the items that were cut: many sequences, and lengths that the call before
has just written."""
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


def make(batch, most, heads, kv_heads, dim, seed, dtype=torch.bfloat16, page=16, pages=96):
    g = torch.Generator().manual_seed(seed)
    k, v = (torch.randn(pages, page, kv_heads, dim, generator=g).to(dtype).to(DEV) for _ in range(2))
    q = torch.randn(batch, heads, dim, generator=g).to(dtype).to(DEV)
    table = torch.randint(pages, (batch, -(-most // page)), generator=g, dtype=torch.int32).to(DEV)     # (shared pages)
    return q, k, v, table


@pytest.mark.parametrize("batch", [600, 4096])
@pytest.mark.parametrize("window", [0, 333])
def test_many_sequences_some_of_them_cut(batch, window):
    """Long sequences among short and idle ones, up to the largest batch; all of the long ones are checked, and some of the
    short ones."""
    q, k, v, table = make(batch, 2600, 2, 1, 64, seed=batch)
    lengths = torch.tensor([(i * 7) % 23 for i in range(batch)], dtype=torch.int32)
    long = list(range(3, batch, batch // 12)) + [0, batch - 1]
    for j, b in enumerate(long):
        lengths[b] = 140 + 173 * j
    lse = torch.zeros(batch, 2, device=DEV)
    out = wsm.paged_attention(q, k, v, table, lengths.to(DEV), window=window, lse=lse)
    some = torch.tensor(sorted(set(long + list(range(0, batch, 97)))), device=DEV)
    want = ref.attention(q[some], k, v, table[some], lengths.to(DEV)[some], 0.125, window)
    ref.check_attention(out[some], lse[some], want, q.dtype, "some")
    assert not out[(lengths == 0).to(DEV)].any() and wsm.operator_status() == 0


@pytest.mark.parametrize("captured", [False, True])
def test_lengths_written_just_before(captured):
    """Each call's lengths are written by the kernel before it, and moved again by the one behind it."""
    q, k, v, table = make(40, 3000, 8, 2, 128, seed=1)
    sets = [torch.tensor([(i * s) % 3000 for i in range(40)], dtype=torch.int32, device=DEV) for s in (71, 997, 1, 2048)]
    want = [wsm.paged_attention(q, k, v, table, n) for n in sets]
    lengths = torch.zeros(40, dtype=torch.int32, device=DEV)

    def steps():
        out = []
        for n in sets:
            lengths.copy_(n)
            out.append(wsm.paged_attention(q, k, v, table, lengths))
        lengths.zero_()
        return out

    if captured:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = steps()
        for _ in range(20):
            graph.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(out, want))
    else:
        for _ in range(20):
            assert all(torch.equal(a, b) for a, b in zip(steps(), want))
