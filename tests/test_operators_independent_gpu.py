"""Independent GEMMs (WSM_FLAG_INDEPENDENT, which wait for nothing) behind the decode-step operators: they may be given the
memory that an operator used as scratch, so they start only when it is through with it; and independent GEMMs whose output
the library allocates, in memory that a call before may still read."""
import time

import pytest
import torch

import weight_streaming_megakernel_b200 as wsm

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
IND = wsm.FLAG_INDEPENDENT


@pytest.fixture(autouse=True)
def _clean():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    torch.cuda.set_device(0)
    wsm.operator_status()
    yield
    wsm.debug_stall(0)
    torch.cuda.synchronize()


def normal(*shape, seed=0, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * scale).to(torch.bfloat16).to(DEV)


def test_independent_call_starts_after_the_experts_last_use_of_scratch():
    """CTA 0 of the expert products waits (bounded, on a flag that nothing sets): the independent GEMM queued behind has
    not written by then, and has afterwards."""
    x, w = normal(30, 2048), normal(1, 300, 2048, seed=1)
    off = torch.tensor([0, 30], dtype=torch.int32, device=DEV)
    gx, gw = normal(16, 512, seed=2), normal(1024, 512, seed=3)
    wsm.expert_gemm(x, w, off)
    want = wsm.skinny_gemm(gx, gw, torch.empty(16, 1024, dtype=torch.bfloat16, device=DEV), flags=IND)
    y = torch.full((16, 1024), 3.0, dtype=torch.bfloat16, device=DEV)
    seen = torch.empty(y.shape, dtype=y.dtype, pin_memory=True)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    wsm.debug_stall(1, 1_000_000_000)
    wsm.expert_gemm(x, w, off)
    wsm.skinny_gemm(gx, gw, y, flags=IND)
    time.sleep(0.2)
    with torch.cuda.stream(side):
        seen.copy_(y, non_blocking=True)
    side.synchronize()
    assert (seen == 3.0).all()
    assert wsm.operator_status() == wsm.WSM_ERR_TIMEOUT
    assert torch.equal(y, want)


def operators():
    """Calls whose scratch is in use to their end: experts cut along K, and attention with items to join."""
    x, w = normal(48, 4096, scale=0.1), normal(3, 1024, 4096, seed=1, scale=0.1)
    off = torch.tensor([0, 20, 21, 48], dtype=torch.int32, device=DEV)
    q, kc, vc = normal(4, 32, 128, seed=2), normal(600, 16, 8, 128, seed=3), normal(600, 16, 8, 128, seed=4)
    table = torch.arange(600, dtype=torch.int32, device=DEV).view(4, 150)
    lengths = torch.tensor([2400, 777, 1, 2000], dtype=torch.int32, device=DEV)
    return {"experts": lambda: wsm.expert_gemm(x, w, off), "attention": lambda: wsm.paged_attention(q, kc, vc, table, lengths)}


@pytest.mark.parametrize("op", ["experts", "attention"])
@pytest.mark.parametrize("captured", [False, True])
def test_independent_call_that_writes_the_freed_scratch(op, captured):
    """The GEMM's output is allocated after the operator returned, in the block that was its scratch."""
    call = operators()[op]
    want = call()
    gx, gw = normal(64, 256, seed=5), normal(16400, 256, seed=6)    # an output of 2 MB, as the scratch from the large pool
    y = wsm.skinny_gemm(gx, gw)
    want_y = y.clone()
    del y
    torch.cuda.synchronize()
    torch.cuda.empty_cache()

    def both():
        out = call()
        y = torch.empty(64, 16400, dtype=torch.bfloat16, device=DEV)
        wsm.skinny_gemm(gx, gw, y, flags=IND)
        return out, y

    if captured:
        side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
        with torch.cuda.stream(side):
            wsm.skinny_gemm(gx, gw)                     # (the GEMM's own scratch of this stream)
        torch.cuda.synchronize()
        with torch.cuda.graph(graph, stream=side):
            out, y = both()
        runs = []
        for _ in range(20):
            graph.replay()
            runs.append((out.clone(), y.clone()))
    else:
        runs = [both() for _ in range(20)]
    torch.cuda.synchronize()
    for out, y in runs:
        assert torch.equal(out, want)
        assert (y.float() - want_y.float()).abs().max() <= 2.0 ** -7 * want_y.float().abs().max()
    assert wsm.operator_status() == 0 and wsm.stream_status() == 0


def test_independent_call_that_allocates_its_output_waits():
    """The output's memory is the allocator's choice, so the caller could not promise that no call before reads it: the call
    starts after them.  (The GEMM before it is held by the stall hook; the memory is that of a tensor dropped before.)"""
    x, w = normal(16, 512, seed=2), normal(2048, 512, seed=3)
    want = wsm.skinny_gemm(x, w, torch.empty(16, 2048, dtype=torch.bfloat16, device=DEV), flags=IND)
    first = wsm.skinny_gemm(x, w)
    seen = torch.empty(want.shape, dtype=want.dtype, pin_memory=True)
    side = torch.cuda.Stream()
    pool = torch.cuda.MemPool()
    with torch.cuda.use_mem_pool(pool):                 # (of its own, so that the dropped tensor's block is the one there is)
        old = torch.full_like(want, 3.0)
    at = old.data_ptr()
    torch.cuda.synchronize()
    wsm.debug_stall(1, 1_000_000_000)
    wsm.skinny_gemm(x, w, first)
    del old
    with torch.cuda.use_mem_pool(pool):
        y = wsm.skinny_gemm(x, w, flags=IND)
    assert y.data_ptr() == at
    time.sleep(0.2)
    with torch.cuda.stream(side):
        seen.copy_(y, non_blocking=True)
    side.synchronize()
    assert (seen == 3.0).all()
    assert wsm.stream_status() == wsm.WSM_ERR_TIMEOUT
    assert torch.equal(y, want)


def test_independent_calls_behind_one_that_allocates():
    """They run beside it, and later work still comes after all of them."""
    x, w = normal(16, 512, seed=2), normal(2048, 512, seed=3)
    want = wsm.skinny_gemm(x, w, flags=IND)
    outs = []
    for _ in range(20):
        outs.append(wsm.skinny_gemm(x, w, flags=IND))
        outs += [wsm.skinny_gemm(x, w, torch.empty_like(want), flags=IND) for _ in range(3)]
    total = torch.stack(outs)
    assert (total == want).all()
    assert wsm.stream_status() == 0
