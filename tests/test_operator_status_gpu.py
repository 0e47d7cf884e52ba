"""wsm.operator_status: errors of different kinds do not hide one another, and none is lost to a query."""
import pytest
import torch

import weight_streaming_megakernel_b200 as wsm

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF = torch.bfloat16


def drain():
    """Every error that is there, in the order of the reports."""
    got = []
    while True:
        code = wsm.operator_status()
        if code == 0:
            return got
        got.append((code, wsm.last_error()))
        assert len(got) < 10


@pytest.fixture(autouse=True)
def _clean():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    torch.cuda.set_device(0)
    drain()
    yield
    wsm.debug_stall(0)
    drain()


def bad_slot(row=0, rows=1, stream=None):
    k, cache = torch.ones(rows, 1, 64, dtype=BF, device=DEV), torch.zeros(2, 16, 1, 64, dtype=BF, device=DEV)
    slots = torch.full((rows,), -1, device=DEV)
    slots[row] = 32
    torch.cuda.synchronize()
    wsm.paged_cache_append(k, k, cache, cache.clone(), slots, stream=stream)


def bad_token():
    wsm.token_logprobs(torch.zeros(3, 100, device=DEV), torch.tensor([1, 2, 100], device=DEV))


def bad_offsets():
    wsm.expert_gemm(torch.ones(8, 64, dtype=BF, device=DEV), torch.ones(2, 32, 64, dtype=BF, device=DEV),
                    torch.tensor([0, 9, 8], dtype=torch.int32, device=DEV))


def stalled():
    x, w = torch.ones(8, 64, dtype=BF, device=DEV), torch.ones(2, 32, 64, dtype=BF, device=DEV)
    wsm.debug_stall(1, 20_000_000)
    wsm.expert_gemm(x, w, torch.tensor([0, 4, 8], dtype=torch.int32, device=DEV))


def test_every_kind_is_reported_once():
    bad_token()
    bad_offsets()
    bad_slot(row=5, rows=9)
    got = drain()
    assert [code for code, _ in got] == [wsm.WSM_ERR_INVALID] * 3
    for (_, say), kind, which in zip(got, ("paged cache", "expert products", "log probabilities"), (5, None, 2)):
        assert kind in say and (which is None or f"expert {which}," in say)
    assert drain() == []


@pytest.mark.parametrize("first,then", [(bad_offsets, stalled), (stalled, bad_offsets), (bad_slot, stalled), (stalled, bad_token)])
def test_a_time_out_is_not_hidden(first, then):
    """Neither by an index out of range of the same call's kind, recorded before it, nor by one of another kind."""
    first()
    then()
    assert [code for code, _ in drain()] == [wsm.WSM_ERR_TIMEOUT, wsm.WSM_ERR_INVALID]


def test_the_first_of_a_kind_is_kept():
    bad_slot(row=3, rows=4)
    bad_slot(row=1, rows=4)
    got = drain()
    assert len(got) == 1 and "expert 3," in got[0][1]


def test_queries_beside_another_stream():
    """Calls on another stream that record while this one asks: each is reported by then or afterwards."""
    side = torch.cuda.Stream()
    for i in range(40):
        bad_slot(row=i % 7, rows=8, stream=side)
        now = wsm.operator_status()                     # (waits for the current stream only)
        side.synchronize()
        later = drain()
        assert (now == wsm.WSM_ERR_INVALID) + len(later) == 1
