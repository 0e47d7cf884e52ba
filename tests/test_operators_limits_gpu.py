"""Sizes of the decode-step operators' Python calls beyond any sequence or list: taken for what they mean, or refused
before anything is allocated for them."""
import pytest
import torch

import weight_streaming_megakernel_b200 as wsm

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    torch.cuda.set_device(0)


@pytest.mark.parametrize("window", [5000, 2 ** 31 - 1, 2 ** 31, 2 ** 32, 2 ** 32 + 1, 2 ** 63 - 1])
def test_a_window_past_every_sequence_is_none(window):
    g = torch.Generator().manual_seed(0)
    q, k, v = (torch.randn(*s, generator=g).to(torch.bfloat16).to(DEV) for s in ((2, 4, 64), (30, 16, 2, 64), (30, 16, 2, 64)))
    table = torch.arange(30, dtype=torch.int32, device=DEV).view(2, 15)
    lengths = torch.tensor([240, 33], dtype=torch.int32, device=DEV)
    assert torch.equal(wsm.paged_attention(q, k, v, table, lengths, window=window), wsm.paged_attention(q, k, v, table, lengths))


@pytest.mark.parametrize("top", [33, 10 ** 9, 2 ** 31, 2 ** 40, -2 ** 31])
def test_too_many_alternatives_are_refused(top):
    held = torch.zeros(1000, 64, device=DEV)
    before = torch.cuda.max_memory_allocated()
    with pytest.raises(wsm.WsmError, match="alternatives"):
        wsm.token_logprobs(held, top=top)
    assert torch.cuda.max_memory_allocated() - before < 1 << 20
    with pytest.raises(wsm.WsmError, match="no more than the vocabulary of 5"):
        wsm.token_logprobs(held[:, :5], top=6)
