"""What the Python calls of the decode-step operators say to tensors that do not fit, and calls on given streams."""
import pytest
import torch

import weight_streaming_megakernel_b200 as wsm

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, I32, I64 = torch.bfloat16, torch.int32, torch.int64


@pytest.fixture(autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    torch.cuda.set_device(0)


def zeros(*shape, dtype=BF, device=DEV):
    return torch.zeros(shape, dtype=dtype, device=device)


def append(**kw):
    a = dict(k=zeros(3, 2, 64), v=zeros(3, 2, 64), k_cache=zeros(4, 16, 2, 64), v_cache=zeros(4, 16, 2, 64), slots=zeros(3, dtype=I64))
    a.update(kw)
    return wsm.paged_cache_append(**a)


def attend(**kw):
    a = dict(q=zeros(3, 4, 64), k_cache=zeros(4, 16, 2, 64), v_cache=zeros(4, 16, 2, 64), block_table=zeros(3, 2, dtype=I32),
             lengths=zeros(3, dtype=I32))
    a.update(kw)
    return wsm.paged_attention(**a)


def experts(**kw):
    a = dict(x=zeros(5, 64), w=zeros(2, 32, 64), offsets=zeros(3, dtype=I32))
    a.update(kw)
    return wsm.expert_gemm(**a)


def logprobs(**kw):
    a = dict(logits=zeros(5, 64), tokens=zeros(5, dtype=I64))
    a.update(kw)
    return wsm.token_logprobs(**a)


@pytest.mark.parametrize("call,kw,error,say", [
    (append, lambda: dict(v=zeros(3, 2, 64, device="cpu")), ValueError, "v must be a CUDA tensor"),
    (append, lambda: dict(k=zeros(3, 2, 64, dtype=torch.float32)), TypeError, "k must be"),
    (append, lambda: dict(v=zeros(3, 2, 64, dtype=torch.float16)), TypeError, "v must be"),
    (append, lambda: dict(v=zeros(3, 2, 32)), ValueError, "v must be"),
    (append, lambda: dict(k_cache=zeros(4, 16, 2, 64, dtype=torch.float16)), TypeError, "k_cache must be"),
    (append, lambda: dict(v_cache=zeros(4, 16, 2, 64, dtype=torch.float8_e4m3fn)), TypeError, "v_cache must be"),
    (append, lambda: dict(v_cache=zeros(5, 16, 2, 64)), ValueError, "v_cache must be"),
    (append, lambda: dict(k_cache=zeros(4, 16, 3, 64), v_cache=zeros(4, 16, 3, 64)), ValueError, "k_cache must be"),
    (append, lambda: dict(slots=zeros(4, dtype=I64)), ValueError, "slots must be"),
    (append, lambda: dict(slots=zeros(3, dtype=I32)), TypeError, "slots must be"),
    (append, lambda: dict(slots=zeros(6, dtype=I64)[::2]), ValueError, "slots must be contiguous"),
    (append, lambda: dict(k=zeros(3, 2, 128)[..., ::2]), ValueError, "k must be contiguous in its last dimension"),
    (append, lambda: dict(k=zeros(3, 2, 68)[..., 4:]), wsm.WsmError, "ALIGN"),
    (append, lambda: dict(k_scale=2.0), wsm.WsmError, "scales of 1"),
    (append, lambda: dict(slots=None), TypeError, "slots must be a torch tensor"),
    (attend, lambda: dict(q=zeros(3, 4, 64, dtype=torch.float32)), TypeError, "q must be"),
    (attend, lambda: dict(q=zeros(3, 4, 128)), ValueError, "k_cache must be"),
    (attend, lambda: dict(q=zeros(4, 64)), ValueError, "q must be"),
    (attend, lambda: dict(q=zeros(3, 5, 64)), wsm.WsmError, "not a multiple"),
    (attend, lambda: dict(block_table=zeros(4, 2, dtype=I32)), ValueError, "block_table must be"),
    (attend, lambda: dict(block_table=zeros(3, 2, dtype=I64)), TypeError, "block_table must be"),
    (attend, lambda: dict(block_table=zeros(2, 3, dtype=I32).T), ValueError, "block_table must be contiguous in its last"),
    (attend, lambda: dict(lengths=zeros(2, dtype=I32)), ValueError, "lengths must be"),
    (attend, lambda: dict(lengths=zeros(3, dtype=I32, device="cpu")), ValueError, "lengths must be a CUDA"),
    (attend, lambda: dict(out=zeros(3, 4, 32)), ValueError, "out must be"),
    (attend, lambda: dict(out=zeros(3, 4, 64, dtype=torch.float16)), TypeError, "out must be"),
    (attend, lambda: dict(lse=zeros(3, 4)), TypeError, "lse must be"),
    (attend, lambda: dict(lse=zeros(4, 3, dtype=torch.float32)), ValueError, "lse must be"),
    (attend, lambda: dict(lse=zeros(3, 8, dtype=torch.float32)[:, ::2]), ValueError, "lse must be contiguous"),
    (attend, lambda: dict(window=-1), wsm.WsmError, "negative"),
    (attend, lambda: dict(out=zeros(3, 1, 64).expand(3, 4, 64)), wsm.WsmError, "overlap"),
    (experts, lambda: dict(w=zeros(2, 32, 72)), ValueError, "w must be"),
    (experts, lambda: dict(w=zeros(2, 32, 64, dtype=torch.float16)), TypeError, "w must be"),
    (experts, lambda: dict(offsets=zeros(2, dtype=I32)), ValueError, "offsets must be"),
    (experts, lambda: dict(offsets=zeros(3, dtype=I64)), TypeError, "offsets must be"),
    (experts, lambda: dict(y=zeros(5, 16)), ValueError, "y must be"),
    (experts, lambda: dict(row_scale=zeros(5)), TypeError, "row_scale must be"),
    (experts, lambda: dict(row_scale=zeros(4, dtype=torch.float32)), ValueError, "row_scale must be"),
    (experts, lambda: dict(epilogue=2), wsm.WsmError, "epilogue"),
    (experts, lambda: dict(w=zeros(2, 24, 64), epilogue=1), wsm.WsmError, "multiple of 16"),
    (experts, lambda: dict(x=zeros(5, 60), w=zeros(2, 32, 60)), wsm.WsmError, "K=60"),
    (experts, lambda: dict(y=zeros(1, 32).expand(5, 32)), wsm.WsmError, "overlap"),
    (logprobs, lambda: dict(logits=zeros(5, 64, dtype=torch.float64)), TypeError, "logits must be"),
    (logprobs, lambda: dict(tokens=zeros(5, dtype=I32)), TypeError, "tokens must be"),
    (logprobs, lambda: dict(tokens=zeros(4, dtype=I64)), ValueError, "tokens must be"),
    (logprobs, lambda: dict(logits=zeros(64, 5).T), ValueError, "contiguous in its last"),
    (logprobs, lambda: dict(top=33), wsm.WsmError, "top 33"),
    (logprobs, lambda: dict(top=-1), wsm.WsmError, "top -1"),
])
def test_refusals(call, kw, error, say):
    with pytest.raises(error, match=say):
        call(**kw())


def test_given_streams():
    """A torch stream, a raw handle; outputs belong to the stream's allocations."""
    side = torch.cuda.Stream()
    x, w, off = torch.randn(5, 64, device=DEV).to(BF), torch.randn(2, 32, 64, device=DEV).to(BF), torch.tensor([0, 2, 5], dtype=I32, device=DEV)
    torch.cuda.synchronize()
    want = wsm.expert_gemm(x, w, off)
    got = [wsm.expert_gemm(x, w, off, stream=side), wsm.expert_gemm(x, w, off, stream=side.cuda_stream)]
    side.synchronize()
    assert all(torch.equal(g, want) for g in got)
