"""Token log probabilities: more rows than the GPU takes at once, and logits on both sides of the border between the
kernel's two forms of an element's exponent."""
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


def check(x, t, tops, what=""):
    lp, ent, ids, best = ref.logprobs(x, t, max(tops))
    for top in tops:
        got = wsm.token_logprobs(x, t, top=top)
        ref.check_logprobs(got, (lp, ent, ids[:, :top], best[:, :top]), x, f"{what} top {top}")


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("vocab", [9, 1003, 9001])
def test_a_second_wave_of_rows(dtype, vocab):
    """Twice as many rows as the SMs hold blocks (three each), hard ones among them all along."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    rows = 2 * 3 * sms + 1
    g = torch.Generator().manual_seed(vocab)
    x = (torch.randn(rows, vocab, generator=g) * 3).to(dtype).to(DEV)
    t = torch.randint(vocab, (rows,), generator=g).to(DEV)
    x[::50] = 1.0                                       # all alike
    x[1::50] = -math.inf                                # nothing left
    x[2::50, vocab // 3:] = -math.inf
    x[3::50] = torch.arange(vocab, device=DEV).to(dtype)    # rising
    x[4::50, vocab // 2:] = torch.finfo(dtype).min
    x[5::50, vocab // 2] = math.nan
    t[6::50] = -1
    check(x, t, sorted({0, min(3, vocab), min(32, vocab)}))
    assert wsm.operator_status() == 0


@pytest.mark.parametrize("vocab", [2, 5, 64, 1003, 40000, 200003])
@pytest.mark.parametrize("centre", [65536.0, -65536.0])
def test_logits_around_the_border(vocab, centre):
    """Logits spread a little around +-65536, where the largest of some threads lies on one side and of others on the
    other: fp32 holds them to 2^-8 there, and the results are as exact as anywhere else."""
    g = torch.Generator().manual_seed(vocab)
    rows = 24
    x = centre + torch.randn(rows, vocab, generator=g) * torch.tensor([0.01, 0.05, 1.0, 8.0]).repeat(rows // 4)[:, None]
    x[4] = centre
    x[5] = torch.where(torch.arange(vocab) % 2 == 0, torch.tensor(centre + 2.0 ** -7), torch.tensor(centre - 2.0 ** -7))
    x[6, vocab // 2:] = -math.inf
    x[7, vocab // 2:] = 0.0 if centre < 0 else -1.0
    t = torch.randint(vocab, (rows,), generator=g)
    check(x.to(DEV), t.to(DEV), sorted({0, min(5, vocab)}))
