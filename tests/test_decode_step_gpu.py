"""The decode-step operators together with the library's GEMMs: one step of a small model with experts, from its qkv
projection to the log probabilities of its answer, each operator's result checked against the 64-bit form of what it
was given; eager, on a stream of its own, and captured in a graph whose lengths, slots and routing move."""
import pytest
import torch

import operators_ref as ref
import oracle
import weight_streaming_megakernel_b200 as wsm
from parity import check_bounded, check_full

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BATCH, HEADS, KV, DIM, PAGE, WIDTH, EXPERTS, INNER, VOCAB, TOP = 6, 8, 2, 64, 16, 512, 5, 256, 5003, 2


@pytest.fixture(autouse=True)
def _clean():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    torch.cuda.set_device(0)
    wsm.operator_status()
    yield
    torch.cuda.synchronize()


class Step:
    """Weights, cache and the buffers of one step, and the step."""

    def __init__(self, seed=0):
        g = torch.Generator().manual_seed(seed)

        def bf(*shape, scale=1.0):
            return (torch.randn(*shape, generator=g) * scale).to(torch.bfloat16).to(DEV)

        self.h = bf(BATCH, WIDTH)
        self.w_qkv = bf((HEADS + 2 * KV) * DIM, WIDTH, scale=WIDTH ** -0.5)
        self.w_o = bf(WIDTH, HEADS * DIM, scale=(HEADS * DIM) ** -0.5)
        self.w_up = bf(EXPERTS, 2 * INNER, WIDTH, scale=WIDTH ** -0.5)
        self.w_down = bf(EXPERTS, WIDTH, INNER, scale=INNER ** -0.5)
        self.w_router = bf(EXPERTS, WIDTH, scale=WIDTH ** -0.5)
        self.w_vocab = bf(VOCAB, WIDTH, scale=3 * WIDTH ** -0.5)
        self.kc, self.vc = bf(40, PAGE, KV, DIM), bf(40, PAGE, KV, DIM)
        # sequence b's pages: b, b + 6, b + 12, ...
        self.table = (torch.arange(6)[None, :] * BATCH + torch.arange(BATCH)[:, None]).int().to(DEV)
        self.lengths = torch.tensor([1, 15, 16, 60, 0, 90], dtype=torch.int32, device=DEV)
        self.tokens = torch.tensor([3, 5000, 17, 400, -1, 2], device=DEV)
        self.logits = torch.empty(BATCH, VOCAB, device=DEV)
        self.y = torch.empty(BATCH, VOCAB, dtype=torch.bfloat16, device=DEV)

    def slots(self):
        last = (self.lengths - 1).clamp(min=0).long()
        at = self.table.long().gather(1, (last // PAGE)[:, None])[:, 0] * PAGE + last % PAGE
        return torch.where(self.lengths > 0, at, -1)

    def run(self):
        s = {}
        s["qkv"] = wsm.skinny_gemm(self.h, self.w_qkv)
        q, k, v = s["qkv"].view(BATCH, HEADS + 2 * KV, DIM).split([HEADS, KV, KV], 1)
        s["slots"] = self.slots()
        wsm.paged_cache_append(k, v, self.kc, self.vc, s["slots"])
        s["lse"] = torch.empty(BATCH, HEADS, device=DEV)
        s["att"] = wsm.paged_attention(q, self.kc, self.vc, self.table, self.lengths, lse=s["lse"])
        s["h1"] = wsm.skinny_gemm(s["att"].view(BATCH, HEADS * DIM), self.w_o, epilogue=wsm.EPI_RESIDUAL, r=self.h)
        # route: the best experts of each token, rows sorted by expert
        weight, chosen = torch.softmax(s["h1"].float() @ self.w_router.float().T, 1).topk(TOP, 1)
        order = chosen.view(-1).sort(stable=True).indices
        s["offsets"] = torch.searchsorted(chosen.view(-1)[order], torch.arange(EXPERTS + 1, device=DEV)).int()
        s["x"] = s["h1"][order // TOP]
        s["scale"] = weight.view(-1)[order].contiguous()
        s["act"] = wsm.expert_gemm(s["x"], self.w_up, s["offsets"], epilogue=wsm.EPI_SILU_MUL)
        s["out"] = wsm.expert_gemm(s["act"], self.w_down, s["offsets"], row_scale=s["scale"])
        s["h2"] = (s["h1"].float().index_add(0, order // TOP, s["out"].float())).to(torch.bfloat16)
        wsm.skinny_gemm(s["h2"], self.w_vocab, self.y, yf32=self.logits)
        s["lp"] = wsm.token_logprobs(self.logits, self.tokens, top=4)
        return s

    def check(self, s, what):
        check_full(self.h, self.w_qkv, s["qkv"], what=what)
        rows = s["qkv"].view(BATCH, HEADS + 2 * KV, DIM)
        for b, at in enumerate(s["slots"].tolist()):
            if at >= 0:
                assert torch.equal(self.kc.view(-1, KV, DIM)[at], rows[b, HEADS:HEADS + KV]), what
                assert torch.equal(self.vc.view(-1, KV, DIM)[at], rows[b, HEADS + KV:]), what
        ref.check_attention(s["att"], s["lse"], ref.attention(rows[:, :HEADS], self.kc, self.vc, self.table, self.lengths, DIM ** -0.5),
                            torch.bfloat16, what)
        want, mag = oracle.gemm_ref(s["att"].view(BATCH, -1).cpu(), self.w_o.cpu())
        check_bounded(s["h1"], None, want + self.h.double().cpu().numpy(), 1e-3 * mag + 1e-6, what)
        ref.check_experts(s["act"], ref.experts(s["x"], self.w_up, s["offsets"], True), what)
        ref.check_experts(s["out"], ref.experts(s["act"], self.w_down, s["offsets"], False, s["scale"]), what)
        check_full(s["h2"], self.w_vocab, self.y, self.logits, what=what)
        ref.check_logprobs(s["lp"], ref.logprobs(self.logits, self.tokens, 4), self.logits, what)
        assert wsm.operator_status() == 0 and wsm.stream_status() == 0, what


def test_step():
    step = Step()
    for i in range(3):
        step.check(step.run(), f"step {i}")
        step.lengths += (step.lengths > 0).int()


def test_step_on_another_stream():
    step, side = Step(1), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        s = step.run()
    side.synchronize()
    step.check(s, "side stream")


def test_step_in_a_graph():
    step, side = Step(2), torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step.run()                                      # (the GEMMs' scratch of this stream)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        s = step.run()
    for i in range(3):
        graph.replay()
        torch.cuda.synchronize()
        step.check(s, f"replay {i}")
        step.lengths += (step.lengths > 0).int()
        step.h.normal_()


FIRST = """
import torch, weight_streaming_megakernel_b200 as wsm
z = lambda *s, dtype=torch.bfloat16: torch.ones(s, dtype=dtype, device="cuda:0")
k, kc, t, n = z(2, 2, 64), z(40, 16, 2, 64), torch.arange(40, dtype=torch.int32, device="cuda:0").view(2, 20), z(2, dtype=torch.int32) * 300
x, w, off, ids = z(6, 128), z(2, 64, 128), torch.tensor([0, 3, 6], dtype=torch.int32, device="cuda:0"), z(2, dtype=torch.int64)
logits = z(2, 70000, dtype=torch.float32)
calls = dict(append=lambda: wsm.paged_cache_append(k, k, kc, kc.clone(), ids), attention=lambda: wsm.paged_attention(k, kc, kc, t, n),
             experts=lambda: wsm.expert_gemm(x, w, off), logprobs=lambda: wsm.token_logprobs(logits, ids, top=3))
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    out = calls["%s"]()
g.replay()
torch.cuda.synchronize()
assert wsm.operator_status() == 0
if "%s" == "attention": assert (out == 1).all()
if "%s" == "experts": assert (out == 128).all()
if "%s" == "logprobs": assert out.top_ids.tolist() == [[0, 1, 2]] * 2
print("captured")
"""


@pytest.mark.parametrize("call", ["append", "attention", "experts", "logprobs"])
def test_first_call_of_a_process_may_be_captured(call):
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    run = subprocess.run([sys.executable, "-c", FIRST.replace("%s", call)], cwd=root, capture_output=True, text=True, timeout=300)
    assert run.returncode == 0 and "captured" in run.stdout, run.stderr[-2000:]
