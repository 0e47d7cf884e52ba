"""The decode-step operators' argument checks, which need no GPU: the C ABI refuses bad arguments before any CUDA
call, the Python calls refuse what is not a CUDA tensor, and the packed structs match include/wsm.h."""
import ctypes
import math
import os
import subprocess
import sys

import pytest
import torch

import operators_ref as ref
import weight_streaming_megakernel_b200 as wsm
from weight_streaming_megakernel_b200 import _build, operators

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module", autouse=True)
def built():
    _build.build()
    yield


def test_packed_structs_match_the_header(tmp_path):
    """Sizes and the last members' offsets, as a C compiler lays the header out."""
    src = tmp_path / "layout.c"
    src.write_text('#include <stdio.h>\n#include "wsm.h"\nint main(void) {\n'
                   'printf("%zu %zu %zu %zu %zu\\n", sizeof(wsm_kv_cache), sizeof(wsm_kv_rows), sizeof(wsm_attention), '
                   'sizeof(wsm_experts), sizeof(wsm_logprobs));\n'
                   'printf("%zu %zu %zu %zu %zu\\n", offsetof(wsm_kv_cache, v_scale), offsetof(wsm_kv_rows, dtype), '
                   'offsetof(wsm_attention, scale), offsetof(wsm_experts, dtype), offsetof(wsm_logprobs, dtype));\n'
                   'return 0;\n}\n')
    exe = tmp_path / "layout"
    subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), "-o", str(exe), str(src)], check=True)
    sizes, lasts = (list(map(int, line.split())) for line in
                    subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.splitlines())
    packs = (operators._CACHE, operators._ROWS, operators._ATTENTION, operators._EXPERTS, operators._LOGPROBS)
    assert [p.size for p in packs] == sizes
    assert [p.size - 4 for p in packs] == lasts


# ------------------------------------------------------------------ C ABI refusals (placeholder addresses, never read)

P = 1 << 20


def cache(**kw):
    a = dict(K=P, V=P, ks=(2 * 16 * 64, 2 * 64, 64), vs=(2 * 16 * 64, 2 * 64, 64), pages=8, page=16, heads=2, dim=64, dtype=0,
             k_scale=1.0, v_scale=1.0)
    a.update(kw)
    return operators._CACHE.pack(a["K"], a["V"], *a["ks"], *a["vs"], a["pages"], a["page"], a["heads"], a["dim"], a["dtype"],
                                 a["k_scale"], a["v_scale"])


def rows(**kw):
    a = dict(k=P, v=P, ks=(128, 64), vs=(128, 64), slots=P, tokens=5, dtype=0)
    a.update(kw)
    return operators._ROWS.pack(a["k"], a["v"], *a["ks"], *a["vs"], a["slots"], a["tokens"], a["dtype"])


def attention(**kw):
    a = dict(Q=P, O=P, lse=0, table=P, lengths=P, qs=(256, 64), os=(256, 64), ts=8, ws=P, wsb=1 << 30, batch=2, heads=4, pages=64,
             window=0, dtype=0, scale=0.125)
    a.update(kw)
    return operators._ATTENTION.pack(a["Q"], a["O"], a["lse"], a["table"], a["lengths"], *a["qs"], *a["os"], a["ts"], a["ws"],
                                     a["wsb"], a["batch"], a["heads"], a["pages"], a["window"], a["dtype"], a["scale"])


def experts(**kw):
    a = dict(X=P, W=P, Y=P, offsets=P, scale=0, xs=64, we=64 * 32, wr=64, ys=32, ws=P, wsb=1 << 40, rows=4, experts=3, N=32, K=64,
             epi=0, dtype=0)
    a.update(kw)
    return operators._EXPERTS.pack(a["X"], a["W"], a["Y"], a["offsets"], a["scale"], a["xs"], a["we"], a["wr"], a["ys"], a["ws"],
                                   a["wsb"], a["rows"], a["experts"], a["N"], a["K"], a["epi"], a["dtype"])


def logprobs(**kw):
    a = dict(x=P, tokens=P, lp=P, ent=P, ids=P, best=P, stride=100, rows=3, vocab=100, top=2, dtype=2)
    a.update(kw)
    return operators._LOGPROBS.pack(a["x"], a["tokens"], a["lp"], a["ent"], a["ids"], a["best"], a["stride"], a["rows"],
                                    a["vocab"], a["top"], a["dtype"])


INVALID, UNSUPPORTED, ALIGN = wsm.WSM_ERR_INVALID, wsm.WSM_ERR_UNSUPPORTED, wsm.WSM_ERR_ALIGN


@pytest.mark.parametrize("kw,code", [
    (dict(K=0), INVALID), (dict(V=0), INVALID), (dict(pages=0), INVALID), (dict(page=0), INVALID), (dict(heads=0), INVALID),
    (dict(dim=0), INVALID), (dict(dtype=2), UNSUPPORTED), (dict(dtype=9), UNSUPPORTED), (dict(pages=1 << 31), UNSUPPORTED),
    (dict(dim=60), UNSUPPORTED), (dict(dim=72, dtype=3), UNSUPPORTED), (dict(K=P + 8), ALIGN),
    (dict(ks=(2048, 130, 64)), ALIGN), (dict(vs=(-2048, 128, 64)), ALIGN), (dict(k_scale=0.0, dtype=3), INVALID),
    (dict(v_scale=math.inf, dtype=3), INVALID), (dict(k_scale=math.nan, dtype=3), INVALID), (dict(k_scale=2.0), INVALID),
])
def test_cache_refusals(kw, code):
    assert wsm.lib().wsm_paged_cache_append(cache(**kw), rows(), None) == code and wsm.last_error()
    assert wsm.lib().wsm_paged_attention(cache(**kw), attention(), None) == code


@pytest.mark.parametrize("kw,code", [
    (dict(tokens=-1), INVALID), (dict(dtype=2), UNSUPPORTED), (dict(dtype=1), INVALID), (dict(k=0), INVALID), (dict(v=0), INVALID),
    (dict(slots=0), INVALID), (dict(k=P + 2), ALIGN), (dict(slots=P + 4), ALIGN), (dict(ks=(129, 64)), ALIGN),
    (dict(vs=(128, -64)), ALIGN),
])
def test_append_refusals(kw, code):
    assert wsm.lib().wsm_paged_cache_append(cache(), rows(**kw), None) == code and wsm.last_error()


def test_append_null_zero_and_overlap():
    L = wsm.lib()
    assert L.wsm_paged_cache_append(None, rows(), None) == INVALID
    assert L.wsm_paged_cache_append(cache(), None, None) == INVALID
    assert L.wsm_paged_cache_append(cache(), rows(tokens=0, k=0, v=0, slots=0), None) == wsm.WSM_OK
    assert L.wsm_paged_cache_append(cache(ks=(2048, 128, 0)), rows(), None) == INVALID   # heads on top of one another


@pytest.mark.parametrize("kw,code", [
    (dict(batch=-1), INVALID), (dict(heads=0), INVALID), (dict(pages=-1), INVALID), (dict(window=-1), INVALID),
    (dict(dtype=2), UNSUPPORTED), (dict(dtype=1), INVALID), (dict(heads=5), INVALID), (dict(batch=4097), UNSUPPORTED),
    (dict(pages=1 << 28), UNSUPPORTED), (dict(scale=math.inf), INVALID), (dict(scale=math.nan), INVALID), (dict(Q=0), INVALID),
    (dict(O=0), INVALID), (dict(lengths=0), INVALID), (dict(table=0), INVALID), (dict(ws=0), INVALID), (dict(Q=P + 8), ALIGN),
    (dict(O=P + 4), ALIGN), (dict(ws=P + 8), ALIGN), (dict(lse=P + 2), ALIGN), (dict(table=P + 2), ALIGN),
    (dict(qs=(260, 64)), ALIGN), (dict(os=(256, -64)), ALIGN), (dict(os=(0, 64)), INVALID), (dict(os=(256, 0)), INVALID),
    (dict(ts=-1), INVALID),
])
def test_attention_refusals(kw, code):
    assert wsm.lib().wsm_paged_attention(cache(), attention(**kw), None) == code and wsm.last_error()


def test_attention_dims_null_and_zero():
    L = wsm.lib()
    for dim in (16, 32, 80, 112, 512):
        c = cache(dim=dim, ks=(32 * dim, 2 * dim, dim), vs=(32 * dim, 2 * dim, dim))
        assert L.wsm_paged_attention(c, attention(), None) == UNSUPPORTED
        assert L.wsm_paged_attention_workspace(1, dim, 0, 1000, 0, ctypes.byref(ctypes.c_size_t())) == UNSUPPORTED
    assert L.wsm_paged_attention(cache(), None, None) == INVALID
    assert L.wsm_paged_attention(cache(), attention(batch=0, Q=0, O=0, lengths=0, table=0, ws=0), None) == wsm.WSM_OK
    n = ctypes.c_size_t(7)
    assert L.wsm_paged_attention_workspace(4097, 64, 0, 1000, 0, ctypes.byref(n)) == UNSUPPORTED
    for bad in ((-1, 64, 0, 1000, 0), (1, 64, 0, -1, 0), (1, 64, 0, 1000, -1)):
        assert L.wsm_paged_attention_workspace(*bad, ctypes.byref(n)) == INVALID
    assert L.wsm_paged_attention_workspace(1, 64, 0, 1000, 0, None) == INVALID
    # sequences that are never cut need none
    assert L.wsm_paged_attention_workspace(9, 64, 0, 128, 0, ctypes.byref(n)) == wsm.WSM_OK and n.value == 0
    assert L.wsm_paged_attention_workspace(9, 64, 0, 10 ** 6, 100, ctypes.byref(n)) == wsm.WSM_OK and n.value == 0


@pytest.mark.parametrize("kw,code", [
    (dict(rows=-1), INVALID), (dict(experts=0), INVALID), (dict(N=0), INVALID), (dict(experts=1025), UNSUPPORTED),
    (dict(K=0), UNSUPPORTED), (dict(K=60), UNSUPPORTED), (dict(dtype=2), UNSUPPORTED), (dict(dtype=3), UNSUPPORTED),
    (dict(epi=2), UNSUPPORTED), (dict(epi=7), UNSUPPORTED), (dict(epi=1, N=24), UNSUPPORTED), (dict(X=0), INVALID),
    (dict(W=0), INVALID), (dict(Y=0), INVALID), (dict(offsets=0), INVALID), (dict(ws=0), INVALID), (dict(X=P + 8), ALIGN),
    (dict(W=P + 2), ALIGN), (dict(ws=P + 4), ALIGN), (dict(Y=P + 1), ALIGN), (dict(offsets=P + 2), ALIGN),
    (dict(scale=P + 2), ALIGN), (dict(xs=68), ALIGN), (dict(wr=68), ALIGN), (dict(we=64 * 32 + 4), ALIGN), (dict(xs=56), INVALID),
    (dict(wr=0), INVALID), (dict(we=0), INVALID), (dict(ys=31), INVALID), (dict(ys=-32), INVALID),
    (dict(xs=1 << 40), UNSUPPORTED), (dict(N=2 ** 31 - 1, rows=2 ** 31 - 1, we=1 << 37, ys=1 << 33), UNSUPPORTED),
])
def test_expert_refusals(kw, code):
    assert wsm.lib().wsm_expert_gemm(experts(**kw), None) == code and wsm.last_error()


def test_expert_null_and_zero():
    L = wsm.lib()
    assert L.wsm_expert_gemm(None, None) == INVALID
    assert L.wsm_expert_gemm(experts(rows=0, X=0, W=0, Y=0, offsets=0, ws=0), None) == wsm.WSM_OK
    assert L.wsm_expert_gemm_workspace_bytes(-1, 1) == 0 and L.wsm_expert_gemm_workspace_bytes(1, 1025) == 0


@pytest.mark.parametrize("kw,code", [
    (dict(rows=-1), INVALID), (dict(vocab=0), INVALID), (dict(top=-1), UNSUPPORTED), (dict(top=33), UNSUPPORTED),
    (dict(vocab=1, top=2), UNSUPPORTED), (dict(vocab=(1 << 30) + 1), UNSUPPORTED), (dict(dtype=3), UNSUPPORTED),
    (dict(stride=-1), INVALID), (dict(x=0), INVALID), (dict(ids=0), INVALID), (dict(best=0), INVALID),
    (dict(lp=0, ent=0, top=0), INVALID), (dict(x=P + 2), ALIGN), (dict(tokens=P + 4), ALIGN), (dict(ids=P + 4), ALIGN),
    (dict(lp=P + 2), ALIGN), (dict(ent=P + 2), ALIGN), (dict(best=P + 2), ALIGN),
])
def test_logprobs_refusals(kw, code):
    assert wsm.lib().wsm_token_logprobs(logprobs(**kw), None) == code and wsm.last_error()


def test_logprobs_null_and_zero():
    assert wsm.lib().wsm_token_logprobs(None, None) == INVALID
    assert wsm.lib().wsm_token_logprobs(logprobs(rows=0, x=0, ids=0, best=0), None) == wsm.WSM_OK


# ------------------------------------------------------------------ Python refusals

def test_python_calls_refuse_what_is_no_cuda_tensor():
    q = torch.zeros(2, 4, 64, dtype=torch.bfloat16)
    c = torch.zeros(3, 16, 2, 64, dtype=torch.bfloat16)
    i = torch.zeros(2, 3, dtype=torch.int32)
    for call in (lambda: wsm.paged_attention(q, c, c, i, i[:, 0]),
                 lambda: wsm.paged_cache_append(q, q, c, c, torch.zeros(2, dtype=torch.int64)),
                 lambda: wsm.expert_gemm(q[0], q, i[0]),
                 lambda: wsm.token_logprobs(q[0])):
        with pytest.raises(ValueError, match="CUDA"):
            call()
    for call in (lambda: wsm.token_logprobs([[1.0]]), lambda: wsm.paged_cache_append(None, q, c, c, i),
                 lambda: wsm.paged_attention(None, c, c, i, i), lambda: wsm.expert_gemm(None, q, i)):
        with pytest.raises(TypeError, match="torch tensor"):
            call()


# ------------------------------------------------------------------ the oracle itself

def test_reference_forms_against_closed_ones():
    """Uniform attention is a mean; one-hot logits have no entropy; an identity expert copies its rows."""
    q = torch.zeros(1, 2, 4)
    k = torch.randn(2, 4, 1, 4)
    out, lse, _, _ = ref.attention(q, k, k, torch.tensor([[1, 0]]), torch.tensor([6]), 1.0)
    v = torch.cat([k[1, :, 0], k[0, :2, 0]]).double()
    assert torch.allclose(out[0], v.mean(0).expand(2, 4)) and torch.allclose(lse, torch.full((1, 2), math.log(6.0), dtype=torch.float64))
    lp, ent, ids, best = ref.logprobs(torch.tensor([[0.0, 0.0, -math.inf, 0.0]]), torch.tensor([3]), 4)
    assert math.isclose(lp[0], -math.log(3)) and math.isclose(ent[0], math.log(3)) and ids.tolist() == [[0, 1, 3, -1]]
    x = torch.randn(5, 8)
    y, _ = ref.experts(x, torch.eye(8).expand(2, 8, 8), torch.tensor([1, 3, 4]), False)
    assert torch.equal(y[1:4], x[1:4].double()) and torch.isnan(y[[0, 4]]).all()
