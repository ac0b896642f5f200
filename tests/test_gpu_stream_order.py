"""What comes right after a decode call on the stream sees the whole output, also where the call's last
grid has nothing of its own to do: no unit is cut, so no merge pass reads a partial result."""
import pytest
import torch

import paged_kv_cache_373_b200 as pkv
from scoremod_ref import build, cuda

pytestmark = pytest.mark.gpu

HQ, HKV, D, BS, SCALE = 16, 8, 128, 16, 0.09

# 16-bit caches: 8 workers per CTA.  (lengths, CTAs): units of one tile, which are never cut, few and
# so many that the CTA-wide merge runs; and as many long units of one length as there are workers,
# so that each takes a whole one and writes late
SHAPES = {"one tile": ([3, 16, 1, 9, 16], 0), "one tile, many": ([1 + i % 16 for i in range(600)], 0),
          "whole long": ([4096] * 15, 15)}


def _inputs(lens, seed=5):
    d = cuda(build(lens, HKV, D, BS, torch.float16, seed))
    q = torch.randn(len(lens), HQ, D, generator=torch.Generator().manual_seed(seed)).to(torch.float16).cuda()
    return d, q


def _follow(call, out):
    """`call` writes `out`; the next node of a captured graph copies it.  Every replay starts from NaN."""
    call()
    torch.cuda.synchronize()
    want, got = out.clone(), torch.empty_like(out)
    assert torch.isfinite(want.float()).all()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out.fill_(float("nan"))
        call()
        got.copy_(out)
    for _ in range(30):
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(got, want)
    for _ in range(30):
        out.fill_(float("nan"))
        call()
        got.copy_(out)
        assert torch.equal(got, want)
    assert pkv.get_device_error() == 0


@pytest.mark.parametrize("name", list(SHAPES))
def test_plain_decode(name):
    lens, ctas = SHAPES[name]
    d, q = _inputs(lens)
    out = torch.empty_like(q)
    ws = torch.empty(pkv.paged_attention_workspace_bytes(len(lens), HQ, HKV, D, ctas), dtype=torch.uint8, device="cuda")
    _follow(lambda: pkv.paged_attention_decode(out, q, d["kc"], d["vc"], d["tables"], d["lens"], SCALE, workspace=ws,
                                               num_ctas=ctas), out)


@pytest.mark.parametrize("name", list(SHAPES))
def test_cascade_without_sharing(name):
    """Groups that share nothing: the suffix pass alone writes `out`, the last pass (finish, or merge and
    combine past 256 sequences) finds nothing to fold."""
    lens, ctas = SHAPES[name]
    S = len(lens)
    d, q = _inputs(lens)
    off = torch.tensor(list(range(0, S, 2)) + [S], dtype=torch.int32, device="cuda")
    mem = torch.arange(S, dtype=torch.int32, device="cuda")
    pre = torch.zeros(len(off) - 1, dtype=torch.int32, device="cuda")
    out, plain = torch.empty_like(q), torch.empty_like(q)

    def call():
        pkv.paged_attention_decode_cascade(out, q, d["kc"], d["vc"], d["tables"], d["lens"], off, mem, pre, 2, SCALE,
                                           num_ctas=ctas)
    _follow(call, out)
    pkv.paged_attention_decode(plain, q, d["kc"], d["vc"], d["tables"], d["lens"], SCALE, num_ctas=ctas)
    assert (out.float() - plain.float()).abs().max() <= 4e-3  # two calls, each within 2e-3 of the exact result


@pytest.mark.parametrize("name", list(SHAPES))
def test_decode_variants(name):
    lens, ctas = SHAPES[name]
    d, q = _inputs(lens)
    out = torch.empty_like(q)
    w = torch.empty(len(lens), HKV, max(lens), device="cuda")
    n = pkv.paged_attention_weights_workspace_bytes(len(lens), HQ, HKV, D, d["tables"].shape[1] * BS, ctas)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    _follow(lambda: pkv.paged_attention_decode_scoremod(out, q, d["kc"], d["vc"], d["tables"], d["lens"], SCALE,
                                                        softcap=20.0, workspace=ws, num_ctas=ctas), out)
    _follow(lambda: pkv.paged_attention_decode_weights(out, w, q, d["kc"], d["vc"], d["tables"], d["lens"], SCALE,
                                                       workspace=ws, num_ctas=ctas), out)
