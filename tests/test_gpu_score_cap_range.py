"""Caps at the ends of the range that both scoremod calls document (positive, softcap and 1 / softcap
finite), against fp64.  A cap near 0 leaves every visible token the same weight, a huge one leaves the
scores alone.  scoremod_ref's bounds hold: near the ends a score's y = x scale / cap has denormal steps of
2^-149, which the multiplication by the cap makes 2^-22 at most, less than the 2^-19 it grants."""
import numpy as np
import pytest
import torch

import paged_kv_cache_373_b200 as pkv
from scoremod_ref import build, cuda
from test_gpu_decode_scoremod import check as check_decode
from test_gpu_prefill_scoremod import check as check_prefill

pytestmark = pytest.mark.gpu

# (scale, cap): ratios 8e38, 9e36, 1e-9 .. 9e-32, 2e-37, 4.5e-40, 5e-42
ENDS = [(8.0, 1e-38), (0.09, 1e-38), (0.09, 1e8), (0.09, 1e30), (0.02, 1e35), (0.09, 2e38), (1e-3, 2e38)]


@pytest.mark.parametrize("scale,cap", ENDS)
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16], ids=["f16", "bf16"])
@pytest.mark.parametrize("bias", [False, True], ids=["", "bias"])
def test_prefill(scale, cap, dtype, bias):
    ctx, chunks, Hq, Hkv, D = [0, 150], [130, 40], 8, 4, 64
    d = cuda(build([a + b for a, b in zip(ctx, chunks)], Hkv, D, 16, dtype, 71))
    d["q"] = torch.randn(sum(chunks), Hq, D, generator=torch.Generator().manual_seed(72)).to(dtype).cuda()
    d["qs"] = torch.tensor([0] + list(np.cumsum(chunks)), dtype=torch.int32).cuda()
    slopes = torch.linspace(0.02, 0.7, Hq).cuda() if bias else None
    out = torch.empty_like(d["q"])
    pkv.paged_prefill_scoremod(out, d["q"], d["kc"], d["vc"], d["tables"], d["lens"], d["qs"], scale, softcap=cap,
                               alibi_slopes=slopes)
    assert pkv.get_device_error() == 0
    check_prefill(d, out, scale, cap, 0, slopes)


@pytest.mark.parametrize("scale,cap", ENDS)
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16, torch.float32], ids=["f16", "bf16", "f32"])
@pytest.mark.parametrize("bias", [False, True], ids=["", "bias"])
def test_decode(scale, cap, dtype, bias):
    lens, Hq, Hkv, D = [130, 1, 40, 300], 8, 4, 64
    d = cuda(build(lens, Hkv, D, 16, dtype, 73))
    d["q"] = torch.randn(len(lens), Hq, D, generator=torch.Generator().manual_seed(74)).to(dtype).cuda()
    slopes = torch.linspace(0.02, 0.7, Hq).cuda() if bias else None
    out = torch.empty_like(d["q"])
    pkv.paged_attention_decode_scoremod(out, d["q"], d["kc"], d["vc"], d["tables"], d["lens"], scale, softcap=cap,
                                        alibi_slopes=slopes)
    assert pkv.get_device_error() == 0
    check_decode(d, out, scale, cap, 0, slopes)
