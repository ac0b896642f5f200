"""The output of paged_attention_decode_weights is the plain decode call's: the same sums of the same
roundings.  f16 and FP8 caches round P to one f16 (u = 2^-11): what numerator and normaliser share of that
cancels in the output, while the weights, fp32, divide by the sum before the rounding."""
import math

import numpy as np
import pytest
import torch

import paged_kv_cache_373_b200 as pkv
from scoremod_ref import build, cuda

pytestmark = pytest.mark.gpu
F16, BF16, FP8 = torch.float16, torch.bfloat16, torch.uint8

# P of most tokens: just below the middle of two f16 values, so every one is rounded down to 1/2
R = 0.5 + 0.98 * 2.0 ** -12


@pytest.mark.parametrize("cache,value", [(F16, 2 - 2.0 ** -10), (FP8, 1.875)], ids=["f16", "fp8"])
@pytest.mark.parametrize("heads", [(8, 2), (4, 4), (20, 2)])
@pytest.mark.parametrize("num_ctas", [0, 1])
def test_roundings_in_common_cancel(cache, value, heads, num_ctas):
    """One token of every 16 scores 0, the others log2 R: V is one constant, so the output is that constant.
    (The sum before the rounding in its place: 15 (R - 1/2) / 8.5 = 4.2e-4 below it, relative, where half an
    output step is 2.4e-4 to 2.6e-4.  fp32 sums of at most 190 tiles: 190 2^-23 = 2.3e-5.)"""
    Hq, Hkv = heads
    D, bs, lens = 128, 16, [16, 50, 777, 3000]
    d = cuda(build(lens, Hkv, D, bs, cache, 41))
    one, minus = (1.0, -1.0) if cache is F16 else (0x38, 0xB8)  # E4M3 codes
    code = value if cache is F16 else 0x3F
    ks = vs = torch.ones(1, device="cuda") if cache is FP8 else None
    d["kc"].zero_()
    for s, L in enumerate(lens):
        for t in range(0, L, bs):
            b = int(d["tables"][s, t // bs])
            d["kc"][b, 1:, :, 0] = minus
    d["vc"].fill_(code)
    q = torch.zeros(len(lens), Hq, D, dtype=F16, device="cuda")
    q[:, :, 0] = 1
    scale = -math.log(R)
    out, plain = torch.empty_like(q), torch.empty_like(q)
    w = torch.zeros(len(lens), Hkv, max(lens), device="cuda")
    pkv.paged_attention_decode_weights(out, w, q, d["kc"], d["vc"], d["tables"], d["lens"], scale, k_scale=ks,
                                       v_scale=vs, num_ctas=num_ctas)
    pkv.paged_attention_decode(plain, q, d["kc"], d["vc"], d["tables"], d["lens"], scale, ks, vs, num_ctas=num_ctas)
    assert pkv.get_device_error() == 0
    assert (plain == value).all()
    assert (out == value).all()
    # the weights: g probabilities each, every one within 2^-19 + L 2^-23 (scoremod_ref; the scores are exact but
    # for the scale's rounding, 2^-24)
    for s, L in enumerate(lens):
        e = np.where(np.arange(L) % bs == 0, 1.0, math.exp(-float(np.float32(scale))))
        ref = Hq // Hkv * e / e.sum()
        got = w[s, :, :L].double().cpu().numpy()
        assert (np.abs(got / ref - 1) <= 2.0 ** -19 + L * 2.0 ** -23 + 2.0 ** -22).all(), L


CASES = [(F16, F16, 8, 2, 64, 16), (F16, F16, 4, 4, 128, 32), (FP8, F16, 8, 8, 128, 16), (FP8, BF16, 16, 2, 128, 32),
         (BF16, BF16, 8, 2, 128, 16), (torch.float32, torch.float32, 4, 2, 64, 16)]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "%s_%s_%dx%d_D%d_b%d" % (str(c[0])[6:], str(c[1])[6:], *c[2:]))
@pytest.mark.parametrize("lens", [[1, 17, 300, 2000], [5 + 7 * i % 260 for i in range(300)]], ids=["few", "many"])
def test_equals_the_plain_call(case, lens):
    """Peaked softmaxes.  The two calls add the same terms, possibly in another order: at most 100 fp32 adds of
    parts, |difference| <= 2^-17 sum p|v| <= 2^-17 max|v|, and each rounds once to the output type.  Where the
    results are apart at all, a rounding boundary lies between them: 2^-17 max|v| against steps of about
    2^-12 (f16; bf16 has longer ones) at |out| of 0.3 bounds the share of them at some 3 %, and it is a tenth of
    that in practice.  fp32 outputs round nothing and are held to the difference alone."""
    cache, qdt, Hq, Hkv, D, bs = case
    d = cuda(build(lens, Hkv, D, bs, cache, 43))
    q = (4 * torch.randn(len(lens), Hq, D, generator=torch.Generator().manual_seed(44))).to(qdt).cuda()
    out, plain = torch.empty_like(q), torch.empty_like(q)
    w = torch.empty(len(lens), Hkv, max(lens), device="cuda")
    scale = D ** -0.5
    pkv.paged_attention_decode_weights(out, w, q, d["kc"], d["vc"], d["tables"], d["lens"], scale, k_scale=d["ks"],
                                       v_scale=d["vs"])
    pkv.paged_attention_decode(plain, q, d["kc"], d["vc"], d["tables"], d["lens"], scale, d["ks"], d["vs"])
    assert pkv.get_device_error() == 0
    a, b = out.double(), plain.double()
    vmax = max(float(abs(v).max()) for v in d["V"])
    near = 2.0 ** -17 * vmax
    step = torch.finfo(qdt).eps * torch.maximum(a.abs(), b.abs())
    assert ((a - b).abs() <= near + step).all()
    if qdt is not torch.float32:
        assert (a != b).double().mean() <= 0.03
