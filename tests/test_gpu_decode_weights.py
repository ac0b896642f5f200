"""paged_attention_decode_weights on the GPU against fp64.

A weight is a sum of g probabilities, each within the relative bound `rel` of
scoremod_ref (fp32 throughout: P's 16-bit form is not used), added in fp32 to
the weight so far: |error| <= sum_h p rel + (g + 2) 2^-24 (|in| + sum_h p)."""
import numpy as np
import pytest
import torch

import paged_kv_cache_373_b200 as pkv
from scoremod_ref import assert_near, attend, build, cuda

pytestmark = pytest.mark.gpu
F16, BF16, F32, FP8 = torch.float16, torch.bfloat16, torch.float32, torch.uint8
LENS = [1, 0, 2, 15, 16, 17, 33, 250, 1300, 64]


def setup(lens, Hq, Hkv, D, bs, cache, qdt, seed, extra=0):
    d = cuda(build(lens, Hkv, D, bs, cache, seed))
    g = torch.Generator().manual_seed(seed + 1)
    d["q"] = (torch.randn(len(lens), Hq, D, generator=g) * 2).to(qdt).cuda()
    d["w"] = torch.rand(len(lens), Hkv, max(lens) + extra, generator=g).cuda()
    return d


def run(d, scale, weights_out=None, weights="w", num_ctas=0):
    out = torch.full_like(d["q"], float("nan"))
    wo = torch.full_like(d["w"], 77.0) if weights_out is None else weights_out
    pkv.paged_attention_decode_weights(out, wo, d["q"], d["kc"], d["vc"], d["tables"], d["lens"], scale,
                                       weights=d[weights] if weights else None, k_scale=d["ks"], v_scale=d["vs"],
                                       num_ctas=num_ctas)
    assert pkv.get_device_error() == 0
    return out, wo


def check(d, out, wo, scale, w_in, untouched=77.0):
    Hkv = d["kc"].shape[2]
    for s, L in enumerate(d["lens"].tolist()):
        tail = wo[s, :, L:]
        assert (tail == untouched).all() if isinstance(untouched, float) else torch.equal(tail, untouched[s, :, L:])
        if L == 0:
            assert (out[s] == 0).all()
            continue
        ref, bound, p, rel = attend(d["q"][s:s + 1].double().cpu().numpy(), d["K"][s], d["V"][s], np.array([L - 1]),
                                    float(np.float32(scale)), d["kc"].dtype, out.dtype)
        assert_near(out[s:s + 1], ref, bound, f"sequence {s} of length {L}")
        g = p.shape[1] // Hkv
        add = p[0].reshape(Hkv, g, L).sum(1)
        off = (p[0] * rel[0][:, None]).reshape(Hkv, g, L).sum(1)
        old = np.zeros((Hkv, L)) if w_in is None else w_in[s, :, :L].double().cpu().numpy().copy()
        old[:, L - 1] = 0
        assert_near(wo[s, :, :L], old + add, off + (g + 2) * 2.0 ** -24 * (old + add), f"weights of sequence {s}")


TYPES = [
    (8, 2, 128, 16, BF16, BF16),
    (4, 4, 64, 32, F16, F16),
    (32, 2, 128, 32, F16, F16),
    (6, 2, 64, 16, BF16, BF16),
    (4, 2, 128, 16, F32, F32),
    (4, 4, 64, 16, F32, F32),
    (20, 2, 128, 16, F32, F32),
    (8, 1, 128, 32, FP8, BF16),
    (4, 4, 128, 16, FP8, F16),
]


@pytest.mark.parametrize("types", TYPES, ids=lambda t: "%dx%d_D%d_b%d_%s" % (*t[:4], str(t[4])[6:]))
@pytest.mark.parametrize("num_ctas", [0, 2])
def test_matches_fp64(types, num_ctas):
    Hq, Hkv, D, bs, cache, qdt = types
    d = setup(LENS, Hq, Hkv, D, bs, cache, qdt, 21, extra=5)
    scale = 1 / D ** 0.5
    out, wo = run(d, scale, num_ctas=num_ctas)
    check(d, out, wo, scale, d["w"])


def test_no_weights_in_and_in_place():
    d = setup([5, 300, 0, 41], 8, 4, 64, 16, F16, F16, 22)
    out, wo = run(d, 0.1, weights=None)
    check(d, out, wo, 0.1, None)
    w0 = d["w"].clone()
    out, wo = run(d, 0.1, weights_out=d["w"])
    assert wo.data_ptr() == d["w"].data_ptr()
    check(d, out, wo, 0.1, w0, untouched=w0)


def test_large_batch_and_repeat():
    lens = [(11 * i) % 83 for i in range(700)]
    d = setup(lens, 4, 2, 64, 16, BF16, BF16, 23)
    out, wo = run(d, 0.125)
    check(d, out, wo, 0.125, d["w"])
    out2, wo2 = run(d, 0.125)          # no atomics: the same bits
    assert torch.equal(wo, wo2) and torch.equal(out, out2)


def test_long_sequence_over_several_items():
    d = setup([5000, 1024, 1025], 4, 1, 64, 32, F16, F16, 24)
    out, wo = run(d, 0.125)
    check(d, out, wo, 0.125, d["w"])
    # every q head's probabilities add up to one: g per kv head (w_in taken off; sums of 5000 fp32 values below 1)
    total = (wo[0, 0].double() - torch.cat([d["w"][0, 0, :-1], d["w"].new_zeros(1)]).double()).sum().item()
    assert abs(total - 4) < 5000 * 2.0 ** -23


def test_weight_rows_shorter_than_a_sequence_are_flagged():
    d = setup([40, 20], 4, 2, 64, 16, F16, F16, 25)
    out = torch.empty_like(d["q"])
    wo = torch.full((2, 2, 32), 5.0, device="cuda")
    pkv.paged_attention_decode_weights(out, wo, d["q"], d["kc"], d["vc"], d["tables"], d["lens"], 0.1)
    assert pkv.get_device_error() == pkv.DEVERR_SEQ_LEN
    assert (wo[1, :, 20:] == 5).all()
    with pytest.raises(pkv.PkvError):
        pkv.paged_attention_decode_weights(out, wo, d["q"], d["kc"], d["vc"], d["tables"], d["lens"], 0.1,
                                           workspace=torch.empty(1024, dtype=torch.uint8, device="cuda"))


def test_graph_replay_accumulates():
    d = setup([100, 30, 700], 8, 2, 128, 16, BF16, BF16, 26)
    n = pkv.paged_attention_weights_workspace_bytes(3, 8, 2, 128, d["tables"].shape[1] * 16)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    out = torch.empty_like(d["q"])
    w0 = d["w"].clone()
    call = lambda w: pkv.paged_attention_decode_weights(out, w, d["q"], d["kc"], d["vc"], d["tables"], d["lens"],
                                                        0.1, weights=w, workspace=ws)
    want = w0.clone()
    for _ in range(3):
        call(want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(d["w"])
    d["w"].copy_(w0)
    for _ in range(3):
        g.replay()
    torch.cuda.synchronize()
    assert torch.equal(d["w"], want)


@pytest.mark.parametrize("S", [1, 32, 33, 200, 256, 257])
@pytest.mark.parametrize("Hkv", [2, 8])
def test_batch_sizes_around_the_length_scans(S, Hkv):
    g = np.random.default_rng(S)
    lens = [int(x) for x in g.choice([0, 0, 1, 15, 16, 17, 130, 260], S)]
    if S == 1:
        lens = [0]     # nothing at all to attend
    d = setup(lens, 2 * Hkv, Hkv, 64, 16, F16, F16, 25, extra=5)  # (rows of no weights at all are refused)
    out, wo = run(d, 0.125)
    check(d, out, wo, 0.125, d["w"])
