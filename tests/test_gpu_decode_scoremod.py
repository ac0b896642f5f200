"""paged_attention_decode_scoremod on the GPU against fp64 (bounds: scoremod_ref)."""
import numpy as np
import pytest
import torch

import paged_kv_cache_373_b200 as pkv
from scoremod_ref import assert_near, attend, build, cuda, visible

pytestmark = pytest.mark.gpu
F16, BF16, F32, FP8 = torch.float16, torch.bfloat16, torch.float32, torch.uint8
LENS = [1, 0, 15, 16, 17, 33, 250, 700, 1, 64]


def setup(lens, Hq, Hkv, D, bs, cache, qdt, seed, window=0, prefixes=None, qscale=1.0):
    prefixes = prefixes if prefixes is not None else [0] * len(lens)
    live = [visible(L, L - 1, window, pre) for L, pre in zip(lens, prefixes)]
    d = cuda(build(lens, Hkv, D, bs, cache, seed, live))
    g = torch.Generator().manual_seed(seed + 1)
    d["q"] = (torch.randn(len(lens), Hq, D, generator=g) * qscale).to(qdt).cuda()
    return d


def run(d, scale, num_ctas=0, **mods):
    out = torch.full_like(d["q"], float("nan"))
    pkv.paged_attention_decode_scoremod(out, d["q"], d["kc"], d["vc"], d["tables"], d["lens"], scale,
                                        k_scale=d["ks"], v_scale=d["vs"], num_ctas=num_ctas, **mods)
    assert pkv.get_device_error() == 0
    return out


def check(d, out, scale, softcap=0.0, window=0, slopes=None, prefixes=None):
    for s, L in enumerate(d["lens"].tolist()):
        if L == 0:
            assert (out[s] == 0).all()
            continue
        ref, bound, _, _ = attend(d["q"][s:s + 1].double().cpu().numpy(), d["K"][s], d["V"][s], np.array([L - 1]),
                                  float(np.float32(scale)), d["kc"].dtype, out.dtype, softcap, window,
                                  None if slopes is None else slopes.double().cpu().numpy(),
                                  0 if prefixes is None else max(prefixes[s], 0))
        assert_near(out[s:s + 1], ref, bound, f"sequence {s} of length {L}")


TYPES = [
    # Hq, Hkv, D, bs, cache, q
    (8, 2, 128, 16, BF16, BF16),
    (4, 4, 64, 32, F16, F16),
    (32, 2, 128, 32, F16, F16),     # 16 heads per kv head: two chunks
    (6, 2, 64, 16, BF16, BF16),     # 3 heads per kv head
    (4, 2, 128, 16, F32, F32),
    (4, 1, 64, 32, F32, F32),
    (8, 1, 128, 32, FP8, BF16),
    (4, 4, 128, 16, FP8, F16),
]
MODS = [
    dict(),
    dict(softcap=5.0),
    dict(softcap=50.0, window=1),
    dict(window=16),
    dict(window=37, alibi=True),
    dict(alibi=True, softcap=1.5),
    dict(window=40, prefix=5),
    dict(window=100, prefix=40, alibi=True, softcap=20.0),
    dict(window=33, prefix=10000),
    dict(prefix=70),
]


@pytest.mark.parametrize("mods", MODS, ids=lambda m: "_".join(f"{k}{v}" for k, v in m.items()) or "plain")
@pytest.mark.parametrize("types", TYPES, ids=lambda t: "%dx%d_D%d_b%d_%s" % (*t[:4], str(t[4])[6:]))
def test_matches_fp64(types, mods):
    Hq, Hkv, D, bs, cache, qdt = types
    mods = dict(mods)
    prefix = mods.pop("prefix", 0)
    prefixes = [prefix] * len(LENS) if prefix else None
    if prefix == 40:
        prefixes = [0, 3, -7, 1, 40, 33, 16, 100, 2, 31]
    slopes = torch.linspace(0.02, 0.7, Hq).cuda() if mods.pop("alibi", False) else None
    d = setup(LENS, Hq, Hkv, D, bs, cache, qdt, 11, mods.get("window", 0), prefixes, qscale=3.0)
    pre = None if prefixes is None else torch.tensor(prefixes, dtype=torch.int32).cuda()
    scale = 1 / D ** 0.5
    out = run(d, scale, alibi_slopes=slopes, prefix_lens=pre, **mods)
    check(d, out, scale, slopes=slopes, prefixes=prefixes, **mods)


@pytest.mark.parametrize("num_ctas", [1, 5, 148, 700])
def test_split_counts(num_ctas):
    lens = [900, 3, 2500, 47]
    d = setup(lens, 8, 2, 128, 16, BF16, BF16, 12, 600, [20] * 4)
    pre = torch.full((4,), 20, dtype=torch.int32).cuda()
    out = run(d, 0.1, num_ctas, softcap=10.0, window=600, prefix_lens=pre)
    check(d, out, 0.1, 10.0, 600, None, [20] * 4)


def test_large_batch_takes_the_wide_scan():
    lens = [(7 * i) % 61 for i in range(600)]
    prefixes = [i % 9 for i in range(600)]
    d = setup(lens, 4, 2, 64, 16, F16, F16, 13, 20, prefixes)
    pre = torch.tensor(prefixes, dtype=torch.int32).cuda()
    out = run(d, 0.125, softcap=8.0, window=20, prefix_lens=pre)
    check(d, out, 0.125, 8.0, 20, None, prefixes)


def test_unmodified_equals_the_plain_decode():
    """Without modifiers and with whole tiles the arithmetic is the plain decode's, bit for bit."""
    lens = [16, 160, 1600]
    d = setup(lens, 8, 2, 128, 16, BF16, BF16, 14)
    a = run(d, 0.09, 40)
    b = torch.empty_like(a)
    pkv.paged_attention_decode(b, d["q"], d["kc"], d["vc"], d["tables"], d["lens"], 0.09, num_ctas=40)
    assert torch.equal(a, b)


def test_extreme_caps_and_scores():
    d = setup([40, 300], 4, 4, 128, 16, F32, F32, 15, qscale=1.0)
    d["q"] *= 1e4     # scores of thousands: a cap of 30 saturates, one of 1e6 hardly acts
    for cap in (30.0, 1e6, 1e-3):
        out = run(d, 1.0, softcap=cap)
        check(d, out, 1.0, cap)
    # infinite scores: the cap makes them +-cap
    d = setup([20], 2, 2, 64, 16, F16, F16, 16)
    d["kc"][d["tables"][0, 0].item(), 3] = float("inf")
    d["q"].abs_()
    out = run(d, 1.0, softcap=4.0)
    d["K"][0][3] = 1e9
    ref, _, p, _ = attend(d["q"].double().cpu().numpy(), d["K"][0], d["V"][0], np.array([19]), 1.0, F16, F16, 4.0)
    assert torch.isfinite(out).all()
    assert np.abs(out.double().cpu().numpy() - ref).max() < 1e-2   # f16 P and output: 2^-11 of |v| < 5, twice


def test_lengths_past_the_table_and_bad_blocks_are_flagged():
    d = setup([40, 30], 4, 2, 64, 16, F16, F16, 17, 20)
    out = torch.empty_like(d["q"])
    call = lambda t, l: pkv.paged_attention_decode_scoremod(out, d["q"], d["kc"], d["vc"], t, l, 0.1, window=20)
    call(d["tables"], torch.tensor([400, 30], dtype=torch.int32, device="cuda"))
    assert pkv.get_device_error() & pkv.DEVERR_SEQ_LEN
    t = d["tables"].clone()
    t[0, 2] = d["kc"].shape[0]
    call(t, d["lens"])
    assert pkv.get_device_error() == pkv.DEVERR_BLOCK_ID
    t = d["tables"].clone()
    t[0, 0] = 1 << 20          # the block before the window is not looked at
    call(t, d["lens"])
    assert pkv.get_device_error() == 0


def test_graph_replay_reads_its_inputs_anew():
    d = setup([100, 30, 700], 8, 2, 128, 16, BF16, BF16, 18)
    ws = pkv.alloc_workspace(3, 8, 2, 128)
    out = torch.empty_like(d["q"])
    call = lambda: pkv.paged_attention_decode_scoremod(out, d["q"], d["kc"], d["vc"], d["tables"], d["lens"], 0.1,
                                                       softcap=9.0, workspace=ws)
    call()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    d["q"].mul_(-2)
    d["lens"].copy_(torch.tensor([1, 0, 640], dtype=torch.int32))
    d["K"], d["V"] = [x[:n] for x, n in zip(d["K"], [1, 0, 640])], [x[:n] for x, n in zip(d["V"], [1, 0, 640])]
    out.fill_(float("nan"))
    g.replay()
    torch.cuda.synchronize()
    check(d, out, 0.1, 9.0)


@pytest.mark.parametrize("S", [1, 32, 33, 200, 256, 257])
def test_batch_sizes_around_the_length_scans(S):
    g = np.random.default_rng(S)
    lens = [int(x) for x in g.choice([0, 0, 1, 15, 16, 17, 130, 260], S)]
    if S == 1:
        lens = [0]     # nothing at all to attend
    prefixes = [int(x) for x in g.integers(-2, 40, S)]
    d = setup(lens, 4, 2, 64, 16, F16, F16, 17, 25, prefixes)
    pre = torch.tensor(prefixes, dtype=torch.int32).cuda()
    out = run(d, 0.125, softcap=8.0, window=25, prefix_lens=pre)
    check(d, out, 0.125, 8.0, 25, None, prefixes)
