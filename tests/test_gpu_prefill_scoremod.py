"""paged_prefill_scoremod on the GPU against fp64 (bounds: scoremod_ref)."""
import numpy as np
import pytest
import torch

import paged_kv_cache_373_b200 as pkv
from scoremod_ref import assert_near, attend, build, cuda, visible

pytestmark = pytest.mark.gpu
F16, BF16 = torch.float16, torch.bfloat16


def setup(ctx, chunks, Hq, Hkv, D, bs, dtype, seed, window=0, prefixes=None, qscale=1.0):
    prefixes = prefixes if prefixes is not None else [0] * len(ctx)
    lens = [a + b for a, b in zip(ctx, chunks)]
    live = []
    for c, n, L, pre in zip(ctx, chunks, lens, prefixes):
        v = np.zeros(L, dtype=bool)
        for i in range(n):
            v |= visible(L, c + i, window, pre)
        # hidden tokens share blocks with attended ones: those hold finite values, whole blocks may hold anything
        for b in range(0, L, bs):
            v[b:b + bs] = v[b:b + bs].any()
        live.append(v)
    d = cuda(build(lens, Hkv, D, bs, dtype, seed, live))
    g = torch.Generator().manual_seed(seed + 1)
    d["q"] = (torch.randn(sum(chunks), Hq, D, generator=g) * qscale).to(dtype).cuda()
    d["qs"] = torch.tensor([0] + list(np.cumsum(chunks)), dtype=torch.int32).cuda()
    return d


def run(d, scale, **mods):
    out = torch.full_like(d["q"], 55.0)
    pkv.paged_prefill_scoremod(out, d["q"], d["kc"], d["vc"], d["tables"], d["lens"], d["qs"], scale, **mods)
    assert pkv.get_device_error() == 0
    return out


def check(d, out, scale, softcap=0.0, window=0, slopes=None, prefixes=None):
    qs = d["qs"].tolist()
    for s, L in enumerate(d["lens"].tolist()):
        a, b = qs[s], qs[s + 1]
        if a == b:
            continue
        pos = np.arange(a, b) - b + L
        ref, bound, _, _ = attend(d["q"][a:b].double().cpu().numpy(), d["K"][s], d["V"][s], pos,
                                  float(np.float32(scale)), d["kc"].dtype, out.dtype, softcap, window,
                                  None if slopes is None else slopes.double().cpu().numpy(),
                                  0 if prefixes is None else max(prefixes[s], 0))
        assert_near(out[a:b], ref, bound, f"sequence {s}, {b - a} rows of {L} tokens")


TYPES = [
    # Hq, Hkv, D, bs, dtype
    (8, 4, 128, 16, BF16),
    (4, 4, 64, 32, F16),
    (16, 2, 64, 16, F16),
    (16, 1, 128, 32, BF16),
    (8, 2, 128, 32, F16),
]
MODS = [
    dict(),
    dict(softcap=3.0),
    dict(softcap=50.0, window=1),
    dict(window=16),
    dict(window=70, alibi=True),
    dict(alibi=True, softcap=1.5),
    dict(window=100, prefix=5),
    dict(window=90, prefix=140, alibi=True, softcap=20.0),
    dict(window=33, prefix=10000),
    dict(prefix=230),
]
CTX, CHUNKS = [0, 300, 37, 0, 500, 64], [200, 129, 1, 0, 1, 64]


@pytest.mark.parametrize("mods", MODS, ids=lambda m: "_".join(f"{k}{v}" for k, v in m.items()) or "plain")
@pytest.mark.parametrize("types", TYPES, ids=lambda t: "%dx%d_D%d_b%d_%s" % (*t[:4], str(t[4])[6:]))
def test_matches_fp64(types, mods):
    Hq, Hkv, D, bs, dtype = types
    mods = dict(mods)
    prefix = mods.pop("prefix", 0)
    prefixes = [prefix] * len(CTX) if prefix else None
    if prefix == 140:
        prefixes = [140, 17, -3, 5, 64, 0]
    slopes = torch.linspace(0.02, 0.7, Hq).cuda() if mods.pop("alibi", False) else None
    d = setup(CTX, CHUNKS, Hq, Hkv, D, bs, dtype, 31, mods.get("window", 0), prefixes, qscale=2.0)
    pre = None if prefixes is None else torch.tensor(prefixes, dtype=torch.int32).cuda()
    scale = 1 / D ** 0.5
    out = run(d, scale, alibi_slopes=slopes, prefix_lens=pre, **mods)
    check(d, out, scale, slopes=slopes, prefixes=prefixes, **mods)


def test_long_context_window_and_sinks():
    # pairs of units far past the prefix: a long gap, odd and even numbers of units
    ctx, chunks = [4000, 3333], [300, 77]
    d = setup(ctx, chunks, 8, 4, 128, 16, BF16, 32, 200, [4, 65])
    pre = torch.tensor([4, 65], dtype=torch.int32).cuda()
    out = run(d, 0.09, window=200, prefix_lens=pre)
    check(d, out, 0.09, 0.0, 200, None, [4, 65])
    assert (d["tables"] < 0).sum() > 300      # most of the context's blocks were never looked at


def test_unmodified_equals_the_plain_prefill():
    d = setup(CTX, CHUNKS, 8, 4, 64, 16, F16, 33)
    out = run(d, 0.125)
    ref = torch.full_like(out, 55.0)
    pkv.paged_prefill(ref, d["q"], d["kc"], d["vc"], d["tables"], d["lens"], d["qs"], 0.125)
    check(d, ref, 0.125)
    check(d, out, 0.125)


def test_one_token_chunks_match_the_decode_form():
    lens = [1, 17, 300, 2049]
    d = setup([L - 1 for L in lens], [1] * 4, 16, 4, 128, 16, BF16, 34, 150, [10] * 4)
    pre = torch.full((4,), 10, dtype=torch.int32).cuda()
    out = run(d, 0.09, window=150, prefix_lens=pre, softcap=4.0)
    dec = torch.empty_like(out)
    pkv.paged_attention_decode_scoremod(dec, d["q"], d["kc"], d["vc"], d["tables"], d["lens"], 0.09, window=150,
                                        prefix_lens=pre, softcap=4.0)
    check(d, out, 0.09, 4.0, 150, None, [10] * 4)
    check(d, dec, 0.09, 4.0, 150, None, [10] * 4)


def test_large_scores_move_the_reference_on_every_tile():
    # keys grow along the sequence: each tile's maximum passes the last one's by far more than 2^8
    d = setup([0, 100], [250, 140], 8, 2, 128, 16, BF16, 35)
    for s, L in enumerate(d["lens"].tolist()):
        for t in range(L):
            b = int(d["tables"][s, t // 16])
            row = (d["kc"][b, t % 16].float() * (1 + t / 8)).to(BF16)
            d["kc"][b, t % 16] = row
            d["K"][s][t] = row.double().cpu().numpy()
    for cap in (0.0, 30.0):
        out = run(d, 0.2, softcap=cap)
        check(d, out, 0.2, cap)


def test_errors_are_flagged_and_rows_left():
    d = setup([10, 20], [5, 5], 8, 4, 64, 16, F16, 36)
    out = torch.full_like(d["q"], 55.0)
    short = torch.tensor([3, 25], dtype=torch.int32, device="cuda")
    pkv.paged_prefill_scoremod(out, d["q"], d["kc"], d["vc"], d["tables"], short, d["qs"], 0.1, window=8)
    assert pkv.get_device_error() == pkv.DEVERR_SEQ_LEN
    assert (out[:5] == 55).all()
    t = d["tables"].clone()
    t[1, 1] = d["kc"].shape[0] + 3
    pkv.paged_prefill_scoremod(out, d["q"], d["kc"], d["vc"], t, d["lens"], d["qs"], 0.1, window=8)
    assert pkv.get_device_error() == pkv.DEVERR_BLOCK_ID


def test_graph_replay():
    d = setup(CTX, CHUNKS, 8, 4, 128, 16, BF16, 37)
    out = torch.empty_like(d["q"])
    call = lambda: pkv.paged_prefill_scoremod(out, d["q"], d["kc"], d["vc"], d["tables"], d["lens"], d["qs"], 0.1,
                                              softcap=9.0)
    call()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    d["q"].mul_(-1)
    out.fill_(float("nan"))
    g.replay()
    torch.cuda.synchronize()
    check(d, out, 0.1, 9.0)


@pytest.mark.parametrize("stop_tile", [0, 1, 3])
def test_bounded_waits_run_out_then_the_context_recovers(stop_tile):
    """The copies stop before tile `stop_tile`: every wait for them runs out (1 ms here), the call sets
    PKV_DEVERR_TIMEOUT, and the next call on the same SMs finds their tensor memory free and is right."""
    mods = dict(window=300, softcap=6.0)
    d = setup([0, 300, 1000], [200, 64, 1], 16, 8, 128, 16, BF16, 38, 300)
    out = torch.full_like(d["q"], 55.0)
    assert pkv.lib().pkv_testing_prefill_timeout(stop_tile, 1_000_000) == pkv.PKV_OK
    pkv.paged_prefill_scoremod(out, d["q"], d["kc"], d["vc"], d["tables"], d["lens"], d["qs"], 0.09, **mods)
    assert pkv.get_device_error() == pkv.DEVERR_TIMEOUT
    out = run(d, 0.09, **mods)
    check(d, out, 0.09, **mods)


def test_many_short_chunks():
    ctx, chunks = [(13 * i) % 90 for i in range(150)], [(7 * i) % 5 for i in range(150)]
    d = setup(ctx, chunks, 4, 2, 64, 16, F16, 39, 20)
    out = run(d, 0.125, window=20)
    check(d, out, 0.125, 0.0, 20)


@pytest.mark.parametrize("Hq,Hkv,D,dtype", [(2, 2, 128, BF16), (2, 2, 64, F16), (16, 1, 128, BF16)])
@pytest.mark.parametrize("slope", [0.001, 0.5, 8.0])
def test_bias_over_long_contexts(Hq, Hkv, D, dtype, slope):
    # pairs whose second unit ends tiles before the first (one head per kv head), one and two units, one tile
    ctx, chunks = [700, 0, 1500, 0, 65], [260, 600, 129, 3, 64]
    d = setup(ctx, chunks, Hq, Hkv, D, 16, dtype, 51)
    slopes = (slope * torch.linspace(0.5, 1.0, Hq)).cuda()
    out = run(d, 0.1, alibi_slopes=slopes)
    check(d, out, 0.1, slopes=slopes)


def test_bias_with_the_reference_moving_on_every_tile():
    # keys shrink along the sequence: walking back, each tile's maximum passes the last one's
    d = setup([0, 100], [250, 140], 8, 2, 128, 16, BF16, 52)
    for s, L in enumerate(d["lens"].tolist()):
        for t in range(L):
            b = int(d["tables"][s, t // 16])
            row = (d["kc"][b, t % 16].float() * (1 + (L - t) / 8)).to(BF16)
            d["kc"][b, t % 16] = row
            d["K"][s][t] = row.double().cpu().numpy()
    slopes = torch.linspace(0.01, 0.1, 8).cuda()
    out = run(d, 0.2, alibi_slopes=slopes)
    check(d, out, 0.2, slopes=slopes)


@pytest.mark.parametrize("S", [2, 31, 32, 33])
def test_units_of_many_sequences(S):
    # the pairs are ordered by length for up to 32 sequences, empty chunks among them
    g = np.random.default_rng(S)
    chunks = [int(c) for c in g.choice([0, 1, 5, 70, 300], S)]
    chunks[0] = 300
    ctx = [int(c) for c in g.choice([0, 1, 90, 400], S)]
    d = setup(ctx, chunks, 4, 2, 64, 16, F16, 53)
    out = run(d, 0.125, softcap=10.0)
    check(d, out, 0.125, 10.0)


@pytest.mark.parametrize("mods", MODS, ids=lambda m: "_".join(f"{k}{v}" for k, v in m.items()) or "plain")
@pytest.mark.parametrize("types", [(32, 8, 128, 16, BF16), (16, 16, 64, 32, F16), (16, 16, 128, 16, BF16)],
                         ids=lambda t: "%dx%d_D%d_b%d_%s" % (*t[:4], str(t[4])[6:]))
def test_more_units_than_sms(types, mods):
    """Units in pairs: each kv head's rows alone would not fit one unit per SM (148)."""
    Hq, Hkv, D, bs, dtype = types
    ctx, chunks = [0, 300, 37, 0, 700, 64, 0], [200, 129, 1, 0, 106, 64, 300 if Hq > Hkv else 600]
    assert (sum(chunks) * (Hq // Hkv) // 128 + len(ctx)) * Hkv > 160
    mods = dict(mods)
    prefix = mods.pop("prefix", 0)
    prefixes = [prefix] * len(ctx) if prefix else None
    if prefix == 140:
        prefixes = [140, 17, -3, 5, 64, 0, 300]
    slopes = torch.linspace(0.02, 0.7, Hq).cuda() if mods.pop("alibi", False) else None
    d = setup(ctx, chunks, Hq, Hkv, D, bs, dtype, 61, mods.get("window", 0), prefixes, qscale=2.0)
    pre = None if prefixes is None else torch.tensor(prefixes, dtype=torch.int32).cuda()
    scale = 1 / D ** 0.5
    out = run(d, scale, alibi_slopes=slopes, prefix_lens=pre, **mods)
    check(d, out, scale, slopes=slopes, prefixes=prefixes, **mods)


def test_pairs_with_the_reference_moving_on_every_tile():
    for grow in (True, False):  # keys that grow along the sequence, and keys that shrink (with a bias)
        d = setup([0, 100, 0], [250, 140, 300], 32, 8, 128, 16, BF16, 62)
        for s, L in enumerate(d["lens"].tolist()):
            t = torch.arange(L, device="cuda")
            f = (1 + (t if grow else L - t) / 8)[:, None, None]
            rows = (d["kc"][d["tables"][s, t // 16].long(), t % 16].float() * f).to(BF16)
            d["kc"][d["tables"][s, t // 16].long(), t % 16] = rows
            d["K"][s] = rows.double().cpu().numpy()
        slopes = None if grow else torch.linspace(0.01, 0.1, 32).cuda()
        out = run(d, 0.2, alibi_slopes=slopes, softcap=30.0 if grow else 0.0)
        check(d, out, 0.2, 30.0 if grow else 0.0, 0, slopes)


@pytest.mark.parametrize("stop_tile", [0, 1, 3])
@pytest.mark.parametrize("bias", [False, True])
def test_bounded_waits_of_pairs_run_out(stop_tile, bias):
    d = setup([0, 300, 1000], [300, 200, 106], 32, 8, 128, 16, BF16, 63, 300)
    slopes = torch.linspace(0.02, 0.7, 32).cuda() if bias else None
    out = torch.full_like(d["q"], 55.0)
    assert pkv.lib().pkv_testing_prefill_timeout(stop_tile, 1_000_000) == pkv.PKV_OK
    pkv.paged_prefill_scoremod(out, d["q"], d["kc"], d["vc"], d["tables"], d["lens"], d["qs"], 0.09, window=300,
                               alibi_slopes=slopes)
    assert pkv.get_device_error() == pkv.DEVERR_TIMEOUT
    out = run(d, 0.09, window=300, alibi_slopes=slopes)
    check(d, out, 0.09, 0.0, 300, slopes)
