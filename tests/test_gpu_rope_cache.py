"""qk_norm_rope_and_cache on the GPU against the formulas in fp64.

Tolerances, from the arithmetic.  The kernel works in fp32 from the loaded
values: the norm's sum of D <= 128 squares (relative error below D * 2^-24 in
the sum, half of that in its root, measured against sqrt), rsqrtf (2 ulp), two
products, then two products and a sum for the rotation.  In all below
100 * 2^-24 of the pair's length sqrt(a^2 + b^2), which bounds |a c - b d| for
c^2 + d^2 = 1; then one rounding to the output type, eps(type)/2 relative.
FP8 codes: the value may cross a rounding border, so a code may be off by one
step (2^-3 relative, 2^-9 absolute in the subnormal range, in units of the scale),
and all but a few must be the very codes of the fp64 result."""
import numpy as np
import pytest
import torch

import paged_kv_cache_373_b200 as pkv

pytestmark = pytest.mark.gpu
EPS = 1e-5


def make(T, Hq, Hkv, D, dtype, cache, rot, norm, seed=0, bs=16, fused=True, max_pos=500):
    g = torch.Generator().manual_seed(seed)
    n = (Hq + 2 * Hkv) * D
    qkv = torch.randn(T, n, generator=g).to(dtype).cuda()
    s = {}
    q, k, v = qkv.split([Hq * D, Hkv * D, Hkv * D], 1)
    if not fused:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    s["q"], s["k"], s["v"] = (x.view(T, -1, D) for x in (q, k, v))
    nb = -(-T // bs) + 3
    kd = torch.uint8 if cache == "fp8" else dtype
    s["kc"] = (torch.randn(nb, bs, Hkv, D, generator=g) * 3).to(dtype).cuda()
    if cache == "fp8":
        s["kc"] = torch.randint(0, 120, (nb, bs, Hkv, D), generator=g, dtype=torch.uint8).cuda()
    s["vc"] = s["kc"].clone()
    assert s["kc"].dtype == kd
    s["slots"] = torch.randperm(nb * bs, generator=g)[:T].cuda()
    s["pos"] = torch.randint(0, max_pos, (T,), generator=g).cuda()
    s["cs"] = None
    if rot:
        a = torch.arange(max_pos, dtype=torch.float64)[:, None] * 10000.0 ** (-torch.arange(rot // 2, dtype=torch.float64) / (rot // 2))
        s["cs"] = torch.cat([a.cos(), a.sin()], 1).float().cuda()
    s["qw"] = s["kw"] = None
    if norm:
        s["qw"] = (1 + 0.3 * torch.randn(D, generator=g)).to(dtype).cuda()
        s["kw"] = (1 + 0.3 * torch.randn(D, generator=g)).to(dtype).cuda()
    s["ks"] = torch.tensor([0.013]).cuda() if cache == "fp8" else None
    s["vs"] = torch.tensor([0.011]).cuda() if cache == "fp8" else None
    return s


def call(s, interleaved=False, out=None, **kw):
    out = torch.full(s["q"].shape, 7.0, dtype=s["q"].dtype, device="cuda") if out is None else out
    pkv.qk_norm_rope_and_cache(out, s["q"], s["k"], s["v"], s["kc"], s["vc"], s["slots"], s["pos"], s["cs"],
                               s["qw"], s["kw"], EPS, interleaved, s["ks"], s["vs"], **kw)
    return out


def formula(s, x, w, interleaved):
    """fp64 rows, and per element the length of its pair (of its own value where it is not rotated)."""
    x = x.double().cpu()
    if w is not None:
        x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + EPS) * w.double().cpu()
    size = x.abs()
    if s["cs"] is not None:
        r = s["cs"].shape[1]
        t = s["cs"].double().cpu()[s["pos"].cpu()][:, None]
        c, d = t[..., :r // 2], t[..., r // 2:]
        ia = torch.arange(0, r, 2) if interleaved else torch.arange(r // 2)
        ib = ia + 1 if interleaved else ia + r // 2
        a, b = x[..., ia], x[..., ib]
        size = size.clone()
        size[..., ia] = size[..., ib] = torch.hypot(a, b)
        x = x.clone()
        x[..., ia], x[..., ib] = a * c - b * d, b * c + a * d
    return x, size


def near(got, want, size, dtype):
    got = got.double().cpu()
    tol = 100 * 2.0 ** -24 * size + (torch.finfo(dtype).eps / 2) * want.abs() * (1 + 1e-6) + torch.finfo(dtype).tiny * torch.finfo(dtype).eps
    assert torch.isfinite(got).all()
    worst = ((got - want).abs() - tol).max().item() if got.numel() else 0.0
    assert worst <= 0, worst


def check(s, out, interleaved=False, kc0=None, vc0=None, live=None):
    dtype = s["q"].dtype
    T, Hkv, D = s["k"].shape
    live = torch.arange(T) if live is None else live
    wq, sq = formula(s, s["q"], s["qw"], interleaved)
    wk, sk = formula(s, s["k"], s["kw"], interleaved)
    near(out[live], wq[live], sq[live], dtype)
    slots = s["slots"].cpu()[live]
    kc, vc = s["kc"].view(-1, Hkv, D).cpu(), s["vc"].view(-1, Hkv, D).cpu()
    if s["ks"] is None:
        near(kc[slots], wk[live], sk[live], dtype)
        assert torch.equal(vc[slots].view(torch.uint8), s["v"].cpu()[live].contiguous().view(torch.uint8))
    else:
        ks, vs = s["ks"].item(), s["vs"].item()
        for got, want in ((kc[slots], wk[live] / ks), (vc[slots], s["v"].double().cpu()[live] / vs)):
            got8 = got.view(torch.float8_e4m3fn).double()
            want8 = want.clamp(-448, 448).float().to(torch.float8_e4m3fn)
            assert ((got8 - want.clamp(-448, 448)).abs() <= want.abs() * 2.0 ** -3 + 2.0 ** -9).all()
            assert (got != want8.view(torch.uint8)).float().mean() < 1e-3
    # every other slot as it was
    rest = torch.ones(kc.shape[0], dtype=torch.bool)
    rest[slots] = False
    if kc0 is not None:
        assert torch.equal(kc[rest].view(torch.uint8), kc0.view(-1, Hkv, D).cpu()[rest].view(torch.uint8))
        assert torch.equal(vc[rest].view(torch.uint8), vc0.view(-1, Hkv, D).cpu()[rest].view(torch.uint8))


CASES = [
    # T, Hq, Hkv, D, dtype, cache, rotary, interleaved, norm, fused
    (1, 32, 8, 128, torch.bfloat16, "same", 128, False, True, True),
    (5, 4, 4, 64, torch.float16, "same", 64, False, True, False),
    (7, 8, 2, 128, torch.float32, "same", 128, False, True, True),
    (7, 8, 2, 64, torch.float32, "same", 48, True, True, True),
    (33, 3, 1, 64, torch.bfloat16, "same", 16, False, False, True),
    (33, 6, 3, 128, torch.float16, "same", 96, False, True, True),
    (9, 16, 2, 128, torch.float16, "same", 64, True, False, True),
    (300, 32, 8, 128, torch.bfloat16, "same", 128, False, True, True),      # four rows per lane group
    (1025, 7, 7, 64, torch.float16, "same", 32, True, True, True),
    (700, 16, 8, 128, torch.float32, "same", 0, False, True, True),
    (40, 8, 8, 128, torch.bfloat16, "same", 0, False, False, False),        # neither norm nor rotation: a copy
    (65, 64, 8, 128, torch.bfloat16, "fp8", 128, False, True, True),
    (700, 10, 2, 64, torch.float16, "fp8", 48, False, False, True),
    (12, 2, 1, 64, torch.float32, "fp8", 64, True, True, True),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "T%d_%dx%d_D%d_%s_%s_r%d_%s%s" % (
    c[0], c[1], c[2], c[3], str(c[4])[6:], c[5], c[6], "i" if c[7] else "h", "n" if c[8] else ""))
def test_matches_the_formula(case):
    T, Hq, Hkv, D, dtype, cache, rot, inter, norm, fused = case
    s = make(T, Hq, Hkv, D, dtype, cache, rot, norm, seed=T + Hq, fused=fused)
    kc0, vc0 = s["kc"].clone(), s["vc"].clone()
    out = call(s, inter)
    assert pkv.get_device_error() == 0
    check(s, out, inter, kc0, vc0)


def test_padding_bad_slots_and_positions_write_nothing():
    s = make(20, 8, 2, 128, torch.bfloat16, "same", 128, True, seed=3)
    s["slots"][[2, 19]] = -1
    kc0, vc0 = s["kc"].clone(), s["vc"].clone()
    live = torch.tensor([i for i in range(20) if i not in (2, 19)])
    out = call(s)
    assert pkv.get_device_error() == 0
    assert (out[[2, 19]] == 7).all()
    check(s, out, False, kc0, vc0, live)
    # a slot past the pool, and positions outside the table
    s["kc"].copy_(kc0), s["vc"].copy_(vc0)
    s["slots"][4] = s["kc"].shape[0] * 16
    out = call(s)
    assert pkv.get_device_error() == pkv.DEVERR_SLOT
    s["slots"][4] = -1
    for bad in (-1, 500, 1 << 40):
        s["pos"][7] = bad
        out = call(s)
        assert pkv.get_device_error() == pkv.DEVERR_POSITION
        assert (out[[2, 4, 7, 19]] == 7).all()
    s["pos"][7] = 0
    live = torch.tensor([i for i in range(20) if i not in (2, 4, 7, 19)])
    check(s, out, False, live=live)


def test_in_place_and_reshape_and_cache_agree():
    s = make(50, 8, 4, 64, torch.float16, "same", 64, True, seed=4, fused=False)
    want = call(s)
    again = s["q"].clone()
    s["q"] = again
    got = call(s, out=again)
    assert got.data_ptr() == again.data_ptr() and torch.equal(got, want)
    # no norm, no rotation: the bits of reshape_and_cache, NaN payloads included, in every cache type
    for dtype, cache in ((torch.bfloat16, "same"), (torch.float16, "fp8"), (torch.float32, "fp8")):
        s = make(50, 4, 4, 64, dtype, cache, 0, False, seed=5, fused=False)
        s["v"][3, 1, 5] = float("nan")
        s["k"][4, 0, :9] = float("inf")
        a, b = s["kc"].clone(), s["vc"].clone()
        call(s)
        pkv.reshape_and_cache(s["k"], s["v"], a, b, s["slots"], s["ks"], s["vs"])
        assert torch.equal(s["kc"].view(torch.uint8), a.view(torch.uint8))
        assert torch.equal(s["vc"].view(torch.uint8), b.view(torch.uint8))


def test_zero_rows_and_large_values():
    # a zero row: the norm's eps keeps it zero; bf16 values whose squares sum to near the fp32 maximum stay finite
    s = make(3, 2, 1, 128, torch.bfloat16, "same", 128, True, seed=6)
    s["q"][0, 0] = 0
    s["q"][1] *= 1e17
    out = call(s)
    assert pkv.get_device_error() == 0
    assert (out[0, 0] == 0).all()
    check(s, out)


def test_graph_replay_and_side_stream():
    s = make(64, 8, 2, 128, torch.bfloat16, "same", 128, True, seed=8)
    want = call(s)
    kc = s["kc"].clone()
    s["kc"].zero_()
    out = torch.zeros_like(want)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        call(s, out=out)
    torch.cuda.current_stream().wait_stream(st)
    live = s["slots"]
    assert torch.equal(out, want) and torch.equal(s["kc"].view(-1, 2, 128)[live], kc.view(-1, 2, 128)[live])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(s, out=out)
    out.zero_()
    s["pos"].copy_((s["pos"] + 3) % 500)   # the captured call reads its inputs anew
    g.replay()
    torch.cuda.synchronize()
    check(s, out)
