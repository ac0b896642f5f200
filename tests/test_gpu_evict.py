"""evict_tokens on the GPU.  It selects and copies: every result is compared bit for bit."""
import numpy as np
import pytest
import torch

import paged_kv_cache_373_b200 as pkv

pytestmark = pytest.mark.gpu
F16, BF16, F32, FP8 = torch.float16, torch.bfloat16, torch.float32, torch.uint8


def setup(lens, Hkv, D, bs, dtype, budget, seed, kind="heavy", extra=0, new_extra=0):
    g = torch.Generator().manual_seed(seed)
    S = len(lens)
    need = sum(-(-L // bs) for L in lens)
    nb = -(-budget // bs)
    fresh = sum(nb for L in lens if L > budget)
    NB = need + fresh + 2
    order = torch.randperm(NB, generator=g).tolist()
    width = max([-(-L // bs) for L in lens] + [1])
    t = torch.full((S, width), -1, dtype=torch.int32)
    nt = torch.full((S, nb), -1, dtype=torch.int32)
    for s, L in enumerate(lens):
        for b in range(-(-L // bs)):
            t[s, b] = order.pop()
        if L > budget:
            for b in range(nb):
                nt[s, b] = order.pop()
    size = torch.empty(0, dtype=dtype).element_size()
    kc = torch.randint(0, 256, (NB, bs, Hkv, D * size), generator=g, dtype=torch.uint8).view(dtype)
    vc = torch.randint(0, 256, (NB, bs, Hkv, D * size), generator=g, dtype=torch.uint8).view(dtype)
    W = max(lens + [1]) + extra
    if kind == "heavy":
        w = torch.exp(2 * torch.randn(S, Hkv, W, generator=g))
        w[w < 0.3] = 0
    elif kind == "ties":
        w = torch.randint(0, 4, (S, Hkv, W), generator=g).float()
    elif kind == "equal":
        w = torch.full((S, Hkv, W), 0.25)
    else:  # every kind of number
        w = torch.randint(-2 ** 31, 2 ** 31 - 1, (S, Hkv, W), generator=g, dtype=torch.int32).view(torch.float32).clone()
        for j, v in enumerate((0.0, -0.0, float("inf"), -float("inf"), float("nan"), -float("nan"), 1e-45, -1e-45)):
            w[..., j::17] = v
    d = dict(kc=kc, vc=vc, t=t, nt=nt, lens=torch.tensor(lens, dtype=torch.int32), w=w)
    d = {k: x.cuda() for k, x in d.items()}
    d["nl"] = torch.full((S,), -9, dtype=torch.int32, device="cuda")
    d["nw"] = torch.full((S, Hkv, min(budget, W) + new_extra), 123.0, device="cuda")
    d["kept"] = torch.full((S, Hkv, budget), -5, dtype=torch.int32, device="cuda")
    return d


def run(d, budget, recent, err=0):
    pkv.evict_tokens(d["kc"], d["vc"], d["t"], d["lens"], d["w"], d["nt"], d["nl"], d["nw"], d["kept"],
                     budget=budget, recent=recent)
    assert pkv.get_device_error() == err


def chosen(w, L, budget, recent):
    if L <= budget:
        return list(range(L))
    key = np.where(np.isnan(w[:L]), -np.inf, w[:L].astype(np.float64))
    isnan = np.isnan(w[:L])
    old = sorted(range(L - recent), key=lambda t: (isnan[t], -key[t], t))[:budget - recent]
    return sorted(old) + list(range(L - recent, L))


def expect(d, budget, recent):
    """The state after the call, from the state before it (CPU tensors)."""
    c = {k: x.cpu().clone() for k, x in d.items()}
    bs = c["kc"].shape[1]
    raw = lambda x: x.view(torch.uint8)
    kb, vb = raw(c["kc"]), raw(c["vc"])
    S, Hkv, W = c["w"].shape
    for s in range(S):
        L = int(c["lens"][s])
        c["nl"][s] = min(L, budget)
        for h in range(Hkv):
            ids = chosen(c["w"][s, h].numpy(), L, budget, recent)
            n = len(ids)
            c["kept"][s, h, :n] = torch.tensor(ids, dtype=torch.int32)
            c["kept"][s, h, n:] = -1
            c["nw"][s, h, :n] = c["w"][s, h][torch.tensor(ids, dtype=torch.long)]
            if L > budget:
                a, j = torch.tensor(ids), torch.arange(n)
                for x in (kb, vb):
                    x[c["nt"][s, j // bs].long(), j % bs, h] = x[c["t"][s, a // bs].long(), a % bs, h]
    return c


def same(d, c):
    for k in d:
        a, b = d[k].cpu(), c[k]
        if a.is_floating_point():
            a, b = a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8)
        assert torch.equal(a, b), k


LENS = [1, 0, 100, 101, 37, 500, 1234, 99, 4097]
CASES = [
    # lens, Hkv, D, bs, dtype, budget, recent, kind
    (LENS, 2, 128, 16, BF16, 100, 30, "heavy"),
    (LENS, 1, 64, 32, F16, 100, 0, "ties"),
    (LENS, 4, 64, 16, F32, 100, 100, "heavy"),       # only recent tokens
    (LENS, 3, 128, 32, FP8, 100, 99, "heavy"),       # one other
    (LENS, 2, 64, 16, FP8, 33, 5, "equal"),
    (LENS, 2, 128, 16, F32, 64, 10, "bits"),
    (LENS, 8, 128, 16, F16, 1, 0, "heavy"),
    (LENS, 8, 64, 16, BF16, 1, 1, "heavy"),
    (LENS, 2, 64, 32, F16, 4096, 1000, "bits"),
    ([20000, 3000, 40000], 2, 64, 16, F16, 5000, 500, "heavy"),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "H%d_D%d_b%d_%s_%d_%d_%s" % (*c[1:4], str(c[4])[6:], *c[5:]))
def test_selects_and_moves_exactly(case):
    lens, Hkv, D, bs, dtype, budget, recent, kind = case
    d = setup(lens, Hkv, D, bs, dtype, budget, 41, kind, extra=3, new_extra=2)
    want = expect(d, budget, recent)
    run(d, budget, recent)
    same(d, want)
    run(d, budget, recent)           # the old blocks are as they were: again, the same
    same(d, want)


def test_many_sequences_and_heads():
    lens = [(37 * i) % 300 for i in range(300)]
    d = setup(lens, 5, 64, 16, F16, 48, 42)
    want = expect(d, 48, 16)
    run(d, 48, 16)
    same(d, want)


def test_wrong_lengths_and_ids_are_flagged():
    mk = lambda: setup([200, 30, 90], 2, 64, 16, F16, 40, 43)
    d = mk()
    d["lens"][1] = -4
    run(d, 40, 8, pkv.DEVERR_SEQ_LEN)
    assert d["nl"].tolist() == [40, 0, 40]
    d = mk()
    d["lens"][0] = 5000              # longer than its table row: taken as far as the table goes
    run(d, 40, 8, pkv.DEVERR_SEQ_LEN)
    d = mk()
    d["nw"] = d["nw"][..., :20].contiguous()
    full = expect(dict(mk()), 40, 8)
    run(d, 40, 8, pkv.DEVERR_SEQ_LEN)
    assert torch.equal(d["nw"].cpu(), full["nw"][..., :20])
    d = mk()
    before = d["kc"].clone()
    d["nt"][0, 1] = d["kc"].shape[0]
    run(d, 40, 8, pkv.DEVERR_BLOCK_ID)
    assert torch.equal(d["kc"][d["t"][0].long()].view(torch.uint8), before[d["t"][0].long()].view(torch.uint8))
    d = mk()
    d["t"][2, 0] = -3
    d["w"][2, :, 0] = 1e9
    run(d, 40, 8, pkv.DEVERR_BLOCK_ID)
    d = mk()
    d["nt"] = d["nt"][:, :2].contiguous()      # 32 slots for a budget of 40
    run(d, 40, 8, pkv.DEVERR_SEQ_LEN)


def test_refusals():
    d = setup([200], 2, 64, 16, F16, 40, 44)
    for budget, recent in ((40, 41), (40, -1)):
        with pytest.raises(pkv.PkvError) as e:
            run(d, budget, recent)
        assert e.value.status == pkv.PKV_EINVAL
    d["nw"] = d["w"]
    with pytest.raises(pkv.PkvError):
        run(d, 40, 8)
    d["w"] = d["w"].half()
    with pytest.raises(ValueError):
        run(d, 40, 8)


def test_graph_replay():
    d = setup([500, 20, 300], 2, 128, 16, BF16, 64, 45)
    call = lambda: pkv.evict_tokens(d["kc"], d["vc"], d["t"], d["lens"], d["w"], d["nt"], d["nl"], d["nw"], d["kept"],
                                    budget=64, recent=10)
    call()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    d["w"].copy_(d["w"].flip(-1) + 1)
    want = expect(d, 64, 10)
    g.replay()
    torch.cuda.synchronize()
    same(d, want)
