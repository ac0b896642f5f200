"""The serving operators on a pool of more than 2^31 elements per cache, its last blocks in use: the same bits
as on a small pool that holds the same rows.  And two captured graphs that share one workspace."""
import pytest
import torch

import paged_kv_cache_373_b200 as pkv
from scoremod_ref import build, cuda

pytestmark = pytest.mark.gpu
HQ, HKV, D, BS = 16, 8, 128, 16
LENS = [700, 33, 1200]


def test_blocks_past_two_to_the_31_elements():
    d = cuda(build(LENS, HKV, D, BS, torch.bfloat16, 21, spare=30))
    used = d["kc"].shape[0]
    NB = 2 ** 31 // (BS * HKV * D) + used + 1000
    big = {}
    for name in ("kc", "vc"):  # the last blocks hold the small pool's rows, the others what the memory held
        big[name] = torch.empty(NB, BS, HKV, D, dtype=torch.bfloat16, device="cuda")
        big[name][NB - used:] = d[name]
    assert big["kc"][NB - used:].storage_offset() > 2 ** 31
    shift = NB - used
    high = torch.where(d["tables"] >= 0, d["tables"] + shift, -1)
    g = torch.Generator().manual_seed(22)
    q = torch.randn(len(LENS), HQ, D, generator=g).to(torch.bfloat16).cuda()
    lens = d["lens"]
    pools = [(d["kc"], d["vc"], d["tables"], 0), (big["kc"], big["vc"], high, shift)]

    # each sequence's last row, written through its slot
    rows = lens.long() - 1
    k, v = (torch.randn(len(LENS), HKV, D, generator=g).to(torch.bfloat16).cuda() for _ in range(2))
    angle = torch.rand(1300, D, generator=g).cuda()
    got = []
    for kc, vc, tables, off in pools:
        slots = tables[torch.arange(len(LENS), device="cuda"), rows // BS].long() * BS + rows % BS
        q_out = torch.empty_like(q)
        pkv.qk_norm_rope_and_cache(q_out, q, k, v, kc, vc, slots, rows, angle)
        got.append((q_out, kc[off:off + used].clone(), vc[off:off + used].clone()))
    for a, b in zip(*got):
        assert torch.equal(a.view(torch.int16), b.view(torch.int16))

    chunks = [5, 33, 300]
    start = torch.tensor([0, 5, 38, 338], dtype=torch.int32, device="cuda")
    qc = torch.randn(338, HQ, D, generator=g).to(torch.bfloat16).cuda()
    prefix = torch.tensor([4, 0, 70], dtype=torch.int32, device="cuda")
    budget = 64
    got = []
    for kc, vc, tables, off in pools:
        a, b, c = torch.empty_like(q), torch.empty_like(q), torch.empty_like(qc)
        w = torch.zeros(len(LENS), HKV, 1200, device="cuda")
        pkv.paged_attention_decode_scoremod(a, q, kc, vc, tables, lens, 0.09, softcap=20.0, window=100, prefix_lens=prefix)
        pkv.paged_attention_decode_weights(b, w, q, kc, vc, tables, lens, 0.09, weights=w)
        pkv.paged_prefill_scoremod(c, qc, kc, vc, tables, lens, start, 0.09, softcap=20.0, window=100, prefix_lens=prefix)
        # blocks that nobody uses: the small pool's spares
        mine = set(d["tables"][d["tables"] >= 0].tolist())
        free = [i for i in range(used) if i not in mine]
        fresh = torch.tensor(free[:12], dtype=torch.int32).view(3, 4).cuda() + off
        kept = torch.empty(3, HKV, budget, dtype=torch.int32, device="cuda")
        new_w, new_lens = torch.zeros(3, HKV, budget, device="cuda"), torch.empty_like(lens)
        pkv.evict_tokens(kc, vc, tables, lens, w, fresh, new_lens, new_w, kept, budget=budget, recent=20)
        assert pkv.get_device_error() == 0
        got.append((a, b, c, w, kept, new_w, new_lens, kc[fresh[[0, 2]].long()], vc[fresh[[0, 2]].long()]))
    for a, b in zip(*got):
        assert torch.equal(a, b)
    assert sum(chunks) == 338 and not torch.isnan(got[0][2].float()).any()


def test_two_graphs_share_a_workspace():
    """Graphs that are replayed one after the other may use one workspace: nothing in it outlives a call."""
    out, graphs = [], []
    n = pkv.paged_attention_weights_workspace_bytes(3, HQ, HKV, D, 1200)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    calls = []
    for seed in (31, 32):
        d = cuda(build(LENS if seed == 31 else [9, 1100, 400], HKV, D, BS, torch.float16, seed))
        q = torch.randn(3, HQ, D, generator=torch.Generator().manual_seed(seed)).to(torch.float16).cuda()
        o, c, w = torch.empty_like(q), torch.empty_like(q), torch.zeros(3, HKV, 1200, device="cuda")

        def call(d=d, q=q, o=o, c=c, w=w):
            pkv.paged_attention_decode_weights(o, w, q, d["kc"], d["vc"], d["tables"], d["lens"], 0.09, workspace=ws)
            pkv.paged_attention_decode_scoremod(c, q, d["kc"], d["vc"], d["tables"], d["lens"], 0.09, window=300,
                                                workspace=ws)
        call()
        torch.cuda.synchronize()
        out.append([x.clone() for x in (o, c, w)])
        calls.append((call, (o, c, w)))
    for call, _ in calls:
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            call()
        graphs.append(gr)
    for i in (0, 1, 1, 0, 1):
        for x in calls[i][1]:
            x.zero_()
        ws.fill_(0xFF if i else 0x7F)  # (NaN or large numbers: no call may read what it has not written)
        graphs[i].replay()
        for a, b in zip(calls[i][1], out[i]):
            assert torch.equal(a, b)
    assert pkv.get_device_error() == 0
