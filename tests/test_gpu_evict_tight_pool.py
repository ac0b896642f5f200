"""Eviction in a pool that has no room for the whole batch's fresh blocks: sequence by sequence on one stream,
the later ones into blocks that the earlier ones' calls have just copied from (pkv_block_manager.h)."""
import pytest
import torch

import paged_kv_cache_373_b200 as pkv

pytestmark = pytest.mark.gpu
BS, HKV, D = 16, 4, 64


@pytest.mark.parametrize("lens,budget,spare", [([700, 650, 90, 512], 80, 5), ([3000, 2999, 2500], 1000, 63)])
def test_one_sequence_at_a_time(lens, budget, spare):
    per = -(-budget // BS)
    assert per <= spare < per * sum(L > budget for L in lens)
    nb = sum(-(-L // BS) for L in lens) + spare
    bm = pkv.HostBlockManager(nb, BS, prefix_cache=False)
    sids = [bm.add_sequence(range(1000 * i, 1000 * i + L))[0] for i, L in enumerate(lens)]
    width, S = max(-(-L // BS) for L in lens), len(lens)
    g = torch.Generator().manual_seed(3)
    kc, vc = (torch.randn(nb, BS, HKV, D, generator=g).half().cuda() for _ in range(2))
    w = torch.rand(S, HKV, max(lens), generator=g).cuda()
    tables, _ = bm.batch_tables(sids, width)
    rows = [[c[tables[s, :-(-L // BS)].long()].reshape(-1, HKV, D)[:L].clone() for c in (kc, vc)]
            for s, L in enumerate(lens)]
    with pytest.raises(pkv.PkvError) as e:
        bm.evict_batch(sids, budget)
    assert e.value.status == pkv.PKV_ENOBLOCKS
    recent, kept = budget // 4, torch.empty(S, HKV, budget, dtype=torch.int32, device="cuda")
    nl, nw = torch.empty(S, dtype=torch.int32, device="cuda"), torch.empty(S, HKV, budget, device="cuda")
    torch.cuda.synchronize()
    copies = []  # (device copies made first: nothing below waits for the device)
    for i, sid in enumerate(sids):
        old, old_lens = bm.batch_tables([sid], width)
        new, _ = bm.evict_batch([sid], budget)
        copies.append([x.pin_memory().cuda(non_blocking=True) for x in (old, old_lens, new)])
        pkv.evict_tokens(kc, vc, copies[-1][0], copies[-1][1], w[i:i + 1], copies[-1][2], nl[i:i + 1], nw[i:i + 1],
                         kept[i:i + 1], budget=budget, recent=recent)
    assert pkv.get_device_error() == 0
    tables, new_lens = bm.batch_tables(sids, width)
    assert new_lens.tolist() == nl.tolist() == [min(L, budget) for L in lens]
    for s, L in enumerate(lens):
        n = min(L, budget)
        for c, r in zip((kc, vc), rows[s]):
            now = c[tables[s, :-(-n // BS)].long()].reshape(-1, HKV, D)[:n]
            for h in range(HKV):
                k = kept[s, h, :n].long()
                assert torch.equal(now[:, h], r[k, h])
                assert torch.equal(nw[s, h, :n], w[s, h, k])
        if L > budget:
            for h in range(HKV):  # the heaviest of the others, in order (distinct weights)
                top = w[s, h, :L - recent].topk(budget - recent).indices.sort().values
                assert torch.equal(kept[s, h, :budget - recent].long(), top)
