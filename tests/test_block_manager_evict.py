"""HostBlockManager.evict_batch: fresh blocks for shortened sequences (CPU only)."""
import pytest

import paged_kv_cache_373_b200 as pkv
from paged_kv_cache_373_b200 import _build


@pytest.fixture(scope="module", autouse=True)
def built():
    _build.build()


def test_fresh_blocks_are_disjoint_from_everything_the_batch_reads():
    bm = pkv.HostBlockManager(40, 4, prefix_cache=False)
    a, _ = bm.add_sequence(range(41))      # 11 blocks
    b, _ = bm.add_sequence(range(5))       # stays
    c, _ = bm.add_sequence(range(80, 120))  # 10 blocks
    old, lens = bm.batch_tables([a, b, c], 12)
    new, new_lens = bm.evict_batch([a, b, c], 18, 6)
    assert new_lens.tolist() == [18, 5, 18]
    assert new.shape == (3, 6) and (new[1] == -1).all() and (new[[0, 2], 5] == -1).all()
    fresh = set(new[new >= 0].tolist())
    assert len(fresh) == 10 and not fresh & set(old[old >= 0].tolist())
    t, l = bm.batch_tables([a, b, c], 6)
    assert l.tolist() == [18, 5, 18]
    assert t[0, :5].tolist() == new[0, :5].tolist() and t[1, :2].tolist() == old[1, :2].tolist()
    assert bm.stats()["used_blocks"] == 12 and bm.stats()["free_blocks"] == 28
    # the shortened sequence goes on from its new length, in its new last block
    slot, cow = bm.append_token(a, 7)
    assert cow is None and slot == int(new[0, 4]) * 4 + 2


def test_shared_blocks_stay_with_the_other_holder():
    bm = pkv.HostBlockManager(30, 4, prefix_cache=False)
    p, _ = bm.add_sequence(range(32))
    q = bm.fork(p)
    before = bm.block_table(q)
    bm.evict_batch([p], 10)
    assert bm.block_table(q) == before
    assert bm.stats()["used_blocks"] == 8 + 3
    bm.free_sequence(p)
    bm.free_sequence(q)
    assert bm.stats()["free_blocks"] == 30


def test_all_or_nothing_and_bad_arguments():
    bm = pkv.HostBlockManager(12, 4, prefix_cache=False)
    a, _ = bm.add_sequence(range(20))
    b, _ = bm.add_sequence(range(20))      # 2 blocks left, 4 needed
    before = (bm.block_table(a), bm.block_table(b), bm.stats())
    with pytest.raises(pkv.PkvError) as e:
        bm.evict_batch([a, b], 8)
    assert e.value.status == pkv.PKV_ENOBLOCKS
    assert before == (bm.block_table(a), bm.block_table(b), bm.stats())
    for bad in (lambda: bm.evict_batch([a, a], 8), lambda: bm.evict_batch([a, 99], 8),
                lambda: bm.evict_batch([a], 0, 1), lambda: bm.evict_batch([a], 8, 1)):
        with pytest.raises(pkv.PkvError) as e:
            bad()
        assert e.value.status == pkv.PKV_EINVAL
    assert before == (bm.block_table(a), bm.block_table(b), bm.stats())
    t, lens = bm.evict_batch([a], 20)
    assert lens.tolist() == [20] and (t == -1).all()
    assert bm.evict_batch([], 4)[1].numel() == 0


def test_prefix_cache_keeps_the_old_content_and_never_the_new():
    bm = pkv.HostBlockManager(30, 4, prefix_cache=True)
    prompt = list(range(24))
    a, _ = bm.add_sequence(prompt)
    bm.evict_batch([a], 10)
    b, cached = bm.add_sequence(prompt)    # the parked originals still answer
    assert cached == 24
    for tok in range(8):                   # blocks that the shortened sequence fills get no key
        bm.append_token(a, tok)
    with pytest.raises(pkv.PkvError):
        bm.block_key(a, 0)
    child = bm.fork(a)
    for tok in range(8):
        bm.append_token(child, tok)
    assert bm.stats()["cached_blocks"] == 6
