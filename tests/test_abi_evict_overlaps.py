"""pkv_evict_tokens refuses buffers that it would both read and write (CPU only).  A sequence's kv heads are
separate CTAs, so a result stored over an input changes what the others select.

The batch has more rows than the call takes, which it refuses only behind these checks: nothing is
launched on the made-up addresses, whatever the checks say."""
import itertools

import pytest

import paged_kv_cache_373_b200 as pkv
from test_abi_operators import L, evict  # noqa: F401  (the library and the call with its defaults)

S, HKV = 1 << 30, 2
# bytes, by the defaults of `evict`: tables of 8 and 4 blocks, weight rows of 128 and 64, budget 64
SIZE = dict(lens=4 * S, weights=4 * S * HKV * 128, tables=4 * S * 8, new_tables=4 * S * 4, new_lens=4 * S,
            new_weights=4 * S * HKV * 64, kept=4 * S * HKV * 64)
WRITTEN = ("new_lens", "new_weights", "kept")
BASE = {n: (i + 1) << 44 for i, n in enumerate(SIZE)}
PAIRS = [(w, o) for w, o in itertools.product(WRITTEN, SIZE)
         if w != o and not (o in WRITTEN and WRITTEN.index(o) < WRITTEN.index(w))]


def answer(L, **kw):  # noqa: F811
    return evict(L, num_seqs=S, num_kv_heads=HKV, key_cache=1 << 50, value_cache=1 << 51, **{**BASE, **kw})


def test_apart(L):  # noqa: F811
    assert answer(L) == pkv.PKV_EUNSUPPORTED and b"rows" in L.pkv_last_error_message()


@pytest.mark.parametrize("written,other", PAIRS, ids=lambda n: n)
def test_overlaps_are_refused(L, written, other):  # noqa: F811
    at = BASE[other]
    cases = [at, at + SIZE[other] - 4, at - SIZE[written] + 4]  # the same, in the other's last entry, up to its first
    if SIZE[other] > SIZE[written]:
        cases.append(at + 4)                                    # inside it
    for a in cases:
        assert answer(L, **{written: a}) == pkv.PKV_EINVAL, hex(a)
        msg = L.pkv_last_error_message()
        assert b"overlaps" in msg or b"must not be weights" in msg


@pytest.mark.parametrize("written,other", PAIRS, ids=lambda n: n)
def test_neighbours_are_not_refused(L, written, other):  # noqa: F811
    for a in (BASE[other] + SIZE[other], BASE[other] - SIZE[written]):
        assert answer(L, **{written: a}) == pkv.PKV_EUNSUPPORTED, hex(a)
