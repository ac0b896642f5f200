"""A query_start that decreases or leaves the call's rows is flagged, and no row outside the call is written,
by either prefill call.  (`out` is followed by guard rows in the same buffer.)"""
import numpy as np
import pytest
import torch

import paged_kv_cache_373_b200 as pkv
from scoremod_ref import assert_near, attend, build, cuda

pytestmark = pytest.mark.gpu
T, L, HKV, D, BS, SCALE = 300, 640, 4, 64, 16, 0.125
BIG = 2 ** 31 - 1

# query_start of two sequences, and the sequence whose rows must be right (-1: none is valid)
CASES = [([0, 450, T], -1), ([-30, 100, T], 1), ([0, 100, 400], 0), ([0, 300, 301], 0), ([0, BIG, T], -1),
         ([-BIG - 1, BIG, T], -1), ([-1, 300, 300], -1), ([BIG - 5, BIG, 2], -1), ([100, 0, T], 1), ([200, 100, 250], 1)]


@pytest.mark.parametrize("starts,right", CASES, ids=lambda x: "_".join(map(str, x)) if isinstance(x, list) else "")
@pytest.mark.parametrize("call", ["plain", "scoremod", "bias"])
@pytest.mark.parametrize("empty", [0, 40])  # sequences without rows between: the search by length ends at 32
@pytest.mark.parametrize("g", [1, 16])      # few units, and more than SMs
def test_flagged_and_nothing_outside_written(starts, right, call, empty, g):
    d = cuda(build([L, L], HKV, D, BS, torch.float16, 95))
    Hq, S = HKV * g, 2 + empty
    q = torch.randn(T, Hq, D, generator=torch.Generator().manual_seed(96)).half().cuda()
    room = torch.full((1024, Hq, D), 9.0, dtype=torch.float16, device="cuda")
    out = room[400:400 + T]
    tables = torch.full((S, d["tables"].shape[1]), -1, dtype=torch.int32, device="cuda")
    tables[[0, S - 1]] = d["tables"]
    lens = torch.zeros(S, dtype=torch.int32, device="cuda")
    lens[[0, S - 1]] = L
    qs = torch.tensor(starts[:2] + [starts[1]] * empty + starts[2:], dtype=torch.int32, device="cuda")
    slopes = torch.linspace(0.02, 0.7, Hq).cuda()
    if call == "plain":
        pkv.paged_prefill(out, q, d["kc"], d["vc"], tables, lens, qs, SCALE)
    else:
        pkv.paged_prefill_scoremod(out, q, d["kc"], d["vc"], tables, lens, qs, SCALE,
                                   alibi_slopes=slopes if call == "bias" else None)
    assert pkv.get_device_error() == pkv.DEVERR_SEQ_LEN
    written = torch.zeros(1024, dtype=torch.bool, device="cuda")
    if right >= 0:
        a, b = starts[right], starts[right + 1]
        written[400 + a:400 + b] = True
        ref, bound, _, _ = attend(q[a:b].double().cpu().numpy(), d["K"][right], d["V"][right], np.arange(L - (b - a), L),
                                  SCALE, torch.float16, torch.float16,
                                  slopes=slopes.double().cpu().numpy() if call == "bias" else None)
        assert_near(out[a:b], ref, bound, "the valid sequence")
    assert (room[~written] == 9).all()
