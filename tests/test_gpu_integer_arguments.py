"""Integers that do not fit a C int are refused, not cut to their low 32 bits."""
import pytest
import torch

import paged_kv_cache_373_b200 as pkv
from scoremod_ref import build, cuda

pytestmark = pytest.mark.gpu
WIDE = [2 ** 32 + 1, 2 ** 31, -2 ** 32, -2 ** 31 - 1, 2 ** 63]


@pytest.mark.parametrize("x", WIDE)
def test_refused(x):
    d = cuda(build([40, 7], 2, 64, 16, torch.float16, 81))
    q = torch.randn(2, 4, 64, device="cuda").half()
    out, w = torch.full_like(q, 3.0), torch.full((2, 2, 64), 3.0, device="cuda")
    start = torch.tensor([0, 1, 2], dtype=torch.int32, device="cuda")
    args = d["kc"], d["vc"], d["tables"], d["lens"]
    ws = torch.empty(1 << 24, dtype=torch.uint8, device="cuda")
    with pytest.raises(ValueError, match="window"):
        pkv.paged_attention_decode_scoremod(out, q, *args, 0.1, window=x)
    with pytest.raises(ValueError, match="num_ctas"):
        pkv.paged_attention_decode_scoremod(out, q, *args, 0.1, num_ctas=x, workspace=ws)
    with pytest.raises(ValueError, match="window"):
        pkv.paged_prefill_scoremod(out, q, *args, start, 0.1, window=x)
    with pytest.raises(ValueError, match="num_ctas"):
        pkv.paged_attention_decode_weights(out, w, q, *args, 0.1, num_ctas=x, workspace=ws)
    kept = torch.full((2, 2, 16), 3, dtype=torch.int32, device="cuda")
    lens, nw = torch.full((2,), 3, dtype=torch.int32, device="cuda"), torch.full((2, 2, 16), 3.0, device="cuda")
    for name, kw in (("budget", dict(budget=x, recent=4)), ("recent", dict(budget=16, recent=x))):
        with pytest.raises(ValueError, match=name):
            pkv.evict_tokens(*args, w, d["tables"][:, :1].contiguous(), lens, nw, kept, **kw)
    torch.cuda.synchronize()
    for t in (out, w, nw, kept, lens):
        assert (t == 3).all()
