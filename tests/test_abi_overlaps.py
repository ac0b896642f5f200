"""Results that would be stored over rows still to be read are refused by the norm + rotary call and by decode
with weights.  CPU only: the addresses are made up, and an accepted call ends at the missing device, before
anything is launched."""
import pytest
import torch

import paged_kv_cache_373_b200 as pkv
from test_abi_operators import L, rope, weights  # noqa: F401

pytestmark = pytest.mark.skipif(torch.cuda.is_available(), reason="made-up addresses")
AT = 1 << 30


def overlaps(out, rows, stride, row, n, out_row):
    return any(rows + i * stride < out + n * out_row and out < rows + i * stride + row for i in range(n))


@pytest.mark.parametrize("tokens", [1, 2, 5])
@pytest.mark.parametrize("extra", [0, 16, 5000])
def test_rope(L, tokens, extra):  # noqa: F811
    """bf16, 2 / 1 heads of 64: rows of 256 and 128 bytes; query, key and value each in turn near query_out."""
    seen = set()
    for which, row in (("query", 256), ("key", 128), ("value", 128)):
        stride = row + extra
        if stride % 16:
            stride += 16 - stride % 16
        for off in sorted({d + m for d in (0, stride, tokens * stride, -256 * tokens, row, row - 256 * tokens)
                           for m in (-16, 0, 16)}):
            p = {n: AT + (i + 2) * (1 << 24) for i, n in enumerate(("query", "key", "value"))}
            p[which] = AT - off
            kw = {f"{n}_stride": (128 if n == "query" else 64) for n in p}
            kw[f"{which}_stride"] = stride // 2
            st = rope(L, query_out=AT, **p, **kw, key_cache=1 << 40, value_cache=1 << 41, slots=1 << 42, positions=1 << 43,
                      cos_sin=1 << 44, rotary_dim=64, head_dim=64, num_heads=2, num_kv_heads=1, num_tokens=tokens)
            msg = L.pkv_last_error_message()
            if which == "query" and off == 0:  # in place: only a contiguous query
                want = stride != 256
                assert (st == pkv.PKV_EINVAL) == want and (not want or b"in place" in msg)
                continue
            want = overlaps(AT, p[which], stride, row, tokens, 256)
            seen.add(want)
            assert (st == pkv.PKV_EINVAL) == want, (which, off, msg)
            assert want or st == pkv.PKV_ECUDA
            assert not want or f"query_out overlaps {which}".encode() in msg
    assert seen == {True, False}


def test_weights(L):  # noqa: F811
    p = dict(out=1 << 40, query=1 << 41, key_cache=1 << 42, value_cache=1 << 43, tables=1 << 44, lens=1 << 45,
             workspace=1 << 46, workspace_bytes=1 << 30, weight_len=100)
    n = 2 * 2 * 100 * 4
    for off in (4, -4, n - 4, 4 - n, 16):
        assert weights(L, **p, weights_out=AT, weights_in=AT + off) == pkv.PKV_EINVAL, off
        assert b"weights_in overlaps weights_out" in L.pkv_last_error_message()
    for off in (0, n, -n):
        assert weights(L, **p, weights_out=AT, weights_in=AT + off) == pkv.PKV_ECUDA, off
