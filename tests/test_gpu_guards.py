"""Guards that a refused call alone does not exercise: a workspace that holds the split scratch but not the
scores, and a timeout test that a refused call uses up."""
import pytest
import torch

import paged_kv_cache_373_b200 as pkv
from scoremod_ref import build, cuda
from test_gpu_decode_weights import check, setup

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16], ids=["f16", "bf16"])
def test_weights_workspace_to_the_byte(dtype):
    lens, Hq, Hkv, D, bs, ctas = [300, 20, 77], 8, 2, 64, 16, 4
    d = setup(lens, Hq, Hkv, D, bs, dtype, dtype, 27)
    width = d["tables"].shape[1] * bs
    need = pkv.paged_attention_weights_workspace_bytes(3, Hq, Hkv, D, width, ctas)
    split = pkv.paged_attention_workspace_bytes(3, Hq, Hkv, D, ctas)
    assert need >= split + 3 * Hq * width * 4
    room = torch.full((need + 4096,), 0xAB, dtype=torch.uint8, device="cuda")
    out, wo = torch.full_like(d["q"], 5.0), torch.full_like(d["w"], 77.0)

    def call(n):
        pkv.paged_attention_decode_weights(out, wo, d["q"], d["kc"], d["vc"], d["tables"], d["lens"], 0.1,
                                           weights=d["w"], workspace=room[:n], num_ctas=ctas)
    for n in (split, need - 1):
        with pytest.raises(pkv.PkvError, match=f"workspace too small: {n} < {need}"):
            call(n)
    torch.cuda.synchronize()
    assert (out == 5).all() and (wo == 77).all() and (room == 0xAB).all()
    call(need)  # enough, and nothing behind it is written
    assert pkv.get_device_error() == 0
    check(d, out, wo, 0.1, d["w"])
    assert (room[need:] == 0xAB).all()


def test_a_refused_prefill_uses_up_the_timeout_test():
    d = cuda(build([200], 4, 64, 16, torch.bfloat16, 29))
    q = torch.randn(200, 8, 64, device="cuda").bfloat16()
    start = torch.tensor([0, 200], dtype=torch.int32, device="cuda")
    args = q, d["kc"], d["vc"], d["tables"], d["lens"], start
    want, out = torch.empty_like(q), torch.empty_like(q)
    pkv.paged_prefill_scoremod(want, *args, 0.1, softcap=5.0)
    assert pkv.get_device_error() == 0
    for bad in (dict(scale=0.0), dict(scale=0.1, softcap=-1.0), dict(scale=0.1, window=-1)):
        assert pkv.lib().pkv_testing_prefill_timeout(0, 1_000_000) == pkv.PKV_OK
        with pytest.raises(pkv.PkvError):
            pkv.paged_prefill_scoremod(out, *args, **bad)
        out.fill_(float("nan"))
        pkv.paged_prefill_scoremod(out, *args, 0.1, softcap=5.0)
        assert pkv.get_device_error() == 0
        assert torch.equal(out, want)
