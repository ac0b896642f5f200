"""Host-side refusals of the serving operators around the cache (CPU only): nothing is launched."""
import pytest

import paged_kv_cache_373_b200 as pkv
from paged_kv_cache_373_b200 import _build


@pytest.fixture(scope="module")
def L():
    _build.build()
    return pkv.lib()


def rope(L, **kw):
    a = dict(query_out=None, query=None, query_stride=1024, key=None, key_stride=256, value=None, value_stride=256,
             dtype=pkv.PKV_BF16, key_cache=None, value_cache=None, cache_dtype=pkv.PKV_BF16, slots=None,
             positions=None, cos_sin=None, max_position=100, rotary_dim=128, interleaved=0, q_weight=None,
             k_weight=None, eps=1e-6, num_tokens=4, num_blocks=16, block_size=16, num_heads=8, num_kv_heads=2,
             head_dim=128, k_scale=None, v_scale=None, stream=None)
    assert set(kw) <= set(a)
    a.update(kw)
    return L.pkv_qk_norm_rope_and_cache(*a.values())


def test_rope_refusals(L):
    assert rope(L, num_tokens=0) == pkv.PKV_OK
    assert rope(L) == pkv.PKV_EINVAL and b"null" in L.pkv_last_error_message()
    assert rope(L, num_tokens=-1) == pkv.PKV_EINVAL
    assert rope(L, head_dim=96) == pkv.PKV_EUNSUPPORTED
    assert rope(L, rotary_dim=40) == pkv.PKV_EUNSUPPORTED
    assert rope(L, rotary_dim=144) == pkv.PKV_EUNSUPPORTED
    assert rope(L, rotary_dim=-16) == pkv.PKV_EUNSUPPORTED
    assert rope(L, num_heads=7) == pkv.PKV_EINVAL
    assert rope(L, cache_dtype=pkv.PKV_F16) == pkv.PKV_EUNSUPPORTED
    assert rope(L, dtype=pkv.PKV_FP8_E4M3) == pkv.PKV_EUNSUPPORTED
    assert rope(L, dtype=9) == pkv.PKV_EINVAL
    assert rope(L, query_stride=1023) == pkv.PKV_EINVAL        # shorter than the row
    assert rope(L, query_stride=1028) == pkv.PKV_EINVAL        # not 16 bytes
    assert rope(L, value_stride=0) == pkv.PKV_EINVAL
    assert rope(L, q_weight=64) == pkv.PKV_EINVAL              # one weight without the other
    assert rope(L, q_weight=64, k_weight=64, eps=-1.0) == pkv.PKV_EINVAL
    assert rope(L, q_weight=64, k_weight=64, eps=float("nan")) == pkv.PKV_EINVAL
    assert rope(L, max_position=0) == pkv.PKV_EINVAL
    p = dict(query_out=64, query=64, key=64, value=64, key_cache=64, value_cache=64, slots=64)
    assert rope(L, **p) == pkv.PKV_EINVAL and b"positions" in L.pkv_last_error_message()
    assert rope(L, cache_dtype=pkv.PKV_FP8_E4M3, **{**p, "positions": 64, "cos_sin": 64}) == pkv.PKV_EINVAL
    assert b"k_scale" in L.pkv_last_error_message()
    assert rope(L, **{**p, "positions": 64, "cos_sin": 68}) == pkv.PKV_EINVAL
    assert b"aligned" in L.pkv_last_error_message()
    assert rope(L, query_stride=1536, **{**p, "positions": 64, "cos_sin": 64}) == pkv.PKV_EINVAL
    assert b"in place" in L.pkv_last_error_message()


def decode(L, **kw):
    a = dict(out=None, query=None, q_dtype=pkv.PKV_F16, key_cache=None, value_cache=None, cache_dtype=pkv.PKV_F16,
             tables=None, max_blocks=4, lens=None, num_seqs=2, num_heads=8, num_kv_heads=2, head_dim=128,
             block_size=16, num_blocks=64, scale=0.1, softcap=0.0, window=0, slopes=None, prefix=None, k_scale=None,
             v_scale=None, workspace=None, workspace_bytes=0, num_ctas=4, stream=None)
    assert set(kw) <= set(a)
    a.update(kw)
    return L.pkv_paged_attention_decode_scoremod(*a.values())


def test_decode_scoremod_refusals(L):
    assert decode(L, num_seqs=0) == pkv.PKV_OK
    assert decode(L) == pkv.PKV_EINVAL and b"null" in L.pkv_last_error_message()
    for cap in (-1.0, float("nan"), float("inf"), 1e-40, 3e38):
        assert decode(L, softcap=cap, num_seqs=0) == pkv.PKV_EINVAL, cap
    assert decode(L, softcap=1e-3, num_seqs=0) == pkv.PKV_OK
    assert decode(L, window=-1, num_seqs=0) == pkv.PKV_EINVAL
    assert decode(L, head_dim=96) == pkv.PKV_EUNSUPPORTED
    assert decode(L, block_size=8) == pkv.PKV_EUNSUPPORTED
    assert decode(L, cache_dtype=pkv.PKV_FP8_E4M3, q_dtype=pkv.PKV_F32) == pkv.PKV_EUNSUPPORTED
    p = dict(out=64, query=64, key_cache=64, value_cache=64, tables=64, lens=64, workspace=64)
    assert decode(L, **p) == pkv.PKV_EINVAL and b"workspace" in L.pkv_last_error_message()


def weights(L, **kw):
    a = dict(out=None, weights_out=64, weights_in=None, weight_len=100, query=None, q_dtype=pkv.PKV_F16,
             key_cache=None, value_cache=None, cache_dtype=pkv.PKV_F16, tables=None, max_blocks=4, lens=None,
             num_seqs=2, num_heads=8, num_kv_heads=2, head_dim=128, block_size=16, num_blocks=64, scale=0.1,
             k_scale=None, v_scale=None, workspace=None, workspace_bytes=0, num_ctas=4, stream=None)
    assert set(kw) <= set(a)
    a.update(kw)
    return L.pkv_paged_attention_decode_weights(*a.values())


def test_decode_weights_refusals(L):
    assert weights(L, num_seqs=0) == pkv.PKV_OK
    assert weights(L, weight_len=0) == pkv.PKV_EINVAL
    assert weights(L, weights_out=None) == pkv.PKV_EINVAL
    assert weights(L) == pkv.PKV_EINVAL and b"null" in L.pkv_last_error_message()
    # a workspace that holds the split scratch but not the scores
    n = pkv.paged_attention_workspace_bytes(2, 8, 2, 128, 4)
    need = pkv.paged_attention_weights_workspace_bytes(2, 8, 2, 128, 64, 4)
    assert need >= n + 2 * 8 * 64 * 4
    assert pkv.paged_attention_weights_workspace_bytes(2, 7, 2, 128, 64, 4) == 0
    assert pkv.paged_attention_weights_workspace_bytes(2, 8, 2, 128, 0, 4) == 0


def prefill(L, **kw):
    a = dict(out=None, query=None, q_dtype=pkv.PKV_BF16, key_cache=None, value_cache=None, cache_dtype=pkv.PKV_BF16,
             tables=None, max_blocks=4, lens=None, start=None, num_seqs=2, tokens=10, num_heads=8, num_kv_heads=4,
             head_dim=128, block_size=16, num_blocks=64, scale=0.1, softcap=0.0, window=0, slopes=None, prefix=None,
             stream=None)
    assert set(kw) <= set(a)
    a.update(kw)
    return L.pkv_paged_prefill_scoremod(*a.values())


def test_prefill_scoremod_refusals(L):
    assert prefill(L, tokens=0) == pkv.PKV_OK
    assert prefill(L) == pkv.PKV_EINVAL and b"null" in L.pkv_last_error_message()
    assert prefill(L, num_heads=12) == pkv.PKV_EUNSUPPORTED
    assert prefill(L, cache_dtype=pkv.PKV_FP8_E4M3) == pkv.PKV_EUNSUPPORTED
    assert prefill(L, scale=0.0) == pkv.PKV_EINVAL
    assert prefill(L, tokens=0, softcap=-2.0) == pkv.PKV_EINVAL
    assert prefill(L, tokens=0, window=-2) == pkv.PKV_EINVAL
    assert prefill(L, tokens=0, max_blocks=1 << 27) == pkv.PKV_EUNSUPPORTED
    # a timeout test armed for this thread's next prefill is consumed by a refused call
    assert L.pkv_testing_prefill_timeout(0, 1_000_000) == pkv.PKV_OK
    assert prefill(L, scale=0.0) == pkv.PKV_EINVAL


def evict(L, **kw):
    a = dict(key_cache=None, value_cache=None, cache_dtype=pkv.PKV_BF16, tables=None, max_blocks=8, lens=None,
             weights=None, weight_len=128, new_tables=None, new_max_blocks=4, new_lens=None, new_weights=None,
             new_weight_len=64, kept=None, budget=64, recent=16, num_seqs=2, num_kv_heads=2, head_dim=128,
             block_size=16, num_blocks=64, stream=None)
    assert set(kw) <= set(a)
    a.update(kw)
    return L.pkv_evict_tokens(*a.values())


def test_evict_refusals(L):
    assert evict(L, num_seqs=0) == pkv.PKV_OK
    assert evict(L) == pkv.PKV_EINVAL and b"null" in L.pkv_last_error_message()
    assert evict(L, num_seqs=-1) == pkv.PKV_EINVAL
    assert evict(L, budget=0) == pkv.PKV_EINVAL
    assert evict(L, recent=65) == pkv.PKV_EINVAL
    assert evict(L, recent=-1) == pkv.PKV_EINVAL
    assert evict(L, head_dim=80) == pkv.PKV_EUNSUPPORTED
    assert evict(L, block_size=64) == pkv.PKV_EUNSUPPORTED
    assert evict(L, cache_dtype=7) == pkv.PKV_EINVAL
    assert evict(L, weight_len=0) == pkv.PKV_EINVAL
    assert evict(L, new_weight_len=-1) == pkv.PKV_EINVAL
    assert evict(L, max_blocks=0) == pkv.PKV_EINVAL
    assert evict(L, max_blocks=1 << 27) == pkv.PKV_EINVAL               # past 32-bit tokens
    assert evict(L, max_blocks=(1 << 26) + 1) == pkv.PKV_EUNSUPPORTED
    p = dict(key_cache=64, value_cache=64, tables=64, lens=64, weights=64, new_tables=64, new_lens=64,
             new_weights=64, kept=64)
    assert evict(L, **p) == pkv.PKV_EINVAL and b"must not be weights" in L.pkv_last_error_message()
    assert evict(L, **{**p, "new_weights": 128, "key_cache": 72}) == pkv.PKV_EINVAL
    assert b"aligned" in L.pkv_last_error_message()
