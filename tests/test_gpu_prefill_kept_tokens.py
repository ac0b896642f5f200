"""A causal prompt with a window and kept first tokens, as the decode form attends it step by step, through
paged_prefill_scoremod: a chunk with rows below the prefix lists its sequence twice (pkv.h)."""
import numpy as np
import pytest
import torch

import paged_kv_cache_373_b200 as pkv
from scoremod_ref import assert_near, build, cuda

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("ctx,chunk,keep,window", [(0, 400, 4, 64), (0, 300, 130, 130), (3, 200, 40, 50),
                                                    (0, 30, 64, 100), (500, 100, 64, 90)])
def test_listed_twice(ctx, chunk, keep, window):
    Hq, Hkv, D, bs, scale = 8, 4, 64, 16, 0.125
    L = ctx + chunk
    d = cuda(build([L], Hkv, D, bs, torch.bfloat16, 91))
    q = torch.randn(chunk, Hq, D, generator=torch.Generator().manual_seed(92)).bfloat16().cuda()
    below = min(max(keep - ctx, 0), chunk)  # rows below the prefix
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")
    out = torch.empty_like(q)
    pkv.paged_prefill_scoremod(out, q, d["kc"], d["vc"], d["tables"].expand(2, -1).contiguous(), i32(ctx + below, L),
                               i32(0, below, chunk), scale, window=window, prefix_lens=i32(0, keep))
    assert pkv.get_device_error() == 0
    # the definition, dense
    pos, t = np.arange(ctx, L), np.arange(L)
    vis = (t[None] <= pos[:, None]) & ((pos[:, None] - t[None] < window) | (t[None] < keep))
    qn, k, v = q.double().cpu().numpy(), d["K"][0].repeat(Hq // Hkv, 1), d["V"][0].repeat(Hq // Hkv, 1)
    x = np.where(vis[:, None], np.einsum("chd,thd->cht", qn, k) * scale, -np.inf)
    p = np.exp(x - x.max(-1, keepdims=True))
    ref = np.einsum("cht,thd->chd", p / p.sum(-1, keepdims=True), v)
    # scoremod_ref's bound: scores off by D 2^-23 scale sum|q k| and 8 roundings of them (dx), P in two bf16 parts
    # (2^-16 each way), fp32 sums of L terms, one rounding of the output (bf16: 2^-8)
    dx = (D + 8) * 2.0 ** -23 * scale * np.einsum("chd,thd->cht", np.abs(qn), np.abs(k)).max(-1)
    A = np.einsum("cht,thd->chd", p / p.sum(-1, keepdims=True), np.abs(v))
    bound = A * (2 * np.expm1(dx) + 2.0 ** -19 + L * 2.0 ** -23 + 2 * 2.0 ** -16)[..., None] + 2.0 ** -8 * np.abs(ref)
    assert_near(out, ref, bound, f"{chunk} rows at {ctx}, {keep} kept, window {window}")
    # and row by row the decode form
    for i in sorted({0, below, chunk // 2, chunk - 1} - {chunk}):
        o = torch.empty(1, Hq, D, dtype=q.dtype, device="cuda")
        pkv.paged_attention_decode_scoremod(o, q[i:i + 1].contiguous(), d["kc"], d["vc"], d["tables"], i32(ctx + i + 1),
                                            scale, window=window, prefix_lens=i32(keep))
        assert_near(o, ref[i:i + 1], bound[i:i + 1], f"decode of row {i}")
