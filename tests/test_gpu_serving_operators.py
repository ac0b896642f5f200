"""The serving operators together, as a step loop uses them: a prompt's chunks go through
qk_norm_rope_and_cache and paged_prefill_scoremod, decode steps accumulate weights, evict_tokens
shortens the sequences into blocks of HostBlockManager.evict_batch, and decoding goes on over
the shortened cache, with positions that keep counting.  Every step is checked against fp64 on the
state that the GPU holds before it (bounds as in the operators' own tests)."""
import numpy as np
import pytest
import torch

import paged_kv_cache_373_b200 as pkv
from scoremod_ref import assert_near, attend
from test_gpu_evict import chosen

pytestmark = pytest.mark.gpu
BS, HQ, HKV, D, EPS = 16, 8, 2, 128, 1e-6
SCALE = 1 / D ** 0.5


def rows(cache, table, L):
    """[L, Hkv, D] in fp64 of one sequence, through its table."""
    t = torch.arange(L, device=cache.device)
    return cache[table.to(cache.device)[t // BS].long(), t % BS].double().cpu().numpy()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_prompt_decode_evict_decode(dtype):
    g = torch.Generator().manual_seed(91)
    budget, recent, cap = 64, 16, 30.0
    bm = pkv.HostBlockManager(64, BS, prefix_cache=False)
    kc = torch.zeros(64, BS, HKV, D, dtype=dtype, device="cuda")
    vc = torch.zeros_like(kc)
    angle = torch.arange(512, dtype=torch.float64)[:, None] * 10000.0 ** (-torch.arange(D // 2, dtype=torch.float64) / (D // 2))
    cos_sin = torch.cat([angle.cos(), angle.sin()], 1).float().cuda()
    qw = (1 + 0.1 * torch.randn(D, generator=g)).to(dtype).cuda()
    kw = (1 + 0.1 * torch.randn(D, generator=g)).to(dtype).cuda()
    prompts = [90, 33, 7]
    sids = [bm.add_sequence(range(n))[0] for n in prompts]
    true_len = list(prompts)

    def write(tokens, slots, positions):
        """The projection of `tokens` rows, normed, rotated and cached: the q rows."""
        qkv = torch.randn(tokens, (HQ + 2 * HKV) * D, generator=g).to(dtype).cuda()
        q, k, v = (x.view(tokens, -1, D) for x in qkv.split([HQ * D, HKV * D, HKV * D], 1))
        out = torch.empty(tokens, HQ, D, dtype=dtype, device="cuda")
        slots = torch.tensor(slots, dtype=torch.int64).cuda()
        pkv.qk_norm_rope_and_cache(out, q, k, v, kc, vc, slots, torch.tensor(positions).cuda(), cos_sin, qw, kw, EPS)
        assert torch.equal(vc.view(-1, HKV, D)[slots], v)
        return out

    # the prompts, each in two chunks
    width = 8
    for part in range(2):
        tables, _ = bm.batch_tables(sids, width)
        chunks = [(n // 2 if part == 0 else n - n // 2) for n in prompts]
        ctx = [0 if part == 0 else n // 2 for n in prompts]
        pos = [c + i for c, n in zip(ctx, chunks) for i in range(n)]
        slots = [int(tables[s, (c + i) // BS]) * BS + (c + i) % BS for s, (c, n) in enumerate(zip(ctx, chunks)) for i in range(n)]
        q = write(sum(chunks), slots, pos)
        start = torch.tensor([0] + list(np.cumsum(chunks)), dtype=torch.int32)
        lens = torch.tensor([c + n for c, n in zip(ctx, chunks)], dtype=torch.int32)
        out = torch.empty_like(q)
        pkv.paged_prefill_scoremod(out, q, kc, vc, tables.cuda(), lens.cuda(), start.cuda(), SCALE, softcap=cap)
        for s in range(3):
            a, b, L = int(start[s]), int(start[s + 1]), int(lens[s])
            ref, bound, _, _ = attend(q[a:b].double().cpu().numpy(), rows(kc, tables[s], L), rows(vc, tables[s], L),
                                      np.arange(ctx[s], L), float(np.float32(SCALE)), dtype, dtype, cap)
            assert_near(out[a:b], ref, bound, f"prompt {s}, part {part}")
    weights = torch.zeros(3, HKV, width * BS, device="cuda")

    for step in range(6):
        slots, pairs = bm.append_batch(sids, [0, 0, 0])
        assert pairs.numel() == 0
        tables, lens = bm.batch_tables(sids, width)
        q = write(3, slots.tolist(), true_len)
        true_len = [n + 1 for n in true_len]
        before = weights.clone()
        out = torch.empty_like(q)
        pkv.paged_attention_decode_weights(out, weights, q, kc, vc, tables.cuda(), lens.cuda(), SCALE, weights=weights)
        capped = torch.empty_like(q)
        pkv.paged_attention_decode_scoremod(capped, q, kc, vc, tables.cuda(), lens.cuda(), SCALE, softcap=cap, window=50)
        for s in range(3):
            L = int(lens[s])
            args = (q[s:s + 1].double().cpu().numpy(), rows(kc, tables[s], L), rows(vc, tables[s], L), np.array([L - 1]),
                    float(np.float32(SCALE)), dtype, dtype)
            ref, bound, p, rel = attend(*args)
            assert_near(out[s:s + 1], ref, bound, f"step {step}, sequence {s}")
            add = p[0].reshape(HKV, -1, L).sum(1)
            old = before[s, :, :L].double().cpu().numpy().copy()
            old[:, L - 1] = 0
            off = (p[0] * rel[0][:, None]).reshape(HKV, -1, L).sum(1)
            assert_near(weights[s, :, :L], old + add, off + 6 * 2.0 ** -24 * (old + add), f"weights, step {step}")
            ref, bound, _, _ = attend(*args, cap, 50)
            assert_near(capped[s:s + 1], ref, bound, f"capped, step {step}, sequence {s}")
        if step in (1, 4):   # shorten what is over the budget
            old_tables, old_lens = bm.batch_tables(sids, width)
            w = weights.cpu().numpy()
            keep = [[chosen(w[s, h], int(old_lens[s]), budget, recent) for h in range(HKV)] for s in range(3)]
            want_k = [rows(kc, old_tables[s], int(old_lens[s])) for s in range(3)]
            new_tables, new_lens = bm.evict_batch(sids, budget)
            got_lens = torch.empty(3, dtype=torch.int32, device="cuda")
            kept = torch.empty(3, HKV, budget, dtype=torch.int32, device="cuda")
            new_weights = torch.zeros_like(weights)
            pkv.evict_tokens(kc, vc, old_tables.cuda(), old_lens.cuda(), weights, new_tables.cuda(), got_lens,
                             new_weights, kept, budget=budget, recent=recent)
            assert got_lens.tolist() == new_lens.tolist()
            now, _ = bm.batch_tables(sids, width)
            for s in range(3):
                n = int(new_lens[s])
                k = rows(kc, now[s], n)
                for h in range(HKV):
                    assert kept[s, h, :n].tolist() == keep[s][h]
                    assert np.array_equal(k[:, h], want_k[s][keep[s][h], h])
                    assert np.array_equal(new_weights[s, h, :n].cpu().numpy(), w[s, h][keep[s][h]])
            weights = new_weights
    assert pkv.get_device_error() == 0
    assert bm.stats()["used_blocks"] == sum(-(-bm.seq_len(s) // BS) for s in sids)


def test_side_streams_run_two_calls_at_once():
    """Two decode calls on two streams with workspaces of their own, interleaved, give each its own result."""
    from scoremod_ref import build, cuda
    from test_gpu_decode_weights import check as check_weights
    ds = []
    for i, lens in enumerate(([300, 5, 1700], [64, 900])):
        d = cuda(build(lens, 2, 128, 16, torch.bfloat16, 70 + i))
        d["q"] = torch.randn(len(lens), 8, 128, generator=torch.Generator().manual_seed(80 + i)).to(torch.bfloat16).cuda()
        d["w"] = torch.rand(len(lens), 2, max(lens), generator=torch.Generator().manual_seed(60 + i)).cuda()
        d["out"], d["wo"] = torch.empty_like(d["q"]), torch.full_like(d["w"], 77.0)
        n = pkv.paged_attention_weights_workspace_bytes(len(lens), 8, 2, 128, d["tables"].shape[1] * 16)
        d["ws"], d["stream"] = torch.empty(n, dtype=torch.uint8, device="cuda"), torch.cuda.Stream()
        ds.append(d)
    torch.cuda.synchronize()
    for _ in range(20):
        for d in ds:
            pkv.paged_attention_decode_weights(d["out"], d["wo"], d["q"], d["kc"], d["vc"], d["tables"], d["lens"], 0.09,
                                               weights=d["w"], workspace=d["ws"], stream=d["stream"])
    torch.cuda.synchronize()
    assert pkv.get_device_error() == 0
    for d in ds:
        check_weights(d, d["out"], d["wo"], 0.09, d["w"])


def test_own_workspace_of_a_call_on_a_side_stream():
    """Without a workspace the call takes its own, which memory asked for on the current stream must not be
    while the side stream still works."""
    from scoremod_ref import build, cuda
    from test_gpu_decode_weights import check as check_weights
    lens = [5000, 3, 4000, 777]
    d = cuda(build(lens, 2, 128, 16, torch.bfloat16, 75))
    d["q"] = torch.randn(len(lens), 8, 128, generator=torch.Generator().manual_seed(85)).to(torch.bfloat16).cuda()
    out, wo = torch.empty_like(d["q"]), torch.empty(len(lens), 2, max(lens), device="cuda").fill_(77.0)
    n = pkv.paged_attention_weights_workspace_bytes(len(lens), 8, 2, 128, d["tables"].shape[1] * 16)
    m = pkv.paged_attention_workspace_bytes(len(lens), 8, 2, 128)
    capped = torch.empty_like(out)
    side = torch.cuda.Stream()
    for stream in (side, side.cuda_stream):
        out.zero_(), capped.zero_()
        torch.cuda.synchronize()
        with torch.cuda.stream(side):  # keep the side stream busy, so that the calls wait on it
            a = torch.randn(4096, 4096, device="cuda")
            for _ in range(20):
                a = a @ a * 1e-3
        pkv.paged_attention_decode_weights(out, wo, d["q"], d["kc"], d["vc"], d["tables"], d["lens"], 0.09, stream=stream)
        pkv.paged_attention_decode_scoremod(capped, d["q"], d["kc"], d["vc"], d["tables"], d["lens"], 0.09,
                                            window=1 << 20, stream=stream)
        held = [torch.empty(x, dtype=torch.uint8, device="cuda").fill_(255) for x in (n, m) for _ in range(8)]
        torch.cuda.synchronize()
        check_weights(d, out, wo, 0.09, None)
        check_weights(d, capped, wo, 0.09, None)
        del held, a
