"""Cases and plain forms of the serving operators around the paged KV cache.

Five operators, each with the calls a serving loop makes of it:

  rope     per-head norm of q and k, rotary embedding and the cache write in one pass
  decode   single-token attention with modified scores (tanh cap, distance bias, window, prefix)
  prefill  the same for chunks of new tokens
  weights  single-token attention that also accumulates each cached token's attention weight
  evict    keeps the heaviest and the most recent tokens of a sequence and compacts them

``run`` computes the plain form from elementary torch operations in fp32, or, where ``own`` is
set, calls the library.  ``exact`` computes the same results in fp64, sequence by sequence.
"""
import math
import random

import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16, "fp8": torch.uint8}
ROPE_THETA = 1.0e6
MAX_POSITION = 32768
EPS = 1e-6


# -- cases ---------------------------------------------------------------------
def listed():
    return [
        # one decode step of a 4-request batch, head shapes of an 8B GQA model: latency
        dict(name="rope step 4", op="rope", tokens=4, pad=0, heads=32, kv_heads=8, head_dim=128, dtype="bf16",
             cache="bf16", rotary=128, interleaved=False, norm=True, block=16),
        # a token budget of 8192 prompt tokens with q and k norms (1.7B-shaped layer)
        dict(name="rope chunk 8192", op="rope", tokens=8192, pad=0, heads=16, kv_heads=8, head_dim=128, dtype="bf16",
             cache="bf16", rotary=128, interleaved=False, norm=True, block=16),
        # a padded step into an FP8 cache: half of the head rotated, pairs side by side
        dict(name="rope fp8 1023", op="rope", tokens=1023, pad=31, heads=64, kv_heads=8, head_dim=128, dtype="bf16",
             cache="fp8", rotary=64, interleaved=True, norm=False, block=32),
        # three requests, capped scores: the smallest decode call
        dict(name="decode cap 3", op="decode", seqs=3, lo=5, hi=301, heads=8, kv_heads=4, head_dim=64, dtype="f16",
             cache="f16", block=16, softcap=30.0, window=0, alibi=False, prefix=0),
        # a full batch of log-uniform lengths, capped scores
        dict(name="decode cap 128", op="decode", seqs=128, lo=64, hi=8192, heads=32, kv_heads=8, head_dim=128,
             dtype="bf16", cache="bf16", block=16, softcap=50.0, window=0, alibi=False, prefix=0),
        # long contexts in FP8 with a window and kept first tokens
        dict(name="decode window fp8", op="decode", seqs=16, lo=16384, hi=32768, heads=64, kv_heads=8, head_dim=128,
             dtype="bf16", cache="fp8", block=32, softcap=0.0, window=4096, alibi=False, prefix=64),
        # ragged small chunks with a distance bias, one head per kv head
        dict(name="prefill bias ragged", op="prefill", ctx="0,100,33", chunks="29,64,1", heads=8, kv_heads=8,
             head_dim=64, dtype="f16", block=32, softcap=0.0, window=0, alibi=True, prefix=0),
        # a step of 8192 prompt tokens with capped scores: two whole inputs, part of a third, a decode row
        dict(name="prefill cap 8192", op="prefill", ctx="4499,0,0,0", chunks="1,3500,3500,1191", heads=16, kv_heads=8,
             head_dim=128, dtype="bf16", block=16, softcap=50.0, window=0, alibi=False, prefix=0),
        # a later chunk of a long prompt: window, and a prefix that every row attends
        dict(name="prefill window 2048", op="prefill", ctx="6100", chunks="2048", heads=32, kv_heads=8, head_dim=128,
             dtype="bf16", block=16, softcap=0.0, window=1024, alibi=False, prefix=200),
        # accumulated weights over a batch of log-uniform lengths
        dict(name="weights 64", op="weights", seqs=64, lo=64, hi=8192, heads=32, kv_heads=8, head_dim=128,
             dtype="bf16", cache="bf16", block=16),
        # a small batch with one head per kv head
        dict(name="weights mha 5", op="weights", seqs=5, lo=1, hi=777, heads=4, kv_heads=4, head_dim=128, dtype="f16",
             cache="f16", block=16),
        # half of each long sequence's tokens leave the cache
        dict(name="evict 32", op="evict", seqs=32, lo=1000, hi=8192, budget=2048, recent=512, kv_heads=8, head_dim=128,
             cache="bf16", block=16),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "decode", "prefill", "weights", "evict"])
    head_dim = rng.choice([64, 128])
    block = rng.choice([16, 32])
    kv_heads = rng.choice([1, 2, 4, 8])
    group = rng.choice([1, 2, 4, 8])
    dtype = rng.choice(["f16", "bf16"])
    if op == "rope":
        tokens = _log(rng, 1, 8192)
        cache = rng.choice([dtype, dtype, "fp8"])
        return dict(op=op, tokens=tokens, pad=rng.randrange(0, 1 + tokens // 4), heads=kv_heads * min(group, 2),
                    kv_heads=kv_heads, head_dim=head_dim, dtype=dtype, cache=cache,
                    rotary=rng.choice([head_dim, head_dim // 2, 48]), interleaved=rng.random() < 0.5,
                    norm=rng.random() < 0.7, block=block)
    if op == "evict":
        seqs = _log(rng, 1, 32)
        hi = _log(rng, 300, 8192)
        budget = _log(rng, 100, 2048)
        return dict(op=op, seqs=seqs, lo=_log(rng, 1, hi), hi=hi, budget=budget, recent=rng.randrange(0, budget + 1),
                    kv_heads=kv_heads, head_dim=head_dim, cache=rng.choice(["bf16", "f16", "fp8"]), block=block)
    mods = dict(softcap=rng.choice([0.0, 0.0, rng.uniform(5.0, 80.0)]), window=rng.choice([0, _log(rng, 1, 4096)]),
                alibi=rng.random() < 0.4, prefix=rng.choice([0, 0, _log(rng, 1, 600)]))
    if op == "prefill":
        seqs = rng.randint(1, 4)
        ctx = [rng.choice([0, _log(rng, 1, 4000)]) for _ in range(seqs)]
        chunks = [_log(rng, 1, 2000) for _ in range(seqs)]
        return dict(op=op, ctx=",".join(map(str, ctx)), chunks=",".join(map(str, chunks)),
                    heads=kv_heads * min(group, 2), kv_heads=kv_heads, head_dim=head_dim, dtype=dtype, block=block,
                    **mods)
    cache = rng.choice([dtype, dtype, "fp8"])
    seqs = _log(rng, 1, 64)
    hi = _log(rng, 16, 8192)
    case = dict(op=op, seqs=seqs, lo=_log(rng, 1, hi), hi=hi, heads=kv_heads * group, kv_heads=kv_heads,
                head_dim=128 if cache == "fp8" else head_dim, dtype=dtype, cache=cache, block=block)
    return {**case, **mods} if op == "decode" else case


# -- sizes that follow from the case alone ---------------------------------------
def _lengths(case):
    """Lengths spread log-uniformly over [lo, hi], the longest included, in a fixed shuffled order."""
    n, lo, hi = case["seqs"], case["lo"], case["hi"]
    lens = [max(1, int(round(lo * (hi / lo) ** ((i + 0.5) / n)))) for i in range(n)]
    lens[-1] = hi
    random.Random(7).shuffle(lens)
    return lens


def _chunks(case):
    return [int(x) for x in case["ctx"].split(",")], [int(x) for x in case["chunks"].split(",")]


def _visible(L, p, window, prefix):
    """Tokens that the row at position p of a sequence of L tokens attends."""
    first = max(0, p + 1 - window) if window else 0
    pre = min(prefix, L)
    return p + 1 - first + min(pre, first) + max(0, pre - p - 1)


def work(case):
    op = case["op"]
    D, Hkv = case["head_dim"], case["kv_heads"]
    if op == "evict":
        lens = _lengths(case)
        eb = 1 if case["cache"] == "fp8" else 2
        kept = sum(min(L, case["budget"]) for L in lens)
        moved = sum(case["budget"] for L in lens if L > case["budget"])
        return {"bytes": 4 * Hkv * (sum(lens) + 2 * kept) + 2 * 2 * moved * Hkv * D * eb, "flops": 0}
    eb = 4 if case["dtype"] == "f32" else 2
    H = case["heads"]
    if op == "rope":
        live = case["tokens"] - case["pad"]
        cb = 1 if case["cache"] == "fp8" else eb
        row = (H + 2 * Hkv) * D * eb + H * D * eb + 2 * Hkv * D * cb + 4 * case["rotary"] + 16
        return {"bytes": live * row, "flops": 10 * live * (H + Hkv) * D}
    if op == "prefill":
        ctx, chunks = _chunks(case)
        pairs, kv = 0, 0
        for c, n in zip(ctx, chunks):
            pairs += sum(_visible(c + n, c + i, case["window"], case["prefix"]) for i in range(n))
            first = max(0, c + 1 - case["window"]) if case["window"] else 0
            kv += c + n - first + min(first, case["prefix"])
        return {"bytes": 2 * sum(chunks) * H * D * eb + 2 * kv * Hkv * D * eb, "flops": 4 * pairs * H * D}
    lens = _lengths(case)
    cb = 1 if case["cache"] == "fp8" else eb
    tokens = sum(lens) if op == "weights" else sum(_visible(L, L - 1, case["window"], case["prefix"]) for L in lens)
    size = 2 * tokens * Hkv * D * cb + 2 * len(lens) * H * D * eb
    if op == "weights":
        size += 2 * 4 * tokens * Hkv
    return {"bytes": size, "flops": 4 * tokens * H * D}


# -- inputs --------------------------------------------------------------------------
def _normal(gen, shape, dtype):
    out = torch.empty(shape, dtype=dtype, device="cuda")
    flat = out.view(-1)
    for i in range(0, flat.numel(), 1 << 26):
        part = flat[i:i + (1 << 26)]
        part.copy_(torch.randn(part.numel(), generator=gen, device="cuda"))
    return out


def _pool(gen, blocks, case, scale):
    """A block pool of the case's cache type; FP8 pools hold the codes of N(0, 1) values over `scale`."""
    shape = (blocks, case["block"], case["kv_heads"], case["head_dim"])
    if case["cache"] != "fp8":
        return _normal(gen, shape, DTYPES[case["cache"]])
    x = _normal(gen, shape, torch.bfloat16)
    out = torch.empty(shape, dtype=torch.uint8, device="cuda")
    for i in range(0, blocks, 4096):
        out[i:i + 4096] = (x[i:i + 4096].float() / scale).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    return out


def _tables(gen, lens, block, blocks=None, order=None):
    """Block tables of shuffled physical blocks (unused entries -1), and the shuffled ids left over."""
    need = [-(-L // block) for L in lens]
    total = sum(need)
    if order is None:
        order = torch.randperm(blocks, generator=gen, device="cuda").to(torch.int32)
    width = max(need + [1])
    counts = torch.tensor(need, device="cuda")
    col = torch.arange(width, device="cuda")
    used = col[None, :] < counts[:, None]
    table = torch.full((len(lens), width), -1, dtype=torch.int32, device="cuda")
    table[used] = order[:total]
    return table, order[total:]


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    s = dict(case=case)
    block, D, Hkv = case["block"], case["head_dim"], case["kv_heads"]
    if case.get("cache") == "fp8":
        s["k_scale"] = torch.tensor([6.0 / 448], device="cuda")
        s["v_scale"] = torch.tensor([6.5 / 448], device="cuda")
    if case["op"] == "rope":
        T, H, dtype = case["tokens"], case["heads"], DTYPES[case["dtype"]]
        blocks = max(4, -(-T // block) * 11 // 10) if T > 512 else T + 8
        s["key_cache"] = _pool(gen, blocks, case, 6.0 / 448)
        s["value_cache"] = _pool(gen, blocks, case, 6.5 / 448)
        # q, k and v are column ranges of one projection's output, as the product leaves them
        s["qkv"] = _normal(gen, (T, (H + 2 * Hkv) * D), dtype)
        order = torch.randperm(blocks, generator=gen, device="cuda")
        i = torch.arange(T, device="cuda")
        if T > 512:  # a prompt's tokens fill whole blocks
            slots = order[i // block] * block + i % block
        else:        # one new token per sequence
            slots = order[:T] * block + torch.randint(block, (T,), generator=gen, device="cuda")
        if case["pad"]:
            slots[T - case["pad"]:] = -1
        s["slots"] = slots
        s["positions"] = torch.randint(MAX_POSITION, (T,), generator=gen, device="cuda")
        half = case["rotary"] // 2
        freq = ROPE_THETA ** (-torch.arange(half, device="cuda", dtype=torch.float64) / half)
        angle = torch.arange(MAX_POSITION, device="cuda", dtype=torch.float64)[:, None] * freq
        s["cos_sin"] = torch.cat([angle.cos(), angle.sin()], 1).float()
        s["q_weight"] = s["k_weight"] = None
        if case["norm"]:
            s["q_weight"] = (1 + 0.2 * torch.randn(D, generator=gen, device="cuda")).to(dtype)
            s["k_weight"] = (1 + 0.2 * torch.randn(D, generator=gen, device="cuda")).to(dtype)
        s["query_out"] = torch.zeros((T, H, D), dtype=dtype, device="cuda")
        return s
    if case["op"] == "prefill":
        ctx, chunks = _chunks(case)
        lens = [a + b for a, b in zip(ctx, chunks)]
        s["query"] = _normal(gen, (sum(chunks), case["heads"], D), DTYPES[case["dtype"]])
        start = [0]
        for n in chunks:
            start.append(start[-1] + n)
        s["query_start"] = torch.tensor(start, dtype=torch.int32, device="cuda")
        case = {**case, "cache": case["dtype"]}
    else:
        lens = _lengths(case)
        if case["op"] != "evict":
            s["query"] = _normal(gen, (len(lens), case["heads"], D), DTYPES[case["dtype"]])
    need = sum(-(-L // block) for L in lens)
    if case["op"] == "evict":
        kept = [min(L, case["budget"]) if L > case["budget"] else 0 for L in lens]
        need += sum(-(-n // block) for n in kept)
    blocks = need + need // 10 + 1
    s["block_tables"], rest = _tables(gen, lens, block, blocks)
    s["seq_lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    s["key_cache"] = _pool(gen, blocks, case, 6.0 / 448)
    s["value_cache"] = _pool(gen, blocks, case, 6.5 / 448)
    width = s["block_tables"].shape[1] * block
    if case["op"] in ("weights", "evict"):
        # accumulated weights: heavy-tailed, many tokens that were hardly ever attended
        w = torch.randn((len(lens), Hkv, width), generator=gen, device="cuda").mul_(2.0).exp_()
        w = torch.where(w < 0.2, 0.0, w)
        live = torch.arange(width, device="cuda")[None, None, :] < s["seq_lens"][:, None, None]
        s["weights"] = torch.where(live, w, 0.0)
    if case["op"] == "weights":
        s["weights_out"] = torch.zeros_like(s["weights"])
    if case["op"] == "evict":
        s["new_tables"], _ = _tables(gen, kept, block, order=rest)
        n = min(case["budget"], width)
        s["new_weights"] = torch.zeros((len(lens), Hkv, n), device="cuda")
        s["new_lens"] = torch.zeros(len(lens), dtype=torch.int32, device="cuda")
        s["kept"] = torch.zeros((len(lens), Hkv, case["budget"]), dtype=torch.int32, device="cuda")
    else:
        scores = len(lens) * case["heads"] * width * 4 if case["op"] == "weights" else 0
        s["workspace"] = torch.empty(scores + (64 << 20), dtype=torch.uint8, device="cuda")
    if case.get("alibi"):
        s["slopes"] = torch.tensor([2.0 ** (-8.0 * (h + 1) / case["heads"]) for h in range(case["heads"])], device="cuda")
    if case.get("prefix"):
        s["prefix_lens"] = torch.full((len(lens),), case["prefix"], dtype=torch.int32, device="cuda")
    return s


# -- plain forms --------------------------------------------------------------------
def _scale(case):
    return 1.0 / math.sqrt(case["head_dim"])


def _values(cache, scale=None):
    """Cache entries in fp32."""
    return cache.float() if scale is None else cache.view(torch.float8_e4m3fn).float() * scale


def _seen(cache):
    """What is held in 8 bits, as the values it stands for."""
    return cache.view(torch.float8_e4m3fn) if cache.dtype == torch.uint8 else cache


def _gathered(cache, tables, scale=None):
    """[S, T, Hkv, D] in fp32: the blocks of each table row, one after another."""
    x = _values(cache[tables.clamp(min=0).long()], scale)
    return x.flatten(1, 2)


def _modified(x, s, distance, softcap):
    """Scores x [S, kv, g, ...] capped, then biased by the distance between row and token."""
    if softcap:
        x = softcap * torch.tanh(x / softcap)
    if "slopes" in s:
        slope = s["slopes"].view(x.shape[1], x.shape[2], *([1] * (x.dim() - 3)))
        x = x - slope * distance
    return x


def _plain_rope(s):
    case = s["case"]
    T, H, Hkv, D = case["tokens"], case["heads"], case["kv_heads"], case["head_dim"]
    q, k, v = (x.view(T, -1, D).float() for x in s["qkv"].split([H * D, Hkv * D, Hkv * D], 1))
    r, half = case["rotary"], case["rotary"] // 2
    table = s["cos_sin"][s["positions"]]
    cos, sin = table[:, None, :half], table[:, None, half:]

    def turned(x, w):
        if w is not None:
            x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * w.float()
        if case["interleaved"]:
            a, b = x[..., 0:r:2], x[..., 1:r:2]
            y = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
        else:
            a, b = x[..., :half], x[..., half:r]
            y = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
        return torch.cat([y, x[..., r:]], -1)

    q, k = turned(q, s["q_weight"]), turned(k, s["k_weight"])
    live = s["slots"] >= 0
    s["query_out"].copy_(torch.where(live[:, None, None], q.to(s["query_out"].dtype), s["query_out"]))
    rows = s["slots"][live]
    if case["cache"] == "fp8":
        k, v = k / s["k_scale"], v / s["v_scale"]
        k, v = (x.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8) for x in (k, v))
    s["key_cache"].view(-1, Hkv, D)[rows] = k[live].to(s["key_cache"].dtype)
    s["value_cache"].view(-1, Hkv, D)[rows] = v[live].to(s["value_cache"].dtype)
    return [s["query_out"], _seen(s["key_cache"]), _seen(s["value_cache"])]


def _decode_probabilities(s, softcap=0.0, window=0):
    case = s["case"]
    S, Hkv, D = len(s["seq_lens"]), case["kv_heads"], case["head_dim"]
    q = s["query"].float().view(S, Hkv, -1, D)
    k = _gathered(s["key_cache"], s["block_tables"], s.get("k_scale"))
    x = torch.einsum("skgd,stkd->skgt", q, k) * _scale(case)
    t = torch.arange(k.shape[1], device="cuda")[None, :]
    p = s["seq_lens"].long()[:, None] - 1
    visible = (t <= p) & (p - t < window) if window else t <= p
    if "prefix_lens" in s:
        visible = visible | (t < torch.minimum(s["prefix_lens"].long()[:, None], p + 1))
    x = _modified(x, s, (p - t).abs()[:, None, None, :], softcap)
    x = torch.where(visible[:, None, None, :], x, -math.inf)
    e = torch.exp(x - x.amax(-1, keepdim=True))
    return e / e.sum(-1, keepdim=True)


def _plain_decode(s):
    case = s["case"]
    p = _decode_probabilities(s, case["softcap"], case["window"])
    v = _gathered(s["value_cache"], s["block_tables"], s.get("v_scale"))
    return [torch.einsum("skgt,stkd->skgd", p, v).reshape(s["query"].shape).to(s["query"].dtype)]


def _plain_weights(s):
    p = _decode_probabilities(s)
    v = _gathered(s["value_cache"], s["block_tables"], s.get("v_scale"))
    out = torch.einsum("skgt,stkd->skgd", p, v).reshape(s["query"].shape).to(s["query"].dtype)
    p = p.sum(2)
    t = torch.arange(p.shape[2], device="cuda")[None, None, :]
    last = s["seq_lens"].long()[:, None, None] - 1
    new = torch.where(t < last, s["weights"] + p, p)
    s["weights_out"].copy_(torch.where(t <= last, new, s["weights_out"]))
    return [out, s["weights_out"]]


def _plain_prefill(s):
    case = s["case"]
    T, H, D = s["query"].shape
    Hkv, S = case["kv_heads"], len(s["seq_lens"])
    start = s["query_start"].long()
    seq = torch.searchsorted(start, torch.arange(T, device="cuda"), right=True) - 1
    row = torch.arange(T, device="cuda") - start[seq]
    most = int((start[1:] - start[:-1]).max())
    q = torch.zeros((S, most, H, D), device="cuda")
    q[seq, row] = s["query"].float()
    q = q.view(S, most, Hkv, H // Hkv, D)
    k = _gathered(s["key_cache"], s["block_tables"])
    x = torch.einsum("sckgd,stkd->skgct", q, k) * _scale(case)
    lens = s["seq_lens"].long()
    p = (lens - (start[1:] - start[:-1]))[:, None, None] + torch.arange(most, device="cuda")[None, :, None]
    t = torch.arange(k.shape[1], device="cuda")[None, None, :]
    visible = (t <= p) & (p - t < case["window"]) if case["window"] else t <= p
    if "prefix_lens" in s:
        visible = visible | (t < torch.minimum(s["prefix_lens"].long(), lens)[:, None, None])
    visible = visible & (t < lens[:, None, None])
    x = _modified(x, s, (p - t).abs()[:, None, None], case["softcap"])
    x = x.masked_fill_(~visible[:, None, None], -math.inf)
    x = torch.exp(x.sub_(x.amax(-1, keepdim=True).clamp(min=-1e30)))
    total = x.sum(-1)
    v = _gathered(s["value_cache"], s["block_tables"])
    out = torch.einsum("skgct,stkd->sckgd", x, v) / total.permute(0, 3, 1, 2)[..., None]
    return [out.reshape(S, most, H, D)[seq, row].to(s["query"].dtype)]


def _plain_evict(s):
    case = s["case"]
    budget, recent, block = case["budget"], case["recent"], case["block"]
    w, lens = s["weights"], s["seq_lens"].long()[:, None, None]
    t = torch.arange(w.shape[2], device="cuda")[None, None, :]
    rank = torch.where(t >= lens - recent, math.inf, w)
    rank = torch.where(t < lens, rank, -math.inf)
    order = torch.argsort(rank, dim=-1, descending=True, stable=True)
    n = s["new_weights"].shape[2]
    j = torch.arange(n, device="cuda")[None, None, :]
    keep = torch.where(j < lens, order[..., :n], w.shape[2]).sort(-1).values
    held = j < lens
    source = torch.where(held, keep, 0)
    s["new_weights"].copy_(torch.where(held, w.gather(2, source), s["new_weights"]))
    s["kept"].fill_(-1)
    s["kept"][..., :n] = torch.where(held, keep, -1).int()
    s["new_lens"].copy_(lens.view(-1).clamp(max=budget))
    moves = (held & (lens > budget)).expand_as(source)
    seq = torch.arange(w.shape[0], device="cuda")[:, None, None].expand_as(moves)[moves]
    head = torch.arange(w.shape[1], device="cuda")[None, :, None].expand_as(moves)[moves]
    src, dst = source[moves], j.expand_as(moves)[moves]
    from_block = s["block_tables"][seq, src // block].long()
    to_block = s["new_tables"][seq, dst // block].long()
    for cache in (s["key_cache"], s["value_cache"]):
        cache[to_block, dst % block, head] = cache[from_block, src % block, head]
    return [s["new_lens"], s["kept"], s["new_weights"], _seen(s["key_cache"]), _seen(s["value_cache"])]


# -- the library's calls ---------------------------------------------------------------
def _own(s):
    import paged_kv_cache_373_b200 as pkv
    case = s["case"]
    op = case["op"]
    if op == "rope":
        T, H, Hkv, D = case["tokens"], case["heads"], case["kv_heads"], case["head_dim"]
        q, k, v = (x.view(T, -1, D) for x in s["qkv"].split([H * D, Hkv * D, Hkv * D], 1))
        pkv.qk_norm_rope_and_cache(s["query_out"], q, k, v, s["key_cache"], s["value_cache"], s["slots"],
                                   positions=s["positions"], cos_sin=s["cos_sin"], q_weight=s["q_weight"],
                                   k_weight=s["k_weight"], eps=EPS, interleaved=case["interleaved"],
                                   k_scale=s.get("k_scale"), v_scale=s.get("v_scale"))
        return [s["query_out"], _seen(s["key_cache"]), _seen(s["value_cache"])]
    if op == "evict":
        pkv.evict_tokens(s["key_cache"], s["value_cache"], s["block_tables"], s["seq_lens"], s["weights"],
                         s["new_tables"], s["new_lens"], s["new_weights"], s["kept"], budget=case["budget"],
                         recent=case["recent"])
        return [s["new_lens"], s["kept"], s["new_weights"], _seen(s["key_cache"]), _seen(s["value_cache"])]
    out = torch.empty_like(s["query"])
    if op == "weights":
        pkv.paged_attention_decode_weights(out, s["weights_out"], s["query"], s["key_cache"], s["value_cache"],
                                           s["block_tables"], s["seq_lens"], _scale(case), weights=s["weights"],
                                           k_scale=s.get("k_scale"), v_scale=s.get("v_scale"),
                                           workspace=s["workspace"])
        return [out, s["weights_out"]]
    mods = dict(softcap=case["softcap"], window=case["window"], alibi_slopes=s.get("slopes"),
                prefix_lens=s.get("prefix_lens"))
    if op == "decode":
        pkv.paged_attention_decode_scoremod(out, s["query"], s["key_cache"], s["value_cache"], s["block_tables"],
                                            s["seq_lens"], _scale(case), k_scale=s.get("k_scale"),
                                            v_scale=s.get("v_scale"), workspace=s["workspace"], **mods)
    else:
        pkv.paged_prefill_scoremod(out, s["query"], s["key_cache"], s["value_cache"], s["block_tables"],
                                   s["seq_lens"], s["query_start"], _scale(case), **mods)
    return [out]


def run(state):
    if own:
        return _own(state)
    op = state["case"]["op"]
    if op == "rope":
        return _plain_rope(state)
    if op == "decode":
        return _plain_decode(state)
    if op == "prefill":
        return _plain_prefill(state)
    if op == "weights":
        return _plain_weights(state)
    return _plain_evict(state)


# -- 64 bits, sequence by sequence -------------------------------------------------------
def _sequence(cache, s, i, L, scale):
    """[L, Hkv, D] in fp64."""
    b = s["case"]["block"]
    t = torch.arange(L, device="cuda")
    rows = cache[s["block_tables"][i, t // b].long(), t % b]
    return rows.double() if scale is None else rows.view(torch.float8_e4m3fn).to(torch.float64) * scale.double()


def _attend(q, k, v, pos, case, slopes, prefix):
    """q [C, H, D] at positions pos against one sequence's k, v [L, Hkv, D]: (out, probabilities [H, C, L])."""
    C, H, D = q.shape
    L, Hkv = k.shape[0], k.shape[1]
    g = H // Hkv
    outs, probs = [], []
    t = torch.arange(L, device="cuda")
    allowed = t[None, :] <= pos[:, None]
    if case.get("window"):
        allowed &= t[None, :] > pos[:, None] - case["window"]
    if prefix:
        allowed |= t[None, :] < prefix
    far = (pos[:, None] - t[None, :]).abs().double()
    for h in range(H):
        z = (q[:, h].double() @ k[:, h // g].T) / math.sqrt(D)
        if case.get("softcap"):
            z = torch.tanh(z / case["softcap"]) * case["softcap"]
        if slopes is not None:
            z = z - float(slopes[h]) * far
        z = torch.softmax(z.masked_fill(~allowed, -math.inf), -1)
        outs.append(z @ v[:, h // g])
        probs.append(z if case["op"] == "weights" else None)
    return torch.stack(outs, 1), probs


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    D, Hkv = case["head_dim"], case["kv_heads"]
    if op == "evict":
        w, lens = s["weights"].cpu().numpy(), s["seq_lens"].tolist()
        budget, recent = case["budget"], case["recent"]
        kept, new_w = s["kept"].cpu(), s["new_weights"].cpu()
        kc, vc = s["key_cache"].clone(), s["value_cache"].clone()
        kept.fill_(-1)
        for i, L in enumerate(lens):
            for h in range(Hkv):
                if L > budget:
                    old = sorted(range(L - recent), key=lambda a: (-w[i, h, a], a))[:budget - recent]
                    ids = sorted(old) + list(range(L - recent, L))
                else:
                    ids = list(range(L))
                ids = torch.tensor(ids)
                kept[i, h, :len(ids)] = ids.int()
                new_w[i, h, :len(ids)] = torch.from_numpy(w[i, h])[ids]
                if L > budget:
                    a, d = ids.cuda(), torch.arange(len(ids), device="cuda")
                    b = case["block"]
                    for c in (kc, vc):
                        c[s["new_tables"][i, d // b].long(), d % b, h] = c[s["block_tables"][i, a // b].long(), a % b, h]
        return [torch.tensor([min(L, budget) for L in lens], dtype=torch.int32), kept, new_w.double(),
                _seen(kc).to(torch.float64), _seen(vc).to(torch.float64)]
    if op == "rope":
        H, T = case["heads"], case["tokens"]
        x = s["qkv"].double().view(T, H + 2 * Hkv, D)
        half = case["rotary"] // 2
        at = s["cos_sin"][s["positions"]].double()
        turn = torch.complex(at[:, :half], at[:, half:])[:, None]
        parts = []
        for y, w in ((x[:, :H], s["q_weight"]), (x[:, H:H + Hkv], s["k_weight"])):
            if w is not None:
                y = y / torch.sqrt(y.pow(2).sum(-1, keepdim=True) / D + EPS) * w.double()
            y = y.clone()
            first = slice(0, 2 * half, 2) if case["interleaved"] else slice(0, half)
            second = slice(1, 2 * half, 2) if case["interleaved"] else slice(half, 2 * half)
            z = torch.complex(y[..., first], y[..., second]) * turn
            y[..., first], y[..., second] = z.real, z.imag
            parts.append(y)
        live = torch.nonzero(s["slots"] >= 0).view(-1)
        q = torch.zeros((T, H, D), dtype=torch.float64, device="cuda")
        q[live] = parts[0][live]
        if case["cache"] == "fp8":
            return [q, None, None]  # codes of values next to a rounding border
        caches = []
        for cache, rows in ((s["key_cache"], parts[1]), (s["value_cache"], x[:, H + Hkv:])):
            c = cache.double().view(-1, Hkv, D)
            c[s["slots"][live]] = rows[live]
            caches.append(c.view(cache.shape))
        return [q, *caches]
    slopes = s["slopes"].tolist() if "slopes" in s else None
    lens = s["seq_lens"].tolist()
    starts = s["query_start"].tolist() if op == "prefill" else list(range(len(lens) + 1))
    out = torch.empty(s["query"].shape, dtype=torch.float64, device="cuda")
    total = s["weights_out"].double() if op == "weights" else None
    for i, L in enumerate(lens):
        k = _sequence(s["key_cache"], s, i, L, s.get("k_scale"))
        v = _sequence(s["value_cache"], s, i, L, s.get("v_scale"))
        for a in range(starts[i], starts[i + 1], 1024):
            b = min(a + 1024, starts[i + 1])
            pos = torch.arange(a, b, device="cuda") - starts[i + 1] + L
            out[a:b], probs = _attend(s["query"][a:b], k, v, pos, case, slopes, min(case.get("prefix", 0), L))
            if op == "weights":
                p = torch.stack(probs).view(Hkv, -1, L).sum(1)
                p[:, :L - 1] += s["weights"][i, :, :L - 1].double()
                total[i, :, :L] = p
    return [out] if total is None else [out, total]
