"""fp64 attention with modified scores, and what a kernel's result may be off.

The bound, with u(x) the relative size of half a step:
  * a score's fp32 dot product of D terms is off by at most D 2^-23 scale
    sum|q_d k_d| (tensor-core additions may truncate); cap, bias, scaling and the
    conversion to the log2 domain add at most 8 roundings of the largest value on
    the way, 8 * 2^-23 (|x| + |capped x| + |bias|) together (the cap scales what came
    before it by its slope, cosh^-2); an FP8 cache's q is
    held as f16 relative to its largest element: 2^-24 max|q| sum|k_d| scale.
    Call the largest sum over a row's visible tokens dx.  exp(x) is then off by a
    factor within exp(+-dx) (1 + 2^-21) and a probability by twice that;
  * P goes to the tensor core in f16 (u = 2^-11; FP8 caches too), as two bf16
    parts (2^-16) or stays fp32; the sums of up to 2^15 terms add L 2^-24;
  * the output is rounded once, u(out) relative.
With A = sum_t p_t |v_t|, |error| <= A (2 (e^dx - 1) + 2^-19 + 2 u_P + L 2^-23) + u(out) |out|."""
import numpy as np
import torch

U_P = {torch.float16: 2.0 ** -11, torch.uint8: 2.0 ** -11, torch.bfloat16: 2.0 ** -16, torch.float32: 0.0}


def attend(q, k, v, pos, scale, cache_dtype, out_dtype, softcap=0.0, window=0, slopes=None, prefix=0):
    """q [C, Hq, D] at positions pos [C], k and v [L, Hkv, D] (fp64): (out, bound, probabilities
    [C, Hq, L], relative bound of the probabilities [C, Hq])."""
    C, Hq, D = q.shape
    L, Hkv = k.shape[:2]
    g = Hq // Hkv
    t = np.arange(L)
    vis = t[None] <= pos[:, None]
    if window:
        vis &= pos[:, None] - t[None] < window
    vis |= t[None] < min(prefix, L)
    kk = np.where(np.isfinite(k), k, 0.0).repeat(g, 1)
    vv = np.where(np.isfinite(v), v, 0.0).repeat(g, 1)
    x = np.einsum("chd,thd->cht", q, kk) * scale
    size = np.einsum("chd,thd->cht", np.abs(q), np.abs(kk)) * abs(scale)
    dx = D * 2.0 ** -23 * size + 8 * 2.0 ** -23 * np.abs(x)
    if cache_dtype == torch.uint8:
        dx += 2.0 ** -24 * abs(scale) * np.einsum("ch,th->cht", np.abs(q).max(-1), np.abs(kk).sum(-1))
    if softcap:
        with np.errstate(over="ignore"):  # the cap's slope nowhere on x +- dx exceeds its value nearest to 0
            dx = dx / np.cosh(np.maximum(np.abs(x) - dx, 0) / softcap) ** 2
        x = softcap * np.tanh(x / softcap)
        dx += 8 * 2.0 ** -23 * np.abs(x)
    if slopes is not None:
        bias = np.asarray(slopes)[None, :, None] * np.abs(pos[:, None] - t[None])[:, None]
        x = x - bias
        dx += 8 * 2.0 ** -23 * np.abs(bias)
    x = np.where(vis[:, None], x, -np.inf)
    dx = np.where(vis[:, None], dx, 0.0).max(-1)
    m = x.max(-1, keepdims=True)
    p = np.exp(x - m)
    p /= p.sum(-1, keepdims=True)
    out = np.einsum("cht,thd->chd", p, vv)
    A = np.einsum("cht,thd->chd", p, np.abs(vv))
    rel = 2 * np.expm1(np.minimum(dx, 50.0)) + 2.0 ** -19 + L * 2.0 ** -23
    u = torch.finfo(out_dtype).eps / 2
    bound = A * (rel + 2 * U_P[cache_dtype])[..., None] + u * np.abs(out) + float(torch.finfo(out_dtype).tiny)
    return out, bound, p, rel


def build(lens, Hkv, D, bs, cache_dtype, seed, live=None, spare=3):
    """A pool whose every slot holds NaN but the live tokens of each sequence (live[s]: bool [L],
    default all): dict of CPU tensors; blocks without a live token have table entry -1."""
    g = torch.Generator().manual_seed(seed)
    S = len(lens)
    width = max([-(-L // bs) for L in lens] + [1])
    NB = sum(-(-L // bs) for L in lens) + spare
    order = torch.randperm(NB, generator=g).tolist()
    fp8 = cache_dtype == torch.uint8
    if fp8:
        kc = torch.full((NB, bs, Hkv, D), 0x7F, dtype=torch.uint8)
    else:
        kc = torch.full((NB, bs, Hkv, D), float("nan"), dtype=cache_dtype)
    vc = kc.clone()
    tables = torch.full((S, width), -1, dtype=torch.int32)
    ks, vs = (0.02, 0.03) if fp8 else (1.0, 1.0)
    K, V = [], []
    for s, L in enumerate(lens):
        ok = torch.ones(L, dtype=torch.bool) if live is None else torch.as_tensor(live[s])
        rows = []
        for cache, sc in ((kc, ks), (vc, vs)):
            x = torch.randn(L, Hkv, D, generator=g)
            x = (x / sc).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8) if fp8 else x.to(cache_dtype)
            for b in range(-(-L // bs)):
                lo, hi = b * bs, min(L, b * bs + bs)
                if not ok[lo:hi].any():
                    continue
                if tables[s, b] < 0:
                    tables[s, b] = order.pop()
                part = cache[tables[s, b], :hi - lo]
                part[ok[lo:hi]] = x[lo:hi][ok[lo:hi]]
            val = x.view(torch.float8_e4m3fn).double() * float(np.float32(sc)) if fp8 else x.double()
            val[~ok] = float("nan")
            rows.append(val.numpy())
        K.append(rows[0])
        V.append(rows[1])
    d = dict(kc=kc, vc=vc, tables=tables, lens=torch.tensor(lens, dtype=torch.int32), K=K, V=V, ks=None, vs=None)
    if fp8:
        d["ks"], d["vs"] = torch.tensor([ks]), torch.tensor([vs])
    return d


def cuda(d):
    return {k: x.cuda() if isinstance(x, torch.Tensor) else x for k, x in d.items()}


def visible(L, p, window, prefix):
    t = np.arange(L)
    v = t <= p
    if window:
        v &= p - t < window
    return v | (t < min(max(prefix, 0), L))


def assert_near(got, want, bound, what=""):
    got = got.double().cpu().numpy()
    assert np.isfinite(got).all(), f"{what}: not finite"
    over = np.abs(got - want) - bound
    assert (over <= 0).all(), f"{what}: off by {np.abs(got - want).max():.3e}, {over.max():.3e} over the bound"
