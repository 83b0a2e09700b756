"""Serving and training on packed, ragged batches: the operators that are
measured, their plain forms in torch, and their definitions in 64 bits.

A server keeps the keys and values of its requests in pages of a cache held in
8 bits (e4m3) with one scale for each page and head.  One step of it
  pages    gives the requests' new tokens their pages and slots,
  append   rounds the new keys and values into those slots,
  decode   attends from the newest tokens of every request to its whole cache,
and a prompt is first attended to as a whole, packed with others of different
lengths (prompt); training runs over the same packed batches, backward pass
included (train).
"""
import math
import random

import numpy as np
import torch

own = False

E4M3_MAX = 448.0
SCALE_EXP_MIN, SCALE_EXP_MAX = -64, 60  # scales are powers of two in this range


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one decoding step of a full server: 256 requests get one token each
        dict(name="pages-step", op="pages", B=256, lo=1, hi=8192, add_lo=1, add_hi=1, page=64, short=False, mix=1),
        # prompts of very different lengths arrive at once, more than there are pages for
        dict(name="pages-prompts", op="pages", B=48, lo=1, hi=500, add_lo=1, add_hi=4096, page=16, short=True, mix=2),
        # the same decoding step: 256 new keys and values in pages that are partly filled
        dict(name="append-step", op="append", B=256, lo=1, hi=8192, add_lo=1, add_hi=1, Hkv=8, d=128, page=64,
             dtype="bf16", mix=3),
        # whole prompts go into the cache after their attention
        dict(name="append-prompts", op="append", B=13, lo=1, hi=33, add_lo=5, add_hi=8192, Hkv=4, d=64, page=16,
             dtype="fp16", mix=4),
        # one user, a short history: latency alone counts
        dict(name="decode-single", op="decode", B=1, Nq=1, lo=1000, hi=1000, Hq=32, Hkv=8, d=128, page=64,
             dtype="bf16", mix=5),
        # a full batch of chats of different lengths
        dict(name="decode-batch", op="decode", B=64, Nq=1, lo=100, hi=8192, Hq=32, Hkv=8, d=128, page=64,
             dtype="bf16", mix=6),
        # a few very long documents
        dict(name="decode-long", op="decode", B=4, Nq=1, lo=50001, hi=131072, Hq=32, Hkv=4, d=128, page=128,
             dtype="bf16", mix=7),
        # five drafted tokens a request are checked at once; some requests are shorter than the draft
        dict(name="decode-draft", op="decode", B=17, Nq=5, lo=1, hi=4096, Hq=14, Hkv=2, d=64, page=16,
             dtype="fp16", mix=8),
        # prompts that go on after a cached prefix
        dict(name="prompt-continued", op="prompt", B=24, lo=1, hi=400, pre_lo=0, pre_hi=2000, Hq=12, Hkv=4, d=64,
             causal=True, dtype="fp16", mix=9),
        # long documents packed with shorter ones
        dict(name="prompt-long", op="prompt", B=5, lo=700, hi=8192, pre_lo=0, pre_hi=0, Hq=16, Hkv=4, d=128,
             causal=True, dtype="bf16", mix=10),
        # a training batch packed from short texts, a head of keys for each of queries
        dict(name="train-ragged", op="train", B=16, lo=16, hi=2048, pre_lo=0, pre_hi=0, Hq=12, Hkv=12, d=64,
             causal=True, dtype="fp16", mix=11),
        # a training batch of longer texts, grouped heads
        dict(name="train-long", op="train", B=5, lo=300, hi=4096, pre_lo=0, pre_hi=0, Hq=16, Hkv=4, d=128,
             causal=True, dtype="bf16", mix=12),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["pages", "append", "decode", "decode", "prompt", "train"])
    c = dict(op=op, mix=rng.randrange(1 << 30))
    if op == "pages":
        c.update(B=_log(rng, 1, 1000), lo=0, hi=_log(rng, 1, 8192), page=rng.choice([16, 32, 64, 128]),
                 short=rng.random() < 0.3)
        c.update(add_lo=0, add_hi=max(1, _log(rng, 1, 4096) // max(1, c["B"] // 32)))
        return c
    d, dtype = rng.choice([64, 128]), rng.choice(["fp16", "bf16"])
    hkv = rng.choice([1, 2, 3, 4, 5, 8])
    c.update(d=d, dtype=dtype, Hkv=hkv)
    if op == "append":
        c.update(B=_log(rng, 1, 300), lo=0, hi=_log(rng, 1, 4096), page=rng.choice([16, 32, 64, 128]))
        c.update(add_lo=1, add_hi=max(1, _log(rng, 1, 8192) // max(1, c["B"] // 8)))
        return c
    g = rng.choice([1, 2, 3, 4, 7, 8, 16])
    c.update(Hq=hkv * g)
    if op == "decode":
        c.update(B=_log(rng, 1, 96), Nq=rng.choice([1, 1, 1, 2, 3, 8]), page=rng.choice([16, 32, 64, 128]))
        hi = max(1, min(100000, _log(rng, 1, 600000) // c["B"]))
        c.update(lo=rng.choice([1, max(1, hi // 8)]), hi=hi)
        return c
    c.update(B=_log(rng, 1, 40), causal=rng.random() < 0.8)
    top = 8192 if op == "prompt" else 4096
    while True:  # no dearer than the largest listed case of the kind
        hi = _log(rng, 1, top)
        pre = rng.choice([0, 0, _log(rng, 1, 2000)]) if op == "prompt" else 0
        if c["B"] * c["Hq"] * hi * (hi + pre) * d <= (5 * 16 * top * top * 128) // 4:
            break
    c.update(lo=hi // rng.choice([1, 8, 300]), hi=hi, pre_lo=0, pre_hi=pre)
    return c


def _spread(n, lo, hi, mix):
    """n whole numbers in [lo, hi], spread over their logarithm, both ends among them."""
    rng = random.Random(mix)
    v = [max(lo, min(hi, _log(rng, lo + 1, hi + 1) - 1)) for _ in range(n)]
    if n > 1:
        v[rng.randrange(n // 2)] = hi
        v[n // 2 + rng.randrange(n - n // 2)] = lo
    elif n:
        v[0] = hi
    return v


def _lens(c):
    """(lengths before, lengths added) of a case of the cache, (query, key lengths) of a packed one."""
    if c["op"] in ("pages", "append"):
        return _spread(c["B"], c["lo"], c["hi"], c["mix"]), _spread(c["B"], c["add_lo"], c["add_hi"], c["mix"] + 1)
    lq = _spread(c["B"], c["lo"], c["hi"], c["mix"])
    if c["op"] == "decode":
        return lq, lq
    pre = _spread(c["B"], c["pre_lo"], c["pre_hi"], c["mix"] + 1)
    return lq, [a + p for a, p in zip(lq, pre)]


def _ceil(a, b):
    return -(-a // b)


def _pairs(lq, lk, causal):
    """Scores that the mask keeps, one head."""
    if not causal:
        return sum(a * b for a, b in zip(lq, lk))
    return sum(a * (b - a) + a * (a + 1) // 2 for a, b in zip(lq, lk))


def work(c):
    a, b = _lens(c)
    if c["op"] == "pages":
        new = sum(_ceil(x + y, c["page"]) - _ceil(x, c["page"]) for x, y in zip(a, b))
        return {"bytes": 20 * c["B"] + 8 * sum(b) + 8 * new + 4 * c["B"], "flops": sum(b)}
    if c["op"] == "append":
        n = sum(b) * c["Hkv"] * c["d"] * 2  # keys and values
        touched = sum(_ceil(x + y, c["page"]) - x // c["page"] for x, y in zip(a, b))
        return {"bytes": 3 * n + 8 * sum(b) + 16 * touched * c["Hkv"], "flops": 3 * n}
    if c["op"] == "decode":
        rows = c["B"] * c["Nq"] * c["Hq"]
        pages = sum(_ceil(x, c["page"]) for x in a)
        return {"bytes": 2 * sum(a) * c["Hkv"] * c["d"] + pages * (8 * c["Hkv"] + 4) + rows * (4 * c["d"] + 4),
                "flops": 4 * sum(a) * c["Nq"] * c["Hq"] * c["d"]}
    p = _pairs(a, b, c["causal"]) * c["Hq"]
    q, kv = 2 * sum(a) * c["Hq"] * c["d"], 2 * sum(b) * c["Hkv"] * c["d"]
    lse = 4 * sum(a) * c["Hq"]
    if c["op"] == "prompt":
        return {"bytes": 2 * q + 2 * kv + lse, "flops": 4 * p * c["d"]}
    return {"bytes": 4 * q + 4 * kv + lse, "flops": 14 * p * c["d"]}


# ------------------------------------------------------------------ inputs
def _dtype(c):
    return torch.bfloat16 if c["dtype"] == "bf16" else torch.float16


def _pow2_scale(amax):
    """Smallest power of two s with amax <= 448 s, its exponent kept in range."""
    e = ((amax.float().contiguous().view(torch.int32) + 0x1FFFFF) >> 23) - 127 - 8
    e = e.clamp(SCALE_EXP_MIN, SCALE_EXP_MAX)
    return ((e + 127) << 23).view(torch.float32)


def _fill_cache(gen, pages, heads, page, d, dev):
    """A cache of normal values, pages of different sizes, some channels larger: (codes, scales)."""
    x = torch.randn((pages, heads, page, d), generator=gen, device=dev)
    x *= torch.exp2(torch.randint(-2, 2, (pages, heads, 1, 1), generator=gen, device=dev).float())
    x[..., ::29] *= 3.0
    s = _pow2_scale(x.abs().amax((2, 3)))
    return (x / s[..., None, None]).to(torch.float8_e4m3fn), s


def _cu(lens, dev):
    return torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device=dev)


def _tables(gen, counts, width, total, dev):
    """Block tables [B, width] of `counts` pages a request out of `total`, in no order; -1 behind them."""
    perm = torch.randperm(total, generator=gen, device=dev).to(torch.int32)
    cnt = torch.tensor(counts, device=dev)
    at = torch.cumsum(cnt, 0) - cnt
    j = torch.arange(width, device=dev)
    idx = (at[:, None] + j[None, :]).clamp(max=total - 1)
    return torch.where(j[None, :] < cnt[:, None], perm[idx], -1).to(torch.int32).contiguous(), perm[sum(counts):].contiguous()


def prepare(c, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    a, b = _lens(c)
    s = {"c": c}
    if c["op"] in ("pages", "append"):
        ps = c["page"]
        old = [_ceil(x, ps) for x in a]
        new = [_ceil(x + y, ps) for x, y in zip(a, b)]
        width, spare = max(max(new), 1), 3
        total = sum(new) + spare
        table, free = _tables(gen, old, width, total, dev)
        count = sum(new) - sum(old) + spare
        if c.get("short"):
            count = max(1, (6 * count) // 10)
        s.update(lens=torch.tensor(a, dtype=torch.int32, device=dev), add=torch.tensor(b, dtype=torch.int32, device=dev),
                 table=table, free=free, count=torch.tensor([count], dtype=torch.int32, device=dev), T=max(1, sum(b)))
        if c["op"] == "pages":
            return s
        slots = _plain_pages(s)[3]
        h, d, T = c["Hkv"], c["d"], s["T"]
        kc, ks = _fill_cache(gen, total, h, ps, d, dev)
        vc, vs = _fill_cache(gen, total, h, ps, d, dev)
        k = torch.randn((T, h, d), generator=gen, device=dev)
        k[..., ::29] *= 3.0
        v = torch.randn((T, h, d), generator=gen, device=dev)
        # now and then a token that the page's scale does not reach
        big = torch.rand((T, 1, 1), generator=gen, device=dev) < 0.03
        k, v = torch.where(big, 8 * k, k), torch.where(big, 8 * v, v)
        return {"c": c, "k": k.to(_dtype(c)), "v": v.to(_dtype(c)), "slots": slots, "kc": kc, "vc": vc, "ks": ks, "vs": vs}
    h, hq, d = c["Hkv"], c["Hq"], c["d"]
    if c["op"] == "decode":
        ps = c["page"]
        cnt = [_ceil(x, ps) for x in a]
        total = sum(cnt) + 1
        table, _ = _tables(gen, cnt, max(cnt), total, dev)
        kc, ks = _fill_cache(gen, total, h, ps, d, dev)
        vc, vs = _fill_cache(gen, total, h, ps, d, dev)
        lens = torch.tensor(a, dtype=torch.int32, device=dev)
        # the slots behind a request's last token hold what memory held: not numbers
        last = table.long().gather(1, ((lens.long() + ps - 1) // ps - 1)[:, None])[:, 0]
        row = torch.arange(ps, device=dev)[None, :] >= ((lens.long() - 1) % ps + 1)[:, None]
        for cache in (kc, vc):
            raw = cache.view(torch.uint8)
            raw[last] = torch.where(row[:, None, :, None], 0x7F, raw[last])
        q = torch.randn((c["B"], c["Nq"], hq, d), generator=gen, device=dev).to(_dtype(c))
        s.update(q=q, kc=kc, vc=vc, ks=ks, vs=vs, table=table, lens=lens, longest=max(a), scale=d ** -0.5)
        return s
    q = torch.randn((sum(a), hq, d), generator=gen, device=dev).to(_dtype(c))
    k = torch.randn((sum(b), h, d), generator=gen, device=dev).to(_dtype(c))
    v = torch.randn((sum(b), h, d), generator=gen, device=dev).to(_dtype(c))
    s.update(q=q, k=k, v=v, cu_q=_cu(a, dev), cu_k=_cu(b, dev), max_q=max(a), max_k=max(b), scale=d ** -0.5)
    if c["op"] == "train":
        s["do"] = torch.randn((sum(a), hq, d), generator=gen, device=dev).to(_dtype(c))
    return s


# ------------------------------------------------------------------ one pass
def run(s):
    op = s["c"]["op"]
    if own:
        return _own(op, s)
    if op == "pages":
        return _plain_pages(s)
    if op == "append":
        return _plain_append(s)
    if op == "decode":
        return _plain_decode(s)
    return _plain_packed(s, op == "train")


def _own(op, s):
    from exact_tiled_attention_22_gb300 import attn
    if op == "pages":
        new, granted, cu, slots, left = attn.pages_extend(s["lens"], s["add"], s["table"], s["free"], s["count"],
                                                          s["c"]["page"], s["T"])
        return new, granted, cu, slots, left, s["table"]
    if op == "append":
        attn.kv8_append(s["k"], s["v"], s["slots"], s["kc"], s["vc"], s["ks"], s["vs"])
        return s["kc"], s["vc"], s["ks"], s["vs"]
    if op == "decode":
        return attn.kv8_decode(s["q"], s["kc"], s["vc"], s["ks"], s["vs"], s["table"], s["lens"], s["scale"], True)
    o, lse = attn.varlen_fwd(s["q"], s["k"], s["v"], s["cu_q"], s["cu_k"], s["scale"], s["c"]["causal"])
    if op == "prompt":
        return o, lse
    dq, dk, dv = attn.varlen_bwd(s["q"], s["k"], s["v"], o, lse, s["do"], s["cu_q"], s["cu_k"], s["scale"],
                                 s["c"]["causal"])
    return o, lse, dq, dk, dv


def _plain_pages(s):
    """Requests in order take their new pages from the top of the stack of free ones; a request whose pages, with those of
    all before it, are more than there are gets none of its tokens in."""
    ps, T, table = s["c"]["page"], s["T"], s["table"]
    old, add, width = s["lens"].long(), s["add"].long(), table.shape[1]
    count = s["count"].long()
    p_old, p_new = (old + ps - 1) // ps, (old + add + ps - 1) // ps
    valid = (add >= 0) & (p_new <= width)
    need = torch.where(valid, p_new - p_old, 0)
    incl = torch.cumsum(need, 0)
    served = valid & ((need == 0) | (incl <= count))
    granted = torch.where(served, add, 0)
    cu = torch.nn.functional.pad(torch.cumsum(add.clamp(min=0), 0), (1, 0))
    j = torch.arange(width, device=table.device)
    fresh = served[:, None] & (j >= p_old[:, None]) & (j < p_new[:, None])
    at = count - 1 - ((incl - need)[:, None] + j - p_old[:, None])
    table.copy_(torch.where(fresh, s["free"].long()[at.clamp(0, s["free"].shape[0] - 1)], table.long()))
    t = torch.arange(T, device=table.device)
    b = torch.searchsorted(cu[1:], t, right=True).clamp(max=old.shape[0] - 1)
    pos = old[b] + t - cu[b]
    page = table[b, (pos // ps).clamp(max=width - 1)].long()
    slots = torch.where((t < cu[-1]) & served[b] & (page >= 0), page * ps + pos % ps, -1)
    left = count - torch.where(served, need, 0).sum()
    return (old + granted).int(), granted.int(), cu.int(), slots, left.int(), table


def _plain_append(s):
    """A page's scale is the smallest power of two that reaches every value put into it; when a new token needs a larger
    one, the tokens before it in the page are rounded again.  A page that starts anew forgets its old scale."""
    slots = s["slots"]
    ps = s["kc"].shape[2]
    page, off = slots // ps, slots % ps
    used = slots >= 0
    page = torch.where(used, page, 0)
    for x, cache, scale in ((s["k"], s["kc"], s["ks"]), (s["v"], s["vc"], s["vs"])):
        x = x.float()
        n, h = scale.shape
        top = torch.zeros((n, h), device=x.device).scatter_reduce_(
            0, page[:, None].expand(-1, h), torch.where(used[:, None], x.abs().amax(2), 0.0), "amax")
        first = torch.full((n,), ps, device=x.device).scatter_reduce_(0, page, torch.where(used, off, ps), "amin")
        touched = (first < ps)[:, None]
        new = _pow2_scale(top)
        new = torch.where((first > 0)[:, None], torch.maximum(new, scale), new)
        new = torch.where(touched, new, scale)
        kept = cache.float() * (scale / new)[..., None, None]
        row = torch.arange(ps, device=x.device)
        again = touched[..., None, None] & (row[None, None, :, None] < first[:, None, None, None]) & (new > scale)[..., None, None]
        codes = torch.where(again, kept.to(torch.float8_e4m3fn).view(torch.uint8), cache.view(torch.uint8))
        q = (x / new[page][..., None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn).view(torch.uint8)
        # tokens without a slot are written to a page behind the last one, which is left out
        room = torch.cat([codes, torch.zeros_like(codes[:1])])
        room[torch.where(used, page, n), :, off] = q
        cache.view(torch.uint8).copy_(room[:n])
        scale.copy_(new)
    return s["kc"], s["vc"], s["ks"], s["vs"]


def _softmax_rows(scores, keep):
    """exp(scores - log-sum-exp) in place and the log-sum-exp; rows that keep nothing are zeros and -inf."""
    scores.masked_fill_(~keep, -math.inf)
    top = scores.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    scores.sub_(top).exp_()
    total = scores.sum(-1, keepdim=True)
    scores.div_(torch.where(total > 0, total, 1.0))
    return scores, (torch.log(total) + top)[..., 0]


def _plain_decode(s):
    c = s["c"]
    B, nq, hq, h, d, ps = c["B"], c["Nq"], c["Hq"], c["Hkv"], c["d"], c["page"]
    table = s["table"].long()
    n = table.shape[1] * ps
    j = torch.arange(n, device=table.device)
    live = (j[None, :] < s["lens"][:, None])[:, None, :, None]

    def whole(cache, scale):
        page = table.clamp(min=0)
        x = cache.view(torch.uint8)[page].view(torch.float8_e4m3fn).float() * scale[page][..., None, None]
        return torch.where(live, x.permute(0, 2, 1, 3, 4).reshape(B, h, n, d), 0.0)

    q = s["q"].float().view(B, nq, h, hq // h, d).permute(0, 2, 3, 1, 4).reshape(B, h, -1, d)
    scores = torch.matmul(q, whole(s["kc"], s["ks"]).transpose(2, 3)).view(B, h, hq // h, nq, n)
    scores *= s["scale"]
    last = s["lens"][:, None] - nq + torch.arange(nq, device=table.device)
    p, lse = _softmax_rows(scores, (j <= last[:, :, None])[:, None, None])
    o = torch.matmul(p.view(B, h, -1, n), whole(s["vc"], s["vs"])).view(B, h, hq // h, nq, d)
    return o.permute(0, 3, 1, 2, 4).reshape(B, nq, hq, d).to(s["q"].dtype), lse.reshape(B, hq, nq)


def _plain_packed(s, train):
    c = s["c"]
    B, hq, h, d = c["B"], c["Hq"], c["Hkv"], c["d"]
    g, nq, nk = hq // h, s["max_q"], s["max_k"]
    dev = s["q"].device

    def unpack(x, cu, n):  # packed [T, heads, d] -> [B, heads, n, d] in 32 bits, zeros behind the end
        i = torch.arange(n, device=dev)
        at = (cu[:-1, None] + i).clamp(max=x.shape[0] - 1).long()
        live = (i < (cu[1:] - cu[:-1])[:, None])[..., None, None]
        return torch.where(live, x[at].float(), 0.0).transpose(1, 2)

    def places(cu, total):
        t = torch.arange(total, device=dev, dtype=torch.int32)
        b = torch.searchsorted(cu[1:].contiguous(), t, right=True)
        return b, t - cu[b]

    def pack(x, cu, total):  # [B, heads, n, ...] -> packed
        b, i = places(cu, total)
        return x[b, :, i]

    tq, tk = s["q"].shape[0], s["k"].shape[0]
    q = unpack(s["q"], s["cu_q"], nq).reshape(B, h, g * nq, d)
    k, v = unpack(s["k"], s["cu_k"], nk), unpack(s["v"], s["cu_k"], nk)
    scores = torch.matmul(q, k.transpose(2, 3)).view(B, h, g, nq, nk)
    scores *= s["scale"]
    lq, lk = s["cu_q"][1:] - s["cu_q"][:-1], s["cu_k"][1:] - s["cu_k"][:-1]
    i, j = torch.arange(nq, device=dev), torch.arange(nk, device=dev)
    keep = (i < lq[:, None])[:, :, None] & (j < lk[:, None])[:, None, :]
    if c["causal"]:
        keep = keep & (j[None, None, :] <= (lk - lq)[:, None, None] + i[None, :, None])
    p, lse = _softmax_rows(scores, keep[:, None, None])
    p = p.view(B, h, g * nq, nk)
    o = torch.matmul(p, v).view(B, hq, nq, d)
    out = pack(o, s["cu_q"], tq).to(s["q"].dtype)
    lse = pack(lse.reshape(B, hq, nq), s["cu_q"], tq).t().contiguous()
    if not train:
        return out, lse
    do = unpack(s["do"], s["cu_q"], nq)
    delta = (do * o).sum(-1).view(B, h, g * nq, 1)
    do = do.reshape(B, h, g * nq, d)
    dv = torch.matmul(p.transpose(2, 3), do)
    ds = torch.matmul(do, v.transpose(2, 3))
    ds.sub_(delta).mul_(p)
    dq = (torch.matmul(ds, k) * s["scale"]).view(B, hq, nq, d)
    dk = torch.matmul(ds.transpose(2, 3), q) * s["scale"]
    t = s["q"].dtype
    return (out, lse, pack(dq, s["cu_q"], tq).to(t), pack(dk, s["cu_k"], tk).to(t), pack(dv, s["cu_k"], tk).to(t))


# ------------------------------------------------------------------ definitions in 64 bits
def _pow2(e):
    """2^e in 64 bits, exactly."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _e4m3(y):
    """The e4m3 value nearest to y (64 bits; ties to the even mantissa)."""
    y = y.clamp(-448.0, 448.0)
    e = torch.frexp(y.abs().clamp(min=2.0 ** -6))[1] - 1
    return torch.round(y * _pow2(3 - e)) * _pow2(e - 3)


def _exact_append(c, s):
    ps, slots = c["page"], s["slots"].tolist()
    runs, t = [], 0
    while t < len(slots):  # tokens that go to one page, one after the other
        u = t + 1
        while u < len(slots) and slots[u] >= 0 and slots[u] // ps == slots[t] // ps:
            u += 1
        if slots[t] >= 0:
            runs.append((t, u, slots[t] // ps, slots[t] % ps))
        t = u
    outs = []
    for x, cache, scale in ((s["k"], s["kc"], s["ks"]), (s["v"], s["vc"], s["vs"])):
        x, val, sc = x.double(), cache.double(), scale.double()
        for t, u, page, first in runs:
            top = x[t:u].abs().amax((0, 2))
            m, e = torch.frexp(top / 448.0)  # m 2^e with m in [0.5, 1)
            e = torch.where(top == 0, SCALE_EXP_MIN, torch.where(m == 0.5, e - 1, e))
            new = _pow2(e.clamp(SCALE_EXP_MIN, SCALE_EXP_MAX))
            if first:
                new = torch.maximum(new, sc[page])
                val[page, :, :first] = _e4m3(val[page, :, :first] * (sc[page] / new)[:, None, None])
            val[page, :, first:first + u - t] = _e4m3(x[t:u].transpose(0, 1) / new[:, None, None])
            sc[page] = new
        outs.append((val, sc))
    return outs[0][0], outs[1][0], outs[0][1], outs[1][1]


def _exact_rows(q, k, v, scale, last):
    """Row i of q sees keys j <= last[i]: (o, lse, p) in 64 bits."""
    x = (q @ k.t()) * scale
    x = x.masked_fill(torch.arange(k.shape[0], device=q.device)[None, :] > last[:, None], -math.inf)
    lse = torch.logsumexp(x, 1)
    p = torch.exp(x - torch.where(lse == -math.inf, 0.0, lse)[:, None])
    return p @ v, lse, p


def exact(c, seed):
    if c["op"] == "pages":
        return None
    s = prepare(c, seed)
    if c["op"] == "append":
        return _exact_append(c, s)
    hq, h = c["Hq"], c["Hkv"]
    g = hq // h
    if c["op"] == "decode":
        o = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
        lse = torch.full((c["B"], hq, c["Nq"]), -math.inf, dtype=torch.float64, device="cuda")
        for b, n in enumerate(s["lens"].tolist()):
            pages = s["table"][b, :_ceil(n, c["page"])].long()
            last = n - c["Nq"] + torch.arange(c["Nq"], device="cuda")
            for kv in range(h):
                k, v = ((cache[pages, kv].double() * sc[pages, kv].double()[:, None, None]).reshape(-1, c["d"])[:n]
                        for cache, sc in ((s["kc"].view(torch.float8_e4m3fn), s["ks"]), (s["vc"], s["vs"])))
                for head in range(kv * g, kv * g + g):
                    o[b, :, head], lse[b, head], _ = _exact_rows(s["q"][b, :, head].double(), k, v, s["scale"], last)
        return o, lse
    a, b = _lens(c)
    if _pairs(a, b, False) * hq * c["d"] > 4e11:  # over about 20 seconds in 64 bits
        return None
    train = c["op"] == "train"
    z = lambda x: torch.zeros(x.shape, dtype=torch.float64, device="cuda")  # noqa: E731
    o, lse = z(s["q"]), torch.zeros((hq, s["q"].shape[0]), dtype=torch.float64, device="cuda")
    dq, dk, dv = z(s["q"]), z(s["k"]), z(s["v"])
    q0 = k0 = 0
    for lq, lk in zip(a, b):
        last = (torch.arange(lq, device="cuda") + lk - lq) if c["causal"] else torch.full((lq,), lk, device="cuda")
        rows, keys = slice(q0, q0 + lq), slice(k0, k0 + lk)
        for head in range(hq):
            q, k, v = s["q"][rows, head].double(), s["k"][keys, head // g].double(), s["v"][keys, head // g].double()
            o[rows, head], lse[head, rows], p = _exact_rows(q, k, v, s["scale"], last)
            if train:
                do = s["do"][rows, head].double()
                dp = do @ v.t()
                ds = p * (dp - (p * dp).sum(1, keepdim=True))
                dv[keys, head // g] += p.t() @ do
                dq[rows, head] = ds @ k * s["scale"]
                dk[keys, head // g] += ds.t() @ q * s["scale"]
        q0, k0 = q0 + lq, k0 + lk
    return (o, lse, dq, dk, dv) if train else (o, lse)
