"""Serving from a paged cache held in 4 bits: the operators that are measured,
their plain forms in torch, and their definitions in 64 bits.

A cached key or value is a code of 4 bits times a scale.  The codes stand for
0, 0.5, 1, 1.5, 2, 3, 4, 6 and their negatives (sign, two bits of exponent, one of
mantissa), two to a byte, the even channel in the low half; every 32 channels
of a token and head share a scale in bf16.  A token is rounded by itself, so
nothing that is in the cache is ever rounded again.
  append   rounds new keys and values into their slots,
  decode   attends from the newest tokens of every request to its whole cache,
  read     gives a request's cached keys and values back as packed 16-bit rows,
           which is what a prompt attends to that goes on after a cached prefix;
  read8    the same from the cache in 8 bits (e4m3, a scale for each page and head).
"""
import math
import random

import numpy as np
import torch

own = False

GROUP = 32                              # channels that share a scale
SCALE_MIN, SCALE_MAX = 2.0 ** -64, 2.0 ** 60


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one decoding step of a full server: 256 new keys and values in pages that are partly filled
        dict(name="append-step", op="append", B=256, lo=1, hi=8192, add_lo=1, add_hi=1, H=8, d=128, page=64,
             dtype="bf16", mix=1),
        # whole prompts go into the cache after their attention
        dict(name="append-prompts", op="append", B=13, lo=1, hi=33, add_lo=5, add_hi=8192, H=4, d=64, page=16,
             dtype="fp16", mix=2),
        # one user, a short history: latency alone counts
        dict(name="decode-single", op="decode", B=1, Nq=1, lo=1000, hi=1000, Hq=32, H=8, d=128, page=64,
             dtype="bf16", mix=3),
        # a full batch of chats of different lengths
        dict(name="decode-batch", op="decode", B=64, Nq=1, lo=100, hi=8192, Hq=32, H=8, d=128, page=64,
             dtype="bf16", mix=4),
        # a few very long documents
        dict(name="decode-long", op="decode", B=4, Nq=1, lo=50001, hi=131072, Hq=32, H=8, d=128, page=128,
             dtype="bf16", mix=5),
        # five drafted tokens a request are checked at once; some requests are shorter than the draft
        dict(name="decode-draft", op="decode", B=17, Nq=5, lo=1, hi=4096, Hq=14, H=2, d=64, page=16,
             dtype="fp16", mix=6),
        # short prompts go on after cached prefixes: the prefixes are read in front of the new rows
        dict(name="read-prefix", op="read", B=24, lo=1, hi=2000, room=400, H=4, d=64, page=16, dtype="fp16", mix=7),
        # a turn of a few long conversations
        dict(name="read-long", op="read", B=5, lo=700, hi=32768, room=0, H=8, d=128, page=64, dtype="bf16", mix=8),
        # the same two from the cache in 8 bits
        dict(name="read8-prefix", op="read8", B=24, lo=1, hi=2000, room=400, H=4, d=64, page=16, dtype="fp16", mix=9),
        dict(name="read8-long", op="read8", B=5, lo=700, hi=32768, room=0, H=8, d=128, page=64, dtype="bf16", mix=10),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "decode", "decode", "read", "read8"])
    c = dict(op=op, mix=rng.randrange(1 << 30), d=rng.choice([64, 128]), dtype=rng.choice(["fp16", "bf16"]),
             H=rng.choice([1, 2, 3, 4, 5, 8]), page=rng.choice([16, 32, 64, 128]))
    if op == "append":
        c.update(B=_log(rng, 1, 300), lo=0, hi=_log(rng, 1, 4096))
        c.update(add_lo=1, add_hi=max(1, _log(rng, 1, 8192) // max(1, c["B"] // 8)))
    elif op == "decode":
        c.update(B=_log(rng, 1, 96), Nq=rng.choice([1, 1, 1, 2, 3, 8]), Hq=c["H"] * rng.choice([1, 2, 3, 4, 7, 8, 16]))
        hi = max(1, min(100000, _log(rng, 1, 600000) // c["B"]))
        c.update(lo=rng.choice([1, max(1, hi // 8)]), hi=hi)
    else:
        c.update(B=_log(rng, 1, 100))
        hi = max(1, min(32768, _log(rng, 1, 80000) // c["B"]))
        c.update(lo=rng.choice([0, max(1, hi // 8)]), hi=hi, room=rng.choice([0, 1, _log(rng, 1, 500)]))
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
    """(lengths of the requests, tokens that come after them) of a case."""
    a = _spread(c["B"], c["lo"], c["hi"], c["mix"])
    if c["op"] == "append":
        return a, _spread(c["B"], c["add_lo"], c["add_hi"], c["mix"] + 1)
    return a, _spread(c["B"], 0, c["room"], c["mix"] + 1) if c.get("room") else [0] * c["B"]


def _ceil(a, b):
    return -(-a // b)


def work(c):
    a, b = _lens(c)
    h, d = c["H"], c["d"]
    row = 2 * h * (d // 2 + d // GROUP * 2)  # codes and scales of a token's key and value
    if c["op"] == "append":
        return {"bytes": sum(b) * (4 * h * d + row + 8), "flops": 6 * sum(b) * h * d}
    pages = sum(_ceil(x, c["page"]) for x in a)
    if c["op"] == "decode":
        rows = c["B"] * c["Nq"] * c["Hq"]
        return {"bytes": sum(a) * row + 4 * pages + rows * (4 * d + 4), "flops": 4 * sum(a) * c["Nq"] * c["Hq"] * d}
    if c["op"] == "read8":
        return {"bytes": 6 * sum(a) * h * d + pages * (8 * h + 4), "flops": 2 * sum(a) * h * d}
    return {"bytes": sum(a) * (4 * h * d + row) + 4 * pages, "flops": 2 * sum(a) * h * d}


# ------------------------------------------------------------------ inputs
def _dtype(c):
    return torch.bfloat16 if c["dtype"] == "bf16" else torch.float16


def _quantise(x):
    """Rows of d channels in 32 bits to (codes [.., d / 2] uint8, scales [.., d / 32] bf16): the scale is the largest
    magnitude over 6, the code the nearest of the eight magnitudes (ties to the even one), the sign kept."""
    g = x.reshape(*x.shape[:-1], -1, GROUP)
    s = (g.abs().amax(-1) / 6).clamp(SCALE_MIN, SCALE_MAX).to(torch.bfloat16)
    y = g / s.float()[..., None]
    a = y.abs()
    m = torch.zeros(a.shape, dtype=torch.uint8, device=a.device)
    for low in (0.25, 1.25, 2.5, 5.0):  # a tie goes down
        m += a > low
    for up in (0.75, 1.75, 3.5):  # a tie goes up
        m += a >= up
    m |= torch.signbit(y).to(torch.uint8) << 3
    m = m.reshape(x.shape)
    return m[..., 0::2] | (m[..., 1::2] << 4), s


def _values(codes, scales):
    """What codes and scales stand for, in 32 bits: [.., d]."""
    both = torch.stack((codes & 15, codes >> 4), -1).reshape(*codes.shape[:-1], -1)
    e, f = ((both >> 1) & 3).float(), (both & 1).float()
    v = torch.where(e > 0, (1 + 0.5 * f) * torch.exp2(e - 1), 0.5 * f)
    v = torch.where(both >= 8, -v, v)
    return (v.reshape(*v.shape[:-1], -1, GROUP) * scales.float()[..., None]).reshape(v.shape)


def _normal_pages(gen, pages, heads, page, d, dev):
    """Normal values, pages of different sizes, some channels larger."""
    x = torch.randn((pages, heads, page, d), generator=gen, device=dev)
    x *= torch.exp2(torch.randint(-2, 2, (pages, heads, 1, 1), generator=gen, device=dev).float())
    x[..., ::29] *= 3.0
    return x


def _fill_cache(gen, pages, heads, page, d, dev):
    """A cache of such pages in 4 bits: (codes, scales)."""
    codes = torch.empty((pages, heads, page, d // 2), dtype=torch.uint8, device=dev)
    scales = torch.empty((pages, heads, page, d // GROUP), dtype=torch.bfloat16, device=dev)
    step = max(1, (1 << 26) // (heads * page * d))
    for p in range(0, pages, step):
        n = min(step, pages - p)
        codes[p:p + n], scales[p:p + n] = _quantise(_normal_pages(gen, n, heads, page, d, dev))
    return codes, scales


def _fill_cache8(gen, pages, heads, page, d, dev):
    """A cache of such pages in 8 bits: e4m3 codes, a power of two for each page and head."""
    x = _normal_pages(gen, pages, heads, page, d, dev)
    s = torch.exp2(torch.ceil(torch.log2(x.abs().amax((2, 3)) / 448)))
    return (x / s[..., None, None]).clamp(-448, 448).to(torch.float8_e4m3fn), s


def _cu(lens, dev):
    return torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device=dev)


def _tables(gen, counts, total, dev):
    """Block tables [B, width] of `counts` pages a request out of `total`, in no order; -1 behind them."""
    perm = torch.randperm(total, generator=gen, device=dev)
    cnt = torch.tensor(counts, device=dev)
    at = torch.cumsum(cnt, 0) - cnt
    j = torch.arange(max(max(counts), 1), device=dev)
    idx = (at[:, None] + j[None, :]).clamp(max=total - 1)
    return torch.where(j[None, :] < cnt[:, None], perm[idx], -1).to(torch.int32).contiguous()


def prepare(c, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    a, b = _lens(c)
    h, d, ps = c["H"], c["d"], c["page"]
    ends = [x + y for x, y in zip(a, b)] if c["op"] == "append" else a
    counts = [_ceil(x, ps) for x in ends]
    total = sum(counts) + 1
    table = _tables(gen, counts, total, dev)
    lens = torch.tensor(a, dtype=torch.int32, device=dev)
    fill = _fill_cache8 if c["op"] == "read8" else _fill_cache
    # (one more page behind the cache: where the plain form of append puts tokens that have no slot)
    spare = c["op"] == "append"
    kc, ks = fill(gen, total + spare, h, ps, d, dev)
    vc, vs = fill(gen, total + spare, h, ps, d, dev)
    s = {"c": c, "table": table, "lens": lens, "kc": kc[:total], "vc": vc[:total], "ks": ks[:total], "vs": vs[:total]}
    if c["op"] == "append":
        T = sum(b) + 3
        req = torch.repeat_interleave(torch.arange(len(b), device=dev), torch.tensor(b, device=dev))
        cu = _cu(b, dev).long()
        pos = lens.long()[req] + torch.arange(sum(b), device=dev) - cu[req]
        slots = table.long()[req, pos // ps] * ps + pos % ps
        # (the list is padded, as in a captured step: the last entries have no slot)
        slots = torch.cat([slots, torch.full((3,), -1, device=dev)])
        k = torch.randn((T, h, d), generator=gen, device=dev)
        k[..., ::29] *= 3.0
        v = torch.randn((T, h, d), generator=gen, device=dev)
        s.update(k=k.to(_dtype(c)), v=v.to(_dtype(c)), slots=slots, room=(kc, vc, ks, vs))
    elif c["op"] == "decode":
        q = torch.randn((c["B"], c["Nq"], c["Hq"], d), generator=gen, device=dev).to(_dtype(c))
        s.update(q=q, scale=d ** -0.5)
    else:
        rows = [x + y for x, y in zip(a, b)]
        k = torch.randn((max(1, sum(rows)), h, d), generator=gen, device=dev).to(_dtype(c))
        v = torch.randn((max(1, sum(rows)), h, d), generator=gen, device=dev).to(_dtype(c))
        s.update(cu=_cu(rows, dev), k=k, v=v)
    return s


# ------------------------------------------------------------------ one pass
def run(s):
    op = s["c"]["op"]
    if own:
        return _own(op, s)
    return {"append": _plain_append, "decode": _plain_decode, "read": _plain_read, "read8": _plain_read}[op](s)


def _own(op, s):
    from exact_tiled_attention_22_gb300 import attn
    if op == "append":
        attn.kv4_append(s["k"], s["v"], s["slots"], s["kc"], s["vc"], s["ks"], s["vs"])
        return s["kc"], s["vc"], s["ks"], s["vs"]
    if op == "decode":
        return attn.kv4_decode(s["q"], s["kc"], s["vc"], s["ks"], s["vs"], s["table"], s["lens"], s["scale"], True)
    read = attn.kv4_read if op == "read" else attn.kv8_read
    return read(s["kc"], s["vc"], s["ks"], s["vs"], s["table"], s["lens"], s["cu"], s["k"].shape[0], s["k"].dtype,
                s["k"], s["v"])


def _plain_append(s):
    """Codes are whole numbers, and equal: the scales and the roundings are exact functions of the inputs."""
    ps = s["kc"].shape[2]
    slots = s["slots"]
    page = torch.where(slots >= 0, slots // ps, s["kc"].shape[0])
    off = torch.where(slots >= 0, slots % ps, 0)
    kc, vc, ks, vs = s["room"]
    for x, cache, scale in ((s["k"], kc, ks), (s["v"], vc, vs)):
        codes, sc = _quantise(x.float())
        cache[page, :, off] = codes
        scale[page, :, off] = sc
    return s["kc"], s["vc"], s["ks"], s["vs"]


def _plain_decode(s):
    c = s["c"]
    B, nq, hq, h, d, ps = c["B"], c["Nq"], c["Hq"], c["H"], c["d"], c["page"]
    table = s["table"].long().clamp(min=0)
    n = table.shape[1] * ps
    j = torch.arange(n, device=table.device)
    live = (j[None, :] < s["lens"][:, None])[:, None, :, None]

    def whole(cache, scale):
        x = _values(cache[table], scale[table])
        return torch.where(live, x.permute(0, 2, 1, 3, 4).reshape(B, h, n, d), 0.0)

    q = s["q"].float().view(B, nq, h, hq // h, d).permute(0, 2, 3, 1, 4).reshape(B, h, -1, d)
    x = torch.matmul(q, whole(s["kc"], s["ks"]).transpose(2, 3)).view(B, h, hq // h, nq, n)
    x *= s["scale"]
    last = s["lens"][:, None] - nq + torch.arange(nq, device=table.device)
    x.masked_fill_(~(j <= last[:, :, None])[:, None, None], -math.inf)
    top = x.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    x.sub_(top).exp_()
    total = x.sum(-1, keepdim=True)
    x.div_(torch.where(total > 0, total, 1.0))
    o = torch.matmul(x.view(B, h, -1, n), whole(s["vc"], s["vs"])).view(B, h, hq // h, nq, d)
    lse = (torch.log(total) + top)[..., 0].reshape(B, hq, nq)
    return o.permute(0, 3, 1, 2, 4).reshape(B, nq, hq, d).to(s["q"].dtype), lse


def _plain_read(s):
    """Rows behind a request's cached tokens (its new ones) stay as they are."""
    ps, cu, lens = s["kc"].shape[2], s["cu"].long(), s["lens"].long()
    t = torch.arange(s["k"].shape[0], device=cu.device)
    b = torch.searchsorted(cu[1:].contiguous(), t, right=True).clamp(max=lens.shape[0] - 1)
    i = t - cu[b]
    cached = (i < lens[b])[:, None, None]
    page = s["table"].long()[b, (i // ps).clamp(max=s["table"].shape[1] - 1)].clamp(min=0)
    for out, cache, scale in ((s["k"], s["kc"], s["ks"]), (s["v"], s["vc"], s["vs"])):
        if s["c"]["op"] == "read8":
            x = cache.view(torch.uint8)[page, :, i % ps].view(torch.float8_e4m3fn).float() * scale[page][..., None]
        else:
            x = _values(cache[page, :, i % ps], scale[page, :, i % ps])
        out.copy_(torch.where(cached, x.to(out.dtype), out))
    return s["k"], s["v"]


# ------------------------------------------------------------------ definitions in 64 bits
_GRID = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _exact_codes(x):
    """Codes and scales of rows x [T, H, d] in 64 bits: the scale to 8 bits of mantissa, the nearest of the grid."""
    T, h, d = x.shape
    g = x.double().view(T, h, d // GROUP, GROUP)
    s = g.abs().amax(-1) / 6
    m, e = torch.frexp(s)
    s = torch.ldexp(torch.round(m * 256), e - 8).clamp(SCALE_MIN, SCALE_MAX)
    grid = torch.tensor(_GRID, dtype=torch.float64, device=x.device)
    far = (g.abs()[..., None] - grid * s[..., None, None]).abs()
    # (of two that are equally near, the one with the even code)
    even = torch.arange(8, device=x.device) % 2 == 0
    best = far.amin(-1, keepdim=True)
    near = far == best
    near_even = near & even
    code = torch.where(near_even.any(-1), near_even.int().argmax(-1), near.int().argmax(-1))
    code = (code + 8 * torch.signbit(g)).view(T, h, d // 2, 2)
    return (code[..., 0] + 16 * code[..., 1]).to(torch.uint8), s


def _exact_values(codes, scales):
    grid = torch.tensor(_GRID + tuple(-x for x in _GRID), dtype=torch.float64, device=codes.device)
    x = torch.empty((*codes.shape[:-1], 2 * codes.shape[-1]), dtype=torch.float64, device=codes.device)
    x[..., 0::2] = grid[(codes % 16).long()]
    x[..., 1::2] = grid[(codes // 16).long()]
    return x * scales.double().repeat_interleave(GROUP, -1)


def exact(c, seed):
    s = prepare(c, seed)
    ps, h, d = c["page"], c["H"], c["d"]
    if c["op"] == "append":
        outs = []
        slots = s["slots"]
        used = slots >= 0
        for x, cache, scale in ((s["k"], s["kc"], s["ks"]), (s["v"], s["vc"], s["vs"])):
            codes, sc = _exact_codes(x[used])
            cache, scale = cache.clone(), scale.double()
            cache[slots[used] // ps, :, slots[used] % ps] = codes
            scale[slots[used] // ps, :, slots[used] % ps] = sc
            outs.append((cache, scale))
        return outs[0][0], outs[1][0], outs[0][1], outs[1][1]
    a, b = _lens(c)
    if c["op"] != "decode":
        k, v = s["k"].double(), s["v"].double()
        row = 0
        for i, (n, room) in enumerate(zip(a, b)):
            pages = s["table"][i, :_ceil(n, ps)].long()
            for out, cache, sc in ((k, s["kc"], s["ks"]), (v, s["vc"], s["vs"])):
                x = cache[pages].double() * sc[pages].double()[..., None, None] if c["op"] == "read8" else \
                    _exact_values(cache[pages], sc[pages])
                out[row:row + n] = x.transpose(1, 2).reshape(-1, h, d)[:n]
            row += n + room
        return k, v
    g = c["Hq"] // h
    o = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full((c["B"], c["Hq"], c["Nq"]), -math.inf, dtype=torch.float64, device="cuda")
    for i, n in enumerate(a):
        pages = s["table"][i, :_ceil(n, ps)].long()
        last = n - c["Nq"] + torch.arange(c["Nq"], device="cuda")
        behind = torch.arange(n, device="cuda")[None, :] > last[:, None]
        for kv in range(h):
            k, v = (_exact_values(cache[pages, kv], sc[pages, kv]).reshape(-1, d)[:n]
                    for cache, sc in ((s["kc"], s["ks"]), (s["vc"], s["vs"])))
            for head in range(kv * g, kv * g + g):
                x = (s["q"][i, :, head].double() @ k.t() * s["scale"]).masked_fill(behind, -math.inf)
                r = torch.logsumexp(x, 1)
                lse[i, head] = r
                o[i, :, head] = torch.exp(x - torch.where(r == -math.inf, 0.0, r)[:, None]) @ v
    return o, lse
