"""The paged cache in 4 bits written out in 64 bits (see plain64 for attention and
its bounds).  u is half a step of the 16-bit type relative to the value."""
import math

import torch

import plain64

GRID = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64)


def quantise(x):
    """x [.., d] in float64 -> codes uint8 [.., d / 2], scales float64 [.., d / 32] (NaN where
    the group holds one)."""
    g = x.unflatten(-1, (-1, 32))
    m, e = torch.frexp(g.abs().amax(-1) / 6)
    s = torch.where(torch.isinf(m), 2.0 ** 60, torch.round(m * 256) * torch.exp2((e - 8).double()))
    s = s.clamp(2.0 ** -64, 2.0 ** 60)
    y = (g.abs() / s[..., None]).clamp_max(6.0)
    # nearest of the grid; the borders are ties and go to the even code
    code = torch.zeros(y.shape, dtype=torch.int64)
    for i in range(1, 8):
        border = (GRID[i - 1] + GRID[i]) / 2
        code += (y > border) | ((y == border) & (i % 2 == 0))
    code = (code + 8 * torch.signbit(g)).flatten(-2).unflatten(-1, (-1, 2))
    return (code[..., 0] + 16 * code[..., 1]).to(torch.uint8), s


def values(codes, scales):
    """What codes and scales stand for, [.., d] in float64."""
    two = torch.stack((codes & 15, codes >> 4), -1).reshape(*codes.shape[:-1], -1).long()
    v = torch.where(two >= 8, -GRID[two & 7], GRID[two & 7])
    return v * scales.double().repeat_interleave(32, -1)


def append(x, slots, codes, scales):
    """(codes, scales) after the tokens x [T, H, d] (float64) have gone to `slots`."""
    codes, scales = codes.clone(), scales.clone()
    P, H, page, _ = codes.shape
    at = torch.tensor(slots)
    used = (at >= 0) & (at < P * page)
    c, s = quantise(x[used])
    codes[at[used] // page, :, at[used] % page] = c
    scales[at[used] // page, :, at[used] % page] = s.to(scales.dtype)
    return codes, scales


def cache(P, H, page, d, g, spread=6):
    """Random codes and bf16 scales that differ by 2^spread and are no powers of two."""
    codes = torch.randint(0, 256, (P, H, page, d // 2), generator=g, dtype=torch.uint8)
    s = torch.exp2(spread * torch.rand((P, H, page, d // 32), generator=g) - spread - 1)
    return codes, s.bfloat16()


def rows(val, table, lens, cu, out):
    """out [T, H, d] (float64) with the cached tokens of every request in its rows.
    val [P, H, page, d]: what the cache stands for; pages outside are zeros."""
    P, H, page, d = val.shape
    out = out.clone()
    for b, n in enumerate(lens):
        for i in range(min(max(n, 0), table.shape[1] * page)):
            r, pg = cu[b] + i, int(table[b, i // page])
            if r >= min(cu[b + 1], out.shape[0]):
                break
            out[r] = val[pg, :, i % page] if 0 <= pg < P else 0.0
    return out


def to16(x, dtype):
    """Float64 to the 16-bit type, nearest even, at most the type's largest.  (Products of code
    and scale have 11 bits at most: 32 bits hold them, and are rounded once.)"""
    top = torch.finfo(plain64.DT[dtype]).max
    return x.clamp(-top, top).float().to(plain64.DT[dtype])


def decoded(q, kval, vc, vs, table, lens, scale, causal, dtype):
    """Reference and bounds of attention over the paged cache: (o, bound), (lse, bound).
    kval [P, H, page, d]: keys; vc, vs: the values' codes (as numbers) and scales [P, H, page, d / 32].

    P times a value's scale is carried by two (bf16) or three (fp16) e4m3 terms: off by 2^-9 or
    2^-14 of itself, for bf16 by another 2^-11 (its rounding to fp16 before the second term), and by
    2^-21 or 2^-25 of the largest p u s_g of its tile where it falls among the subnormal codes (half of
    their step is 2^-22 or 2^-26 of the largest product, whose scales are measured by a power of two up to
    twice the largest s_g); u is the largest of a token's scales, each against the largest s_g of its group
    of channels in the tile.
    Tiles hold 128 tokens (d = 128) or 256 (d = 64).  The scores see the query within 2^-21 of its
    row's largest element."""
    u, tiny = plain64.U[dtype], plain64.TINY[dtype]
    up, floor = (2.0 ** -9 + 2.0 ** -11, 2.0 ** -21) if dtype == "bf16" else (2.0 ** -14, 2.0 ** -25)
    B, Nq, Hq, d = q.shape
    P, H, page, _ = kval.shape
    G, tile = Hq // H, 128 * 128 // d
    o = torch.zeros(q.shape, dtype=torch.float64)
    ob = torch.zeros_like(o)
    lse = torch.full((B, Hq, Nq), -math.inf, dtype=torch.float64)
    lb = torch.ones_like(lse)
    for b in range(B):
        n = lens[b]
        pg = table[b, :-(-n // page)].long()
        last = n - Nq + torch.arange(Nq) if causal else torch.full((Nq,), n)
        for h in range(H):
            k, c = (x[pg, h].reshape(-1, d)[:n] for x in (kval, vc))
            s = vs[pg, h].double().reshape(-1, d // 32)[:n]
            v = c * s.repeat_interleave(32, 1)
            for hq in range(h * G, (h + 1) * G):
                qh = q[b, :, hq]
                oh, l, p, es = plain64.attend(qh, k, v, scale, last)
                if n:
                    es = es + 2 * 2.0 ** -21 * scale * qh.abs().amax(1) * k.abs().sum(1).amax()
                    st = torch.nn.functional.pad(s, (0, 0, 0, -n % tile)).view(-1, tile, d // 32)
                    top = st.amax(1)                                                 # [tiles, groups]
                    ut = (st / top.clamp_min(1e-300)[:, None]).amax(2)               # [tiles, tile]
                    w = (torch.nn.functional.pad(p, (0, -n % tile)).view(Nq, -1, tile) * ut).amax(2)
                    mag = torch.nn.functional.pad(c.abs(), (0, 0, 0, -n % tile)).view(-1, tile, d).sum(1)
                    ob[b, :, hq] = (u * oh.abs() + (p @ v.abs()) * (up + es[:, None]) +
                                    floor * (w @ (mag * top.repeat_interleave(32, 1))) + tiny)
                o[b, :, hq], lse[b, hq] = oh, l
                lb[b, hq] = es + 2.0 ** -20 * (1 + torch.where(l == -math.inf, 0.0, l.abs()))
    return (o, ob), (lse, lb)
