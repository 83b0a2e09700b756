"""Packed and cached attention written out in 64 bits, with element-wise error
bounds derived from the roundings the kernels make.

u is half a step of the 16-bit type relative to the value (bf16 2^-8, fp16
2^-11).  The kernels round P and dS once to a type with error `up` per value
before a product, accumulate in fp32, and round the result once:

  |dO|  <= u |O| + sum_j p_j |v_j| (up + es)
  |dLSE| <= es + 2^-20 (1 + |LSE|)
  es     = 2 * 2^-18 * s sum_c |q_c| |k_c|  (fp32 products and exponentials: the
           score's error, doubled for P = exp(S - LSE), where LSE has it too)
           + 2^-17 (the approximate exponential and logarithm)
  |ddS| <= |dS| (u + es) + P (u sum_c |dO_c O_c| + 2^-17 sum_c |dO_c| (|V_c| + |O_c|))
  |ddQ| <= u |dQ| + s sum_j |ddS_ij| |K_j|,  dK alike with Q, summed over the group
  |ddV| <= u |dV| + sum_i P_ij |dO_i| (u + es)
and a value below the type's normal range has an absolute step: `tiny`.
"""
import math

import torch

U = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11}
TINY = {"bf16": 1e-30, "fp16": 2.0 ** -24}
DT = {"bf16": torch.bfloat16, "fp16": torch.float16}


def attend(q, k, v, scale, last, do=None):
    """One head: q [n, d], k, v [m, d] in float64, row i sees keys j <= last[i].
    Returns o, lse, p, es [n] and, with do, what the gradients need."""
    m = k.shape[0]
    x = scale * (q @ k.T)
    hide = torch.arange(m)[None, :] > last[:, None]
    x = x.masked_fill(hide, -math.inf)
    lse = torch.logsumexp(x, 1) if m else torch.full((q.shape[0],), -math.inf, dtype=torch.float64)
    p = torch.exp(x - torch.where(lse == -math.inf, 0.0, lse)[:, None])
    p = p.masked_fill(hide, 0.0)
    size = (q.abs() @ k.abs().T).masked_fill(hide, 0.0)
    es = 2 * 2.0 ** -18 * scale * (size.amax(1) if m else torch.zeros(q.shape[0], dtype=torch.float64))
    es = es + 2.0 ** -17
    vz = torch.where(torch.isfinite(v), v, 0.0)
    return p @ vz, lse, p, es


def packed(q, k, v, cu_q, cu_k, scale, causal, dtype, do=None):
    """Reference and bounds of packed attention (float64 [T, H, d] inputs):
    {name: (value, bound)} for o, lse and, with do, dq, dk, dv.  Rows of no
    sequence have value NaN."""
    u, tiny = U[dtype], TINY[dtype]
    Tq, Hq, d = q.shape
    Tk, H, _ = k.shape
    G = Hq // H
    nan = lambda *s: torch.full(s, math.nan, dtype=torch.float64)  # noqa: E731
    r = {n: [nan(*s), torch.zeros(s, dtype=torch.float64)] for n, s in
         dict(o=(Tq, Hq, d), lse=(Hq, Tq), dq=(Tq, Hq, d), dk=(Tk, H, d), dv=(Tk, H, d)).items()}
    for b in range(len(cu_q) - 1):
        rows, keys = slice(cu_q[b], cu_q[b + 1]), slice(cu_k[b], cu_k[b + 1])
        lq, lk = cu_q[b + 1] - cu_q[b], cu_k[b + 1] - cu_k[b]
        last = torch.arange(lq) + (lk - lq) if causal else torch.full((lq,), lk)
        for n in ("dk", "dv"):
            r[n][0][keys] = 0.0
        for h in range(Hq):
            qh, kh, vh = q[rows, h], k[keys, h // G], v[keys, h // G]
            o, lse, p, es = attend(qh, kh, vh, scale, last)
            r["o"][0][rows, h] = o
            r["o"][1][rows, h] = u * o.abs() + (p @ vh.abs()) * (u + es[:, None]) + tiny
            r["lse"][0][h, rows] = lse
            r["lse"][1][h, rows] = es + 2.0 ** -20 * (1 + torch.where(lse == -math.inf, 0.0, lse.abs()))
            if do is None:
                continue
            g = do[rows, h]
            dp = g @ vh.T
            ds = p * (dp - (g * o).sum(1, keepdim=True))
            e_row = u * (g * o).abs().sum(1) + 2.0 ** -17 * (g.abs() * o.abs()).sum(1)
            dds = ds.abs() * (u + es[:, None]) + p * (e_row[:, None] + 2.0 ** -17 * (g.abs() @ vh.abs().T)) + tiny
            dq = scale * (ds @ kh)
            r["dq"][0][rows, h] = dq
            r["dq"][1][rows, h] = u * dq.abs() + scale * (dds @ kh.abs()) + tiny
            r["dk"][0][keys, h // G] += scale * (ds.T @ qh)
            r["dk"][1][keys, h // G] += scale * (dds.T @ qh.abs()) + tiny
            r["dv"][0][keys, h // G] += p.T @ g
            r["dv"][1][keys, h // G] += (p * (u + es[:, None])).T @ g.abs() + tiny
    for n in ("dk", "dv"):
        r[n][1] += u * torch.nan_to_num(r[n][0]).abs()
    return {n: tuple(x) for n, x in r.items() if do is not None or n in ("o", "lse")}


def check(got, value, bound, what):
    """got (any type) against value within bound, element by element; NaN in
    `value` means the element is not looked at."""
    got = got.double().cpu()
    look = ~torch.isnan(value)
    inf = look & torch.isinf(value)
    assert torch.equal(got[inf], value[inf]), f"{what}: infinities differ"
    look &= ~inf
    off = (got[look] - value[look]).abs()
    assert torch.isfinite(off).all(), f"{what}: not finite"
    over = off / bound[look].clamp_min(1e-300)
    if over.numel():
        worst = over.max().item()
        assert worst <= 1.0, f"{what}: {worst:.3f} times the bound"


# ------------------------------------------------------------------ e4m3 pages
def e4m3(y):
    """Nearest e4m3 value (float64 in and out), ties to even, saturating."""
    y = y.clamp(-448.0, 448.0)
    e = (torch.frexp(y.abs().clamp_min(2.0 ** -6))[1] - 1).double()
    return torch.round(y * torch.exp2(3 - e)) * torch.exp2(e - 3)


def page_scale(top):
    """Smallest power of two s with top <= 448 s, within [2^-64, 2^60]."""
    m, e = torch.frexp(top / 448.0)
    e = torch.where(top == 0, -64, torch.where(m == 0.5, e - 1, e))
    return torch.exp2(e.clamp(-64, 60).double())


def append(x, slots, val, scale):
    """The new code values [P, H, page, d] and scales [P, H] in float64 after the
    tokens x [T, H, d] go to `slots`."""
    val, scale = val.clone(), scale.clone()
    P, H, page, d = val.shape
    t = 0
    while t < len(slots):
        n = 1
        if not 0 <= slots[t] < P * page:
            t += 1
            continue
        while t + n < len(slots) and slots[t + n] == slots[t] + n and slots[t + n] % page:
            n += 1
        pg, first = slots[t] // page, slots[t] % page
        run = x[t:t + n].transpose(0, 1)  # [H, n, d]
        mag = torch.where(torch.isnan(run), 0.0, run.abs()).clamp_max(448.0 * 2.0 ** 60)
        new = page_scale(mag.amax((1, 2)))
        if first:
            new = torch.maximum(new, scale[pg])
            val[pg, :, :first] = e4m3(val[pg, :, :first] * (scale[pg] / new)[:, None, None])
        val[pg, :, first:first + n] = e4m3(run / new[:, None, None])
        scale[pg] = new
        t += n
    return val, scale


def cached(q, kval, vval, ks, vs, table, lens, scale, causal, dtype):
    """Reference and bounds of attention over the paged cache: (o, bound), (lse,
    bound).  P is carried by two (bf16) or three (fp16) e4m3 terms: off by 2^-9
    or 2^-14 of its value, and by 2^-22 or 2^-26 of the largest p vs of its
    128-key tile where it falls among the subnormal codes.  The scores see the
    query within 2^-21 of its row's largest element."""
    u, tiny = U[dtype], TINY[dtype]
    up, floor = (2.0 ** -9, 2.0 ** -22) if dtype == "bf16" else (2.0 ** -14, 2.0 ** -26)
    B, Nq, Hq, d = q.shape
    H = kval.shape[1]
    G = Hq // H
    o = torch.zeros(q.shape, dtype=torch.float64)
    ob = torch.zeros_like(o)
    lse = torch.full((B, Hq, Nq), -math.inf, dtype=torch.float64)
    lb = torch.ones_like(lse)
    page = kval.shape[2]
    for b in range(B):
        n = lens[b]
        pg = table[b, :-(-n // page)].long()
        last = n - Nq + torch.arange(Nq) if causal else torch.full((Nq,), n)
        for h in range(H):
            k, vc = (c[pg, h].reshape(-1, d)[:n] for c in (kval, vval))
            k = k * ks[pg, h].repeat_interleave(page)[:n, None]
            vsc = vs[pg, h].repeat_interleave(page)[:n]
            v = vc * vsc[:, None]
            for hq in range(h * G, (h + 1) * G):
                qh = q[b, :, hq]
                oh, l, p, es = attend(qh, k, v, scale, last)
                if n:
                    # the query terms: 2^-21 of the row's largest times the keys
                    eq = 2 * 2.0 ** -21 * scale * qh.abs().amax(1) * k.abs().sum(1).amax()
                    es = es + eq
                    w = torch.nn.functional.pad(p * vsc, (0, -n % 128)).view(Nq, -1, 128).amax(2)
                    mag = torch.nn.functional.pad(vc.abs(), (0, 0, 0, -n % 128)).view(-1, 128, d).sum(1)
                    ob[b, :, hq] = (u * oh.abs() + (p @ v.abs()) * (up + es[:, None]) + floor * (w @ mag) + tiny)
                o[b, :, hq], lse[b, hq] = oh, l
                lb[b, hq] = es + 2.0 ** -20 * (1 + torch.where(l == -math.inf, 0.0, l.abs()))
    return (o, ob), (lse, lb)
