"""attn_kv4_decode within derived bounds of attention over what the 4-bit cache stands for
(plain4.py), and together with append, read, the block tables and the packed prompt."""
import math

import pytest
import torch

import plain4
import plain64
from plain64 import DT

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from exact_tiled_attention_22_gb300 import build
    build.build()
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    from exact_tiled_attention_22_gb300 import attn
    attn.attn_set_wait_limit(0, 0)
    yield
    assert attn.attn_status() == 0


def i32(x):
    return torch.tensor(x, dtype=torch.int32).cuda()


def problem(lens, Nq, Hq, H, d, page, dtype, seed, spread=6):
    """A cache with pages in no order, NaN scales in every place that must not be looked at, and table
    entries outside the cache behind the last page."""
    g = torch.Generator().manual_seed(seed)
    B = len(lens)
    need = [-(-n // page) for n in lens]
    P = sum(need) + 2
    kc, ks = plain4.cache(P, H, page, d, g, spread)
    vc, vs = plain4.cache(P, H, page, d, g, spread)
    ids = torch.randperm(P, generator=g)
    width = max(need) + 2
    table = torch.full((B, width), 2 ** 30, dtype=torch.int32)
    table[:, -1] = -9
    used, at = torch.zeros(P, page, dtype=torch.bool), 0
    for b, n in enumerate(lens):
        for j in range(need[b]):
            table[b, j] = ids[at]
            used[ids[at], :min(page, n - j * page)] = True
            at += 1
    for s in (ks, vs):
        s[~used[:, None, :].expand(P, H, page)] = math.nan
    q = torch.randn((B, Nq, Hq, d), generator=g).to(DT[dtype])
    return q, kc, vc, ks, vs, table


def reference(args, lens, scale, causal, dtype):
    q, kc, vc, ks, vs, table = args
    ones = torch.ones_like(vs)
    return plain4.decoded(q.double(), plain4.values(kc, ks), plain4.values(vc, ones), vs, table, lens, scale, causal, dtype)


def wide(table):
    """The same block table with room for 70000 tokens a request: the tiles of all requests are dealt to all
    blocks then, where a narrow table lets a cluster of blocks take a request's."""
    room = torch.full((table.shape[0], 70000 // 16), 2 ** 30, dtype=torch.int32, device=table.device)
    return torch.cat([table, room], 1)


def decode_and_check(args, lens, scale, causal, dtype):
    """Through clusters, if the table is narrow enough, and through dealt tiles."""
    from exact_tiled_attention_22_gb300 import attn
    (ro, bo), (rl, bl) = reference(args, lens, scale, causal, dtype)
    for table in (wide(args[-1]), args[-1]):
        o, lse = attn.kv4_decode(*(x.cuda() for x in (*args[:-1], table)), i32(lens), scale, causal)
        attn.check(attn.attn_status())
        plain64.check(lse, rl, bl, "lse")
        plain64.check(o, ro, bo, "o")
    return o, lse


DECODE = [
    # (lens, Nq, Hq, Hkv, d, page, dtype, causal)
    ([1], 1, 1, 1, 64, 16, "fp16", True),
    ([1], 1, 1, 1, 128, 128, "bf16", True),
    ([2], 1, 1, 1, 64, 16, "bf16", True),
    ([0, 5, 0], 1, 4, 2, 64, 16, "bf16", True),
    ([0], 1, 4, 2, 128, 32, "fp16", False),
    ([127, 128, 129, 16, 17], 1, 8, 2, 128, 16, "bf16", True),
    ([255, 256, 257, 16, 17, 511], 1, 8, 2, 64, 16, "fp16", True),
    ([1000, 3, 2049], 1, 32, 8, 128, 64, "bf16", True),
    ([1000, 3, 2049], 1, 32, 4, 64, 128, "bf16", True),
    ([700, 64, 65], 1, 7, 1, 64, 32, "fp16", True),
    ([700, 64, 65], 1, 7, 1, 128, 32, "fp16", True),
    ([3000], 1, 16, 1, 128, 128, "fp16", True),
    ([3000, 130], 1, 16, 1, 128, 128, "bf16", True),
    ([3001, 20], 1, 16, 1, 64, 64, "bf16", True),
    ([5, 2, 300], 5, 14, 2, 64, 16, "fp16", True),       # requests shorter than the draft
    ([5, 2, 300], 5, 14, 2, 64, 16, "bf16", True),
    ([5, 2, 300, 0], 3, 6, 2, 128, 32, "bf16", False),
    ([400, 130], 8, 40, 5, 64, 64, "bf16", True),        # four row blocks
    ([260], 128, 2, 2, 128, 64, "bf16", True),
    ([260], 127, 1, 1, 64, 64, "fp16", True),
    ([33] * 400, 1, 2, 1, 64, 16, "fp16", True),         # more requests than threads
    ([20000, 1, 64], 1, 8, 1, 128, 64, "bf16", True),    # split over many blocks
    ([20001, 1, 64], 1, 4, 1, 64, 64, "fp16", True),
    ([0, 900, 0, 1, 257], 1, 8, 2, 128, 16, "bf16", True),    # empty requests among others' clusters
    ([2000], 1, 4, 1, 128, 16, "bf16", True),                 # a cluster of 16, one tile each
    ([10000], 1, 32, 8, 128, 64, "bf16", True),               # ... five each
    ([16001], 1, 8, 2, 64, 64, "fp16", True),
    ([3000, 2999, 5], 2, 32, 8, 128, 128, "bf16", True),
    ([1300] * 12, 1, 32, 8, 128, 64, "bf16", True),           # clusters of four, three tiles each
    ([400] * 20, 1, 64, 8, 64, 32, "bf16", True),
    ([511, 77] * 8, 1, 16, 1, 128, 16, "bf16", True),
]


@pytest.mark.parametrize("case", DECODE, ids=lambda c: f"B{len(c[0])}q{c[1]}h{c[2]}x{c[3]}d{c[4]}p{c[5]}{c[6]}")
def test_decode(case):
    lens, Nq, Hq, H, d, page, dtype, causal = case
    args = problem(lens, Nq, Hq, H, d, page, dtype, seed=sum(lens) + d)
    decode_and_check(args, lens, d ** -0.5, causal, dtype)


@pytest.mark.parametrize("d,dtype", [(128, "bf16"), (64, "bf16"), (64, "fp16")])
def test_decode_scales_far_apart(d, dtype):
    """Scales of tokens and groups of channels that differ by 2^40 or are zero; values whose channels differ by 2^20
    from group to group keep their own precision."""
    lens = [300, 513]
    args = problem(lens, 1, 8, 2, d, 32, dtype, seed=1, spread=40)
    args[3].copy_(args[3] * 0 + 0.01)                       # (keys of one size: many tokens have weight)
    g = torch.Generator().manual_seed(2)
    args[4][torch.rand(args[4].shape, generator=g) < 0.1] = 0.0
    decode_and_check(args, lens, 0.1, True, dtype)
    args = problem(lens, 1, 8, 2, d, 32, dtype, seed=3)
    args[4][..., 0] *= 2.0 ** -20
    o, _ = decode_and_check(args, lens, 0.02, True, dtype)
    if dtype == "bf16":  # the small channels alone: within 2^-6 of their own size
        (ro, _), _ = reference(args, lens, 0.02, True, dtype)
        small, want = o[..., :32].double().cpu(), ro[..., :32]
        assert ((small - want).abs().amax() <= 2.0 ** -6 * want.abs().amax()).item()


def test_decode_sharp_scores_and_wide_queries():
    """Scores in the hundreds (the running maximum moves) and queries whose elements span 2^-20 .. 2^4."""
    lens = [900]
    args = list(problem(lens, 2, 8, 1, 64, 16, "bf16", seed=8))
    args[3] = args[3] * 64
    decode_and_check(args, lens, 1.0, True, "bf16")
    g = torch.Generator().manual_seed(9)
    args[0] = (torch.randn(args[0].shape, generator=g) *
               torch.exp2(torch.randint(-20, 5, args[0].shape, generator=g).float())).bfloat16()
    decode_and_check(args, lens, 0.01, True, "bf16")


@pytest.mark.parametrize("size", [1e25, 1e-25])
def test_decode_scores_of_any_size(size):
    """Scores of 1e32 and more, of either sign (one key takes all, even where all are far below zero), and next to
    none (a mean)."""
    lens = [300, 1]
    args = list(problem(lens, 1, 4, 1, 64, 16, "bf16", seed=20, spread=1))
    args[0] = (args[0].float() * size).bfloat16()
    args[3] = args[3] * 1e7
    from exact_tiled_attention_22_gb300 import attn
    for q in (args[0], -args[0]):
        (ro, bo), (rl, bl) = reference([q, *args[1:]], lens, 1.0, True, "bf16")
        for t in (args[-1], wide(args[-1])):
            o, lse = attn.kv4_decode(*(x.cuda() for x in (q, *args[1:-1], t)), i32(lens), 1.0)
            if size > 1:  # (the score's own rounding decides between keys whose scores are close: the others' are not)
                far = (o.double().cpu() - ro).abs() <= 2.0 ** -8 * ro.abs() + 1e-3
                assert torch.isfinite(o).all() and far.all()
                assert ((lse.double().cpu() - rl).abs() <= 2.0 ** -16 * rl.abs()).all()
            else:
                plain64.check(lse, rl, bl, "lse")
                plain64.check(o, ro, bo, "o")


def test_decode_a_heavy_token_of_small_value():
    """A first token that takes nearly all the weight and whose value is next to nothing: the others' part stays exact."""
    lens = [200]
    for d in (64, 128):
        args = list(problem(lens, 1, 4, 1, d, 16, "bf16", seed=10))
        q, kc, vc, ks, vs, table = args
        ks.fill_(0.002)
        q.fill_(0.25)
        first = table[0, 0].item()
        kc[first, 0, 0], ks[first, 0, 0] = 0x77, 1.0 * 128 / d       # all sixes: a score of 16 more
        vs[first, 0, 0] = 2.0 ** -30
        decode_and_check(args, lens, 128.0 / d * 0.08, True, "bf16")


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("heavy,large", [(0, 7), (1, 6), (0, 6), (1, 7)])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_decode_small_values_between_a_heavy_token_and_a_large_value(d, heavy, large, dtype):
    """A token with nearly all the weight whose value is zero in half of the channels, one without weight but with a
    scale 700 times the others', on even and odd places: the other tokens' values keep their precision in those
    channels."""
    lens = [8]
    q, kc, vc, ks, vs, table = problem(lens, 1, 4, 1, d, 16, dtype, seed=21)
    page = table[0, 0].item()
    q.fill_(0.25)
    kc[page, 0, :8] = 0x22                                       # ones
    ks[page, 0, :8] = 0.01
    ks[page, 0, heavy] = 0.01 + 6.0 * 4 / d
    ks[page, 0, large] = -9.0 * 4 / d
    vc[page, 0, :8] = 0x55                                       # threes
    vs[page, 0, :8] = 2.0 ** -11
    vs[page, 0, heavy] = 2.0 ** -8
    vs[page, 0, large] = 0.35
    vc[page, 0, heavy, d // 4:] = 0
    vc[page, 0, large, d // 4:] = 0
    decode_and_check((q, kc, vc, ks, vs, table), lens, 1.0, True, dtype)


def test_decode_not_numbers_stay_where_they_are():
    """A NaN in a query or in a cached token reaches the heads that see it, no other."""
    from exact_tiled_attention_22_gb300 import attn
    lens = [200, 200]
    q, kc, vc, ks, vs, table = problem(lens, 2, 4, 2, 64, 16, "fp16", seed=12)
    tables = (table, wide(table))
    clean = [attn.kv4_decode(*(x.cuda() for x in (q, kc, vc, ks, vs, t)), i32(lens))[0] for t in tables]
    q[0, 1, 3] = math.inf
    ks[table[1, 0], 1, 3, 1] = math.nan     # key head 1 of request 1
    vs[table[1, 12], 0, 7, 0] = math.nan    # its last token's value, head 0, channels 0 to 31
    for t, c in zip(tables, clean):
        o, _ = attn.kv4_decode(*(x.cuda() for x in (q, kc, vc, ks, vs, t)), i32(lens))
        nan = torch.isnan(o)
        want = torch.zeros_like(nan)
        want[0, 1, 3] = True
        want[1, :, 2:] = True
        want[1, :, :2, :32] = True          # (a hidden NaN times a zero is one, too)
        assert torch.equal(nan, want)
        assert torch.equal(o[~want], c[~want])


def test_far_into_a_large_cache():
    """Pages whose byte offsets pass 2^32, written by append, decoded and read."""
    from exact_tiled_attention_22_gb300 import attn
    H, d, page = 8, 128, 128
    P = (1 << 32) // (H * d // 2 * page) + 40
    kc = torch.zeros((P, H, page, d // 2), dtype=torch.uint8, device="cuda")
    vc = torch.zeros_like(kc)
    ks, vs = (torch.zeros((P, H, page, d // 32), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    g = torch.Generator().manual_seed(3)
    n = 300
    ids = torch.tensor([P - 1, 5, P - 30])
    pos = torch.arange(n)
    slots = ids[pos // page] * page + pos % page
    k, v = (torch.randn((n, H, d), generator=g).bfloat16() for _ in range(2))
    attn.kv4_append(k.cuda(), v.cuda(), slots.cuda(), kc, vc, ks, vs)
    q = torch.randn((1, 1, H, d), generator=g).bfloat16()
    table = ids.int()[None]
    o, lse = attn.kv4_decode(q.cuda(), kc, vc, ks, vs, table.cuda(), i32([n]))
    few = [x[ids.cuda()].cpu() for x in (kc, vc, ks, vs)]
    args = (q, *few, torch.tensor([[0, 1, 2]]))
    for x, c, s in ((k, few[0], few[2]), (v, few[1], few[3])):
        wc, ws = plain4.quantise(x.double())
        assert torch.equal(c.transpose(1, 2).reshape(-1, H, d // 2)[:n], wc)
        assert torch.equal(s.transpose(1, 2).reshape(-1, H, d // 32)[:n].double(), ws)
    (ro, bo), (rl, bl) = reference(args, [n], d ** -0.5, True, "bf16")
    plain64.check(o, ro, bo, "o")
    plain64.check(lse, rl, bl, "lse")
    rk, rv = attn.kv4_read(kc, vc, ks, vs, table.cuda(), i32([n]), i32([0, n]), n)
    for x, c, s in ((rk, few[0], few[2]), (rv, few[1], few[3])):
        want = plain4.to16(plain4.values(c, s).transpose(1, 2).reshape(-1, H, d)[:n], "bf16")
        assert torch.equal(x.cpu().view(torch.int16), want.view(torch.int16))


@pytest.mark.parametrize("narrow", [False, True])
def test_two_calls_at_once_and_repeats(narrow):
    """Two streams with their own workspaces; equal results every time."""
    from exact_tiled_attention_22_gb300 import attn
    lens = [900, 17, 700] if narrow else [5000, 17, 900]
    args = [x.cuda() for x in problem(lens, 1, 16, 4, 128, 64, "bf16", seed=4)]
    ln = i32(lens)
    want = attn.kv4_decode(*args, ln)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for _ in range(5):
        for s in streams:
            with torch.cuda.stream(s):
                got.append(attn.kv4_decode(*args, ln))
    got.append(attn.kv4_decode(*args, ln, stream=streams[0]))
    torch.cuda.synchronize()
    for o, lse in got:
        assert torch.equal(o, want[0]) and torch.equal(lse, want[1])


def test_pages_that_are_not_there_read_as_zeros():
    """Page ids outside the cache within a request's length: zero keys and values (the scales of page 0 may be
    anything)."""
    from exact_tiled_attention_22_gb300 import attn
    for d in (64, 128):
        lens = [150]
        q, kc, vc, ks, vs, table = problem(lens, 1, 4, 2, d, 16, "bf16", seed=14)
        gone = [1, 4, 7]
        z = [x.clone() for x in (kc, vc, ks, vs)]
        for x in z:
            x[table[0, gone].long()] = 0
        (ro, bo), (rl, bl) = reference((q, *z, table), lens, 0.125, True, "bf16")
        spare = [p for p in range(kc.shape[0]) if p not in table[0].tolist()][0]
        bad = table.clone()
        keep = bad[0] == 0
        if keep.any():  # (page 0 is in use: its contents move to a spare page)
            for c in (kc, vc, ks, vs):
                c[spare] = c[0].clone()
            bad[0][keep] = spare
        ks[0], vs[0] = math.nan, math.nan
        for j, i in zip(gone, (-1, kc.shape[0], 2 ** 31 - 1)):
            bad[0, j] = i
        for t in (bad, wide(bad)):
            o, lse = attn.kv4_decode(q.cuda(), kc.cuda(), vc.cuda(), ks.cuda(), vs.cuda(), t.cuda(), i32(lens), 0.125)
            plain64.check(lse, rl, bl, "lse")
            plain64.check(o, ro, bo, "o")


def test_errors_of_decode():
    """What the tensors cannot be raises ValueError, what the library refuses AttnError with its code; nothing is
    enqueued and the next call works."""
    from exact_tiled_attention_22_gb300 import attn
    lens = [20, 40]
    q, kc, vc, ks, vs, table = (x.cuda() for x in problem(lens, 1, 4, 2, 64, 16, "fp16", seed=16))
    ln = i32(lens)
    want = attn.kv4_decode(q, kc, vc, ks, vs, table, ln)
    for bad in (dict(q=q.float()), dict(q=q[0]), dict(q=q.transpose(0, 1)), dict(q=q.cpu()), dict(kc=kc.float()),
                dict(vc=vc[:-1]), dict(ks=ks.half()), dict(table=table.long()), dict(table=table[:1]),
                dict(ln=ln.cpu()), dict(ln=[20, 40]), dict(ws=torch.zeros(8))):
        a = dict(q=q, kc=kc, vc=vc, ks=ks, vs=vs, table=table, ln=ln, ws=None)
        a.update(bad)
        with pytest.raises(ValueError):
            attn.kv4_decode(a["q"], a["kc"], a["vc"], a["ks"], a["vs"], a["table"], a["ln"], ws=a["ws"])
    for bad, code in ((dict(q=q[:, :, :3].contiguous()), attn.ATTN_ERR_INVALID), (dict(scale=-1.0), attn.ATTN_ERR_INVALID),
                      (dict(ws=torch.zeros(1024, device="cuda")), attn.ATTN_ERR_WORKSPACE)):
        with pytest.raises(attn.AttnError) as e:
            attn.kv4_decode(bad.get("q", q), kc, vc, ks, vs, table, ln, bad.get("scale"), ws=bad.get("ws"))
        assert e.value.code == code and str(e.value)
    got = attn.kv4_decode(q, kc, vc, ks, vs, table, ln)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("lens", [[127, 128, 129, 16, 17], [1, 1, 1], [3000, 5], [128] * 40])
def test_what_the_workspace_held_does_not_matter(lens):
    """A workspace full of NaN: only parts that this call wrote are read, also when there are fewer tiles than blocks."""
    from exact_tiled_attention_22_gb300 import attn
    args = [x.cuda() for x in problem(lens, 1, 8, 2, 128, 16, "bf16", seed=4)]
    args[-1] = wide(args[-1])
    ln = i32(lens)
    n = attn.attn_kv4_decode_workspace_size(1, 8, 2, 128)
    clean = torch.zeros(n, dtype=torch.uint8, device="cuda")
    dirty = torch.full((n // 4,), math.nan, device="cuda").view(torch.uint8)
    a, b = attn.kv4_decode(*args, ln, ws=clean), attn.kv4_decode(*args, ln, ws=dirty)
    assert torch.isfinite(a[0]).all() and torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("n", [64, 1600, 40000])
def test_lengths_beyond_the_table_and_negative_ones(n):
    from exact_tiled_attention_22_gb300 import attn
    lens = [n, n, n]
    q, kc, vc, ks, vs, table = problem(lens, 1, 4, 2, 64, 16, "bf16", seed=5)
    short = table[:, :n // 16].contiguous()
    table = torch.cat([short, short[:, :1]], 1)
    args = [x.cuda() for x in (q, kc, vc, ks, vs)]
    want = attn.kv4_decode(*args, table.cuda(), i32([n, 0, n]), 0.1)
    got = attn.kv4_decode(*args, short.cuda(), i32([2 ** 31 - 1, -5, n]), 0.1)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert (got[0][1] == 0).all() and (got[1][1] == -math.inf).all()


def test_more_rows_than_blocks_of_the_merge():
    """So many requests that a block of the merge takes several rows of several of them, empty ones and ones that
    several blocks of the split share among them."""
    g = torch.Generator().manual_seed(17)
    lens = torch.randint(0, 4, (1000,), generator=g)
    lens[torch.tensor([0, 1, 399, 700, 999])] = torch.tensor([1500, 0, 3000, 257, 0], dtype=lens.dtype)
    lens = lens.tolist()
    for d in (64, 128):
        decode_and_check(problem(lens, 1, 5, 5, d, 16, "bf16", seed=18), lens, 0.125, True, "bf16")


def test_tensors_freed_after_a_call_on_another_stream():
    """The memory of a query that is dropped after the call is not handed on while the call still waits for its
    stream."""
    from exact_tiled_attention_22_gb300 import attn
    lens = [300] * 64
    q, kc, vc, ks, vs, table = (x.cuda() for x in problem(lens, 1, 32, 4, 128, 32, "bf16", seed=19))
    ln = i32(lens)
    want = attn.kv4_decode(q, kc, vc, ks, vs, table, ln)
    side = torch.cuda.Stream()
    big = torch.randn(8192, 8192, device="cuda")
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        for _ in range(4):
            big @ big                       # the call waits behind these
    mine = q.clone()
    torch.cuda.current_stream().synchronize()
    o, lse = attn.kv4_decode(mine, kc, vc, ks, vs, table, ln, stream=side)
    del mine
    others = [torch.full_like(q, math.nan) for _ in range(8)]
    torch.cuda.synchronize()
    assert torch.equal(o, want[0]) and torch.equal(lse, want[1])
    del others


@pytest.mark.parametrize("narrow", [False, True])
@pytest.mark.parametrize("Hq", [2, 8, 16])
def test_wait_limit_reports_a_timeout(narrow, Hq):
    from exact_tiled_attention_22_gb300 import attn
    lens = [300, 0, 700]
    args = [x.cuda() for x in problem(lens, 1, Hq, 1, 64, 16, "bf16", seed=6)]
    args[-1] = args[-1] if narrow else wide(args[-1])
    ln = i32(lens)
    want = attn.kv4_decode(*args, ln)
    try:
        attn.attn_set_wait_limit(50_000_000, 16)
        attn.kv4_decode(*args, ln)
        assert attn.attn_status() == attn.ATTN_ERR_TIMEOUT
    finally:
        attn.attn_set_wait_limit(0, 0)
    got = attn.kv4_decode(*args, ln)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


# ------------------------------------------------------------------ together
@pytest.mark.parametrize("width", [12, 70])
def test_a_serving_run(width):
    """Prompts are attended to as a packed batch and written to the cache; one goes on with a second turn, whose
    queries attend to the cached prefix read back in front of the new keys; then all are decoded token by token from a
    captured step; requests leave and their pages are used again.  Every step against 64 bits over the cache as the
    definition fills it.  (Tables of 70 pages: five tiles a request, clusters.)"""
    from exact_tiled_attention_22_gb300 import attn
    B, Hq, H, d, page = 4, 8, 2, 64, 16
    g = torch.Generator().manual_seed(42)
    P = 40
    kc = torch.full((P, H, page, d // 2), 0xFF, dtype=torch.uint8, device="cuda")  # nothing written yet
    vc = kc.clone()
    ks, vs = (torch.full((P, H, page, d // 32), math.nan, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    table, stack, count = i32([[-1] * width] * B), i32(torch.randperm(P, generator=g).tolist()), i32([P])
    lens = i32([0] * B)
    mine = [x.cpu() for x in (kc, vc, ks, vs)]
    scale = d ** -0.5

    def remember(k, v, slots):
        for i, x in enumerate((k, v)):
            mine[i], mine[2 + i] = plain4.append(x.double().cpu(), slots.tolist(), mine[i], mine[2 + i])

    def turn(new):
        """`new` tokens of each request: pages, attention to prefix and new tokens, and into the cache."""
        T, before = sum(new), lens.tolist()
        q, k, v = (torch.randn((T, h, d), generator=g).half().cuda() for h in (Hq, H, H))
        ends = [a + b for a, b in zip(before, new)]
        cu_k = [0]
        for n in ends:
            cu_k.append(cu_k[-1] + n)
        kk, vv = (torch.empty((cu_k[-1], H, d), dtype=torch.float16, device="cuda") for _ in range(2))
        attn.kv4_read(kc, vc, ks, vs, table, lens, i32(cu_k), cu_k[-1], torch.float16, kk, vv)
        at = 0
        for b, n in enumerate(new):
            kk[cu_k[b] + before[b]:cu_k[b + 1]], vv[cu_k[b] + before[b]:cu_k[b + 1]] = k[at:at + n], v[at:at + n]
            at += n
        _, _, cu, slots, _ = attn.pages_extend(lens, i32(new), table, stack, count, page, T, new_lens=lens,
                                               free_left=count)
        o, _ = attn.varlen_fwd(q, kk, vv, cu, i32(cu_k), scale, True)
        attn.kv4_append(k, v, slots, kc, vc, ks, vs)
        for x, n in ((kk, 0), (vv, 1)):
            ref = plain4.rows(plain4.values(mine[n], mine[2 + n]), table.cpu(), before, cu_k, x.double().cpu())
            assert torch.equal(plain4.to16(ref, "fp16"), x.cpu())
        ref = plain64.packed(*(x.double().cpu() for x in (q, kk, vv)), cu.tolist(), cu_k, scale, True, "fp16")
        plain64.check(o, *ref["o"], "prompt")
        remember(k, v, slots)

    turn([37, 1, 100, 64])
    turn([0, 30, 3, 0])

    add = i32([1] * B)
    qt, kt, vt = (torch.empty((B, h, d), dtype=torch.float16, device="cuda") for h in (Hq, H, H))

    def step():
        _, _, _, slots, _ = attn.pages_extend(lens, add, table, stack, count, page, B, new_lens=lens, free_left=count)
        attn.kv4_append(kt, vt, slots, kc, vc, ks, vs)
        return slots, *attn.kv4_decode(qt.view(B, 1, Hq, d), kc, vc, ks, vs, table, lens, scale)

    side = torch.cuda.Stream()
    keep = [x.clone() for x in (lens, table, count, kc, vc, ks, vs)]
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        step()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        slots, o, lse = step()
    for x, y in zip((lens, table, count, kc, vc, ks, vs), keep):
        x.copy_(y)
    torch.cuda.synchronize()
    for i in range(20):
        if i == 8:  # request 2 is done; another takes its place
            attn.pages_release(lens, i32([0, 0, 1, 0]), table, stack, count, page, new_lens=lens, free_left=count)
        for x in (qt, kt, vt):
            x.copy_(torch.randn(x.shape, generator=g).half())
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        remember(kt, vt, slots)
        assert torch.equal(kc.cpu(), mine[0]) and torch.equal(vs.cpu().nan_to_num(-1), mine[3].nan_to_num(-1))
        (ro, bo), (rl, bl) = reference((qt.view(B, 1, Hq, d).cpu(), *mine[:2], *(x.nan_to_num(1.0) for x in mine[2:]),
                                        table.cpu()), lens.tolist(), scale, True, "fp16")
        plain64.check(o, ro, bo, f"step {i}")
        plain64.check(lse, rl, bl, f"lse of step {i}")
    assert attn.attn_status() == 0
