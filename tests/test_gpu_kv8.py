"""The 8-bit paged cache: attn_kv8_append equal to its definition in 64 bits,
attn_kv8_decode within derived bounds of attention over the dequantised pages
(plain64.py), and both together with the tables and the packed prompt."""
import math

import pytest
import torch

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


F8 = torch.float8_e4m3fn


def cache(P, H, page, d, g):
    """Random code values and power-of-two scales: (float8 codes, fp32 scales)."""
    x = torch.randn((P, H, page, d), generator=g) * 60
    s = torch.exp2(torch.randint(-7, 0, (P, H), generator=g).float())
    return x.clamp(-448, 448).to(F8), s


# ------------------------------------------------------------------ append
@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("H,d,dtype", [(1, 64, "fp16"), (3, 128, "bf16"), (2, 64, "bf16")])
def test_append_is_its_definition(page, H, d, dtype):
    """Runs of every kind: whole pages, ends of pages, single tokens at their
    beginning, middle and end, tokens that are skipped, scales that grow and
    that do not."""
    from exact_tiled_attention_22_gb300 import attn
    g = torch.Generator().manual_seed(page + H)
    P = 12
    kc, ks = cache(P, H, page, d, g)
    vc, vs = cache(P, H, page, d, g)
    slots = []
    slots += list(range(3 * page, 4 * page))                      # page 3, whole
    slots += list(range(7 * page, 7 * page + 5))                  # ... and the next one's beginning
    slots += [-1, -1]
    slots += list(range(page + page // 2, 2 * page))              # page 1 from its middle
    slots += [page * 5]                                           # a single first token
    slots += [page * 9 + page - 1]                                # a single last one
    slots += [page * 10 + 3, P * page, P * page + 5, page * 2 + 1]  # singles; outside the cache
    T = len(slots)
    x = [torch.randn((T, H, d), generator=g) * torch.exp2(torch.randint(-6, 7, (T, 1, 1), generator=g).float())
         for _ in range(2)]
    x[0][3] = 0
    x = [t.to(DT[dtype]) for t in x]
    dk, dv, dks, dvs = kc.cuda(), vc.cuda(), ks.cuda(), vs.cuda()
    attn.kv8_append(x[0].cuda(), x[1].cuda(), torch.tensor(slots).cuda(), dk, dv, dks, dvs)
    for t, c, s, got, got_s in ((x[0], kc, ks, dk, dks), (x[1], vc, vs, dv, dvs)):
        val, sc = plain64.append(t.double(), slots, c.double(), s.double())
        assert torch.equal(got_s.double().cpu(), sc)
        assert torch.equal(got.cpu().double(), val)


def test_append_token_by_token():
    """A page filled token by token (every scale change rounds again) and at once."""
    from exact_tiled_attention_22_gb300 import attn
    g = torch.Generator().manual_seed(77)
    page, H, d = 32, 2, 128
    kc, ks = cache(2, H, page, d, g)
    val, sc = kc.double(), ks.double()
    dk, dv, dks, dvs = kc.cuda(), kc.cuda(), ks.cuda(), ks.cuda()
    for i in range(page + 3):
        x = (torch.randn((1, H, d), generator=g) * 1.2 ** i).bfloat16()
        attn.kv8_append(x.cuda(), x.cuda(), torch.tensor([i]).cuda(), dk, dv, dks, dvs)
        val, sc = plain64.append(x.double(), [i], val, sc)
        assert torch.equal(dks.double().cpu(), sc) and torch.equal(dk.cpu().double(), val)
    assert torch.equal(dv.view(torch.uint8), dk.view(torch.uint8)) and torch.equal(dks, dvs)


def test_append_extremes():
    """Zeros, the smallest and largest numbers, infinities (saturate) and NaN (stay)."""
    from exact_tiled_attention_22_gb300 import attn
    page, H, d = 16, 1, 64
    # (449 is 448 in bf16, whose step between 256 and 512 is 2; 450 is itself, and beyond scale 1)
    for fill, code, scale in ((0.0, 0.0, 2.0 ** -64), (1e-38, 0.0, 2.0 ** -64), (3e38, 448.0, 2.0 ** 60),
                              (math.inf, 448.0, 2.0 ** 60), (-448.0, -448.0, 1.0), (449.0, 448.0, 1.0),
                              (450.0, 224.0, 2.0)):
        x = torch.full((page, H, d), fill).bfloat16()
        dk = torch.zeros((1, H, page, d), dtype=torch.uint8, device="cuda")
        dv, sk, sv = dk.clone(), torch.ones((1, H), device="cuda"), torch.ones((1, H), device="cuda")
        attn.kv8_append(x.cuda(), x.cuda(), torch.arange(page).cuda(), dk, dv, sk, sv)
        want = plain64.e4m3(x.double().clamp(-448.0 * 2.0 ** 60, 448.0 * 2.0 ** 60) / scale)
        assert sk.item() == scale and (dk.view(F8).cpu().double() == want[0, 0, 0]).all(), (fill, sk, dk.view(F8)[0, 0, 0, 0])
        assert want[0, 0, 0].item() == code
    x = torch.ones((page, H, d)).half()
    x[4, 0, 7] = math.nan
    dk = torch.zeros((1, H, page, d), dtype=F8, device="cuda")
    dv, sk, sv = dk.clone(), torch.ones((1, H), device="cuda"), torch.ones((1, H), device="cuda")
    attn.kv8_append(x.cuda(), x.cuda(), torch.arange(page).cuda(), dk, dv, sk, sv)
    nan = torch.isnan(dk.float())
    assert nan.sum() == 1 and nan[0, 0, 4, 7] and sk.item() == 2.0 ** -8


def test_append_slices_and_many_tokens():
    """Strided k and v, and the launch shape of long prompts, equal to the
    definition."""
    from exact_tiled_attention_22_gb300 import attn
    g = torch.Generator().manual_seed(5)
    page, H, d, T = 64, 3, 128, 5000
    P = T // page + 4
    x = torch.randn((T, 2 + 2 * H, d), generator=g).half()
    k, v = x[:, 2:2 + H], x[:, 2 + H:]
    perm = torch.randperm(P, generator=g)
    pos = torch.arange(T) + 37
    slots = perm[pos // page] * page + pos % page
    kc, ks = cache(P, H, page, d, g)
    dk, dv, dks, dvs = kc.cuda(), kc.cuda(), ks.cuda(), ks.cuda()
    xg = x.cuda()
    attn.kv8_append(xg[:, 2:2 + H], xg[:, 2 + H:], slots.cuda(), dk, dv, dks, dvs)
    for t, got, got_s in ((k, dk, dks), (v, dv, dvs)):
        val, sc = plain64.append(t.double(), slots.tolist(), kc.double(), ks.double())
        assert torch.equal(got_s.double().cpu(), sc) and torch.equal(got.cpu().double(), val)


# ------------------------------------------------------------------ decode
def problem(lens, Nq, Hq, H, d, page, dtype, seed, pow2=True):
    """A cache with pages in no order, NaN codes in every place that must not be
    looked at, and table entries outside the cache behind the last page."""
    g = torch.Generator().manual_seed(seed)
    B = len(lens)
    need = [-(-n // page) for n in lens]
    P = sum(need) + 2
    kc, ks = cache(P, H, page, d, g)
    vc, vs = cache(P, H, page, d, g)
    if not pow2:
        ks, vs = ks * (0.5 + torch.rand(ks.shape, generator=g)), vs * (0.5 + torch.rand(vs.shape, generator=g))
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
    for c in (kc, vc):
        raw = c.view(torch.uint8)
        raw[~used[:, None, :].expand(P, H, page)] = 0x7F
    q = torch.randn((B, Nq, Hq, d), generator=g).to(DT[dtype])
    return q, kc, vc, ks, vs, table


def decode_and_check(args, lens, scale, causal, dtype):
    from exact_tiled_attention_22_gb300 import attn
    q, kc, vc, ks, vs, table = args
    o, lse = attn.kv8_decode(q.cuda(), kc.cuda(), vc.cuda(), ks.cuda(), vs.cuda(), table.cuda(),
                             torch.tensor(lens, dtype=torch.int32).cuda(), scale, causal)
    attn.check(attn.attn_status())
    (ro, bo), (rl, bl) = plain64.cached(q.double(), kc.double(), vc.double(), ks.double(), vs.double(), table, lens,
                                        scale, causal, dtype)
    plain64.check(lse, rl, bl, "lse")
    plain64.check(o, ro, bo, "o")
    return o, lse


DECODE = [
    # (lens, Nq, Hq, Hkv, d, page, dtype, causal)
    ([1], 1, 1, 1, 64, 16, "fp16", True),
    ([1], 1, 1, 1, 128, 128, "bf16", True),
    ([0, 5, 0], 1, 4, 2, 64, 16, "bf16", True),
    ([127, 128, 129, 16, 17], 1, 8, 2, 128, 16, "bf16", True),
    ([1000, 3, 2049], 1, 32, 4, 128, 64, "bf16", True),
    ([700, 64, 65], 1, 7, 1, 64, 32, "fp16", True),
    ([3000], 1, 16, 1, 128, 128, "fp16", True),
    ([5, 2, 300], 5, 14, 2, 64, 16, "fp16", True),       # requests shorter than the draft
    ([5, 2, 300, 0], 3, 6, 2, 128, 32, "bf16", False),
    ([400, 130], 8, 40, 5, 64, 64, "bf16", True),        # four row blocks
    ([260], 128, 2, 2, 128, 64, "bf16", True),
    ([33] * 400, 1, 2, 1, 64, 16, "fp16", True),         # more requests than threads
    ([20000, 1, 64], 1, 8, 1, 128, 64, "bf16", True),    # split over many blocks
]


@pytest.mark.parametrize("case", DECODE, ids=lambda c: f"B{len(c[0])}q{c[1]}h{c[2]}x{c[3]}d{c[4]}p{c[5]}{c[6]}")
def test_decode(case):
    lens, Nq, Hq, H, d, page, dtype, causal = case
    args = problem(lens, Nq, Hq, H, d, page, dtype, seed=sum(lens) + d)
    decode_and_check(args, lens, d ** -0.5, causal, dtype)


def test_decode_other_scales():
    """Scales that are no powers of two, and values whose pages differ by 2^40."""
    lens = [300, 513]
    args = problem(lens, 1, 8, 2, 128, 32, "bf16", seed=1, pow2=False)
    decode_and_check(args, lens, 0.1, True, "bf16")
    q, kc, vc, ks, vs, table = problem(lens, 1, 8, 2, 64, 16, "fp16", seed=2)
    vs *= torch.exp2(torch.randint(-20, 21, vs.shape, generator=torch.Generator().manual_seed(3)).float())
    from exact_tiled_attention_22_gb300 import attn
    o, _ = attn.kv8_decode(q.bfloat16().cuda(), kc.cuda(), vc.cuda(), ks.cuda(), vs.cuda(), table.cuda(),
                           torch.tensor(lens, dtype=torch.int32).cuda(), 0.1, True)
    (ro, bo), _ = plain64.cached(q.bfloat16().double(), kc.double(), vc.double(), ks.double(), vs.double(), table,
                                 lens, 0.1, True, "bf16")
    plain64.check(o, ro, bo, "o")


def test_decode_sharp_scores_and_wide_queries():
    """Scores in the hundreds (the running maximum moves) and queries whose
    elements span 2^-20 .. 2^4."""
    lens = [900]
    q, kc, vc, ks, vs, table = problem(lens, 2, 8, 1, 64, 16, "bf16", seed=8)
    ks *= 16
    decode_and_check((q, kc, vc, ks, vs, table), lens, 1.0, True, "bf16")
    g = torch.Generator().manual_seed(9)
    q = (torch.randn(q.shape, generator=g) * torch.exp2(torch.randint(-20, 5, q.shape, generator=g).float())).bfloat16()
    decode_and_check((q, kc, vc, ks, vs, table), lens, 0.01, True, "bf16")


def test_decode_not_numbers_stay_where_they_are():
    """A NaN in a query or a cached token reaches the heads that see it, no other."""
    from exact_tiled_attention_22_gb300 import attn
    lens = [200, 200]
    q, kc, vc, ks, vs, table = problem(lens, 2, 4, 2, 64, 16, "fp16", seed=12)
    clean, _ = attn.kv8_decode(q.cuda(), kc.cuda(), vc.cuda(), ks.cuda(), vs.cuda(), table.cuda(),
                               torch.tensor(lens, dtype=torch.int32).cuda())
    q[0, 1, 3] = math.inf
    kc.view(torch.uint8)[table[1, 0], 1, 3, 5] = 0x7F      # key head 1 of request 1
    vc.view(torch.uint8)[table[1, 12], 0, 7, 9] = 0xFF     # its last token's value, head 0, element 9
    o, _ = attn.kv8_decode(q.cuda(), kc.cuda(), vc.cuda(), ks.cuda(), vs.cuda(), table.cuda(),
                           torch.tensor(lens, dtype=torch.int32).cuda())
    nan = torch.isnan(o)
    want = torch.zeros_like(nan)
    want[0, 1, 3] = True
    want[1, :, 2:] = True
    want[1, :, :2, 9] = True                                # (a hidden NaN times a zero is one, too)
    assert torch.equal(nan, want)
    assert torch.equal(o[~want], clean[~want])


def test_decode_far_into_a_large_cache():
    """Pages whose byte offsets pass 2^32 and 2^31 elements, written by append."""
    from exact_tiled_attention_22_gb300 import attn
    H, d, page = 8, 128, 128
    P = (1 << 32) // (H * d * page) + 40
    kc = torch.zeros((P, H, page, d), dtype=torch.uint8, device="cuda")
    vc = torch.zeros_like(kc)
    ks, vs = torch.ones((P, H), device="cuda"), torch.ones((P, H), device="cuda")
    g = torch.Generator().manual_seed(3)
    n = 300
    ids = torch.tensor([P - 1, 5, P - 30])
    pos = torch.arange(n)
    slots = ids[pos // page] * page + pos % page
    k, v = (torch.randn((n, H, d), generator=g).bfloat16() for _ in range(2))
    attn.kv8_append(k.cuda(), v.cuda(), slots.cuda(), kc, vc, ks, vs)
    q = torch.randn((1, 1, H, d), generator=g).bfloat16()
    table = ids.int()[None]
    o, lse = attn.kv8_decode(q.cuda(), kc, vc, ks, vs, table.cuda(), torch.tensor([n], dtype=torch.int32).cuda())
    few = lambda c: c[ids.cuda()].view(F8).cpu().double()  # noqa: E731
    (ro, bo), (rl, bl) = plain64.cached(q.double(), few(kc), few(vc), ks[ids.cuda()].cpu().double(),
                                        vs[ids.cuda()].cpu().double(), torch.tensor([[0, 1, 2]]), [n], d ** -0.5,
                                        True, "bf16")
    plain64.check(o, ro, bo, "o")
    plain64.check(lse, rl, bl, "lse")


def test_two_calls_at_once_and_repeats():
    """Two streams with their own workspaces; equal results every time."""
    from exact_tiled_attention_22_gb300 import attn
    lens = [5000, 17, 900]
    args = [x.cuda() for x in problem(lens, 1, 16, 4, 128, 64, "bf16", seed=4)]
    ln = torch.tensor(lens, dtype=torch.int32).cuda()
    want = attn.kv8_decode(*args, ln)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for _ in range(5):
        for s in streams:
            with torch.cuda.stream(s):
                got.append(attn.kv8_decode(*args, ln))
    torch.cuda.synchronize()
    for o, lse in got:
        assert torch.equal(o, want[0]) and torch.equal(lse, want[1])


def test_pages_that_are_not_there_read_as_zeros():
    """Page ids outside the cache within a request's length: zero keys and values
    (the scales of page 0 may be anything)."""
    from exact_tiled_attention_22_gb300 import attn
    lens = [150]
    q, kc, vc, ks, vs, table = problem(lens, 1, 4, 2, 64, 16, "bf16", seed=14)
    gone = [1, 4, 7]
    zk, zv = kc.clone(), vc.clone()
    for j in gone:
        zk.view(torch.uint8)[table[0, j]] = 0
        zv.view(torch.uint8)[table[0, j]] = 0
    (ro, bo), (rl, bl) = plain64.cached(q.double(), zk.double(), zv.double(), ks.double(), vs.double(), table, lens,
                                        0.125, True, "bf16")
    spare = [p for p in range(kc.shape[0]) if p not in table[0].tolist()][0]
    bad = table.clone()
    # page 0's scales are NaN, and the pages that are not there have ids -1, P, 2^31 - 1
    keep = bad[0] == 0
    if keep.any():  # (page 0 is in use: its contents move to a spare page)
        for c in (kc, vc, ks, vs):
            c[spare] = c[0].clone()
        bad[0][keep] = spare
    ks[0], vs[0] = math.nan, math.nan
    for j, i in zip(gone, (-1, kc.shape[0], 2 ** 31 - 1)):
        bad[0, j] = i
    o, lse = attn.kv8_decode(q.cuda(), kc.cuda(), vc.cuda(), ks.cuda(), vs.cuda(), bad.cuda(),
                             torch.tensor(lens, dtype=torch.int32).cuda(), 0.125)
    plain64.check(lse, rl, bl, "lse")
    plain64.check(o, ro, bo, "o")


def test_errors_of_the_calls():
    """What the tensors cannot be raises ValueError, what the library refuses
    AttnError with its code; nothing is enqueued and the next call works."""
    from exact_tiled_attention_22_gb300 import attn
    lens = [20, 40]
    q, kc, vc, ks, vs, table = (x.cuda() for x in problem(lens, 1, 4, 2, 64, 16, "fp16", seed=16))
    ln = torch.tensor(lens, dtype=torch.int32).cuda()
    want = attn.kv8_decode(q, kc, vc, ks, vs, table, ln)
    for bad in (dict(q=q.float()), dict(q=q[0]), dict(q=q.transpose(0, 1)), dict(q=q.cpu()), dict(kc=kc.float()),
                dict(vc=vc[:-1]), dict(ks=ks.half()), dict(table=table.long()), dict(table=table[:1]),
                dict(ln=ln.cpu()), dict(ln=[20, 40]), dict(ws=torch.zeros(8))):
        a = dict(q=q, kc=kc, vc=vc, ks=ks, vs=vs, table=table, ln=ln, ws=None)
        a.update(bad)
        with pytest.raises(ValueError):
            attn.kv8_decode(a["q"], a["kc"], a["vc"], a["ks"], a["vs"], a["table"], a["ln"], ws=a["ws"])
    for bad, code in ((dict(q=q[:, :, :3].contiguous()), attn.ATTN_ERR_INVALID), (dict(scale=-1.0), attn.ATTN_ERR_INVALID),
                      (dict(ws=torch.zeros(1024, device="cuda")), attn.ATTN_ERR_WORKSPACE)):
        with pytest.raises(attn.AttnError) as e:
            attn.kv8_decode(bad.get("q", q), kc, vc, ks, vs, table, ln, bad.get("scale"), ws=bad.get("ws"))
        assert e.value.code == code and str(e.value)
    with pytest.raises(attn.AttnError):
        attn.kv8_append(q[0, :, :2], q[0, :, :2], torch.zeros(1, dtype=torch.int64, device="cuda"), kc[:, :, :8].contiguous(),
                        vc[:, :, :8].contiguous(), ks, vs)
    got = attn.kv8_decode(q, kc, vc, ks, vs, table, ln)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_stream_argument():
    """stream= as a torch stream and as a handle; what the call allocates belongs
    to that stream."""
    from exact_tiled_attention_22_gb300 import attn
    lens = [700, 80]
    args = [x.cuda() for x in problem(lens, 1, 8, 2, 64, 32, "fp16", seed=15)]
    ln = torch.tensor(lens, dtype=torch.int32).cuda()
    want = attn.kv8_decode(*args, ln)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    a = attn.kv8_decode(*args, ln, stream=side)
    b = attn.kv8_decode(*args, ln, stream=side.cuda_stream)
    side.synchronize()
    for got in (a, b):
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("lens", [[127, 128, 129, 16, 17], [1, 1, 1], [3000, 5], [128] * 40])
def test_what_the_workspace_held_does_not_matter(lens):
    """A workspace full of NaN: only parts that this call wrote are read, also
    when there are fewer tiles than blocks."""
    from exact_tiled_attention_22_gb300 import attn
    args = [x.cuda() for x in problem(lens, 1, 8, 2, 128, 16, "bf16", seed=4)]
    ln = torch.tensor(lens, dtype=torch.int32).cuda()
    n = attn.attn_kv8_decode_workspace_size(1, 8, 2, 128)
    clean = torch.zeros(n, dtype=torch.uint8, device="cuda")
    dirty = torch.full((n // 4,), math.nan, device="cuda").view(torch.uint8)
    a, b = attn.kv8_decode(*args, ln, ws=clean), attn.kv8_decode(*args, ln, ws=dirty)
    assert torch.isfinite(a[0]).all() and torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_wait_limit_reports_a_timeout():
    from exact_tiled_attention_22_gb300 import attn
    lens = [300]
    args = [x.cuda() for x in problem(lens, 1, 2, 1, 64, 16, "fp16", seed=6)]
    ln = torch.tensor(lens, dtype=torch.int32).cuda()
    want = attn.kv8_decode(*args, ln)
    try:
        attn.attn_set_wait_limit(50_000_000, 16)
        attn.kv8_decode(*args, ln)
        assert attn.attn_status() == attn.ATTN_ERR_TIMEOUT
    finally:
        attn.attn_set_wait_limit(0, 0)
    got = attn.kv8_decode(*args, ln)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


# ------------------------------------------------------------------ together
def test_a_serving_run():
    """Prompts of different lengths are attended to as a packed batch, written to
    the cache, and decoded token by token from a captured step; requests leave
    and their pages are used again.  Every step against 64 bits over the cache
    as the definition fills it."""
    from exact_tiled_attention_22_gb300 import attn
    B, Hq, H, d, page, width = 4, 8, 2, 64, 16, 12
    g = torch.Generator().manual_seed(42)
    P = 40
    i32 = lambda x: torch.tensor(x, dtype=torch.int32).cuda()  # noqa: E731
    kc = torch.full((P, H, page, d), 0x7F, dtype=torch.uint8, device="cuda").view(F8)  # nothing written yet
    vc = kc.clone()
    ks, vs = torch.full((P, H), math.nan, device="cuda"), torch.full((P, H), math.nan, device="cuda")
    table, stack, count = i32([[-1] * width] * B), i32(torch.randperm(P, generator=g).tolist()), i32([P])
    lens = i32([0] * B)
    val = [kc.double().cpu(), vc.double().cpu()]
    sc = [ks.double().cpu(), vs.double().cpu()]
    scale = d ** -0.5

    def remember(k, v, slots):
        for i, x in enumerate((k, v)):
            val[i], sc[i] = plain64.append(x.double().cpu(), slots.tolist(), val[i], sc[i])

    prompts = [37, 1, 100, 64]
    T = sum(prompts)
    q, k, v = (torch.randn((T, h, d), generator=g).half().cuda() for h in (Hq, H, H))
    _, _, cu, slots, _ = attn.pages_extend(lens, i32(prompts), table, stack, count, page, T, new_lens=lens,
                                           free_left=count)
    o, lse = attn.varlen_fwd(q, k, v, cu, cu, scale, True)
    attn.kv8_append(k, v, slots, kc, vc, ks, vs)
    ref = plain64.packed(*(x.double().cpu() for x in (q, k, v)), cu.tolist(), cu.tolist(), scale, True, "fp16")
    plain64.check(o, *ref["o"], "prompt")
    remember(k, v, slots)

    add = i32([1] * B)
    qt, kt, vt = (torch.empty((B, h, d), dtype=torch.float16, device="cuda") for h in (Hq, H, H))

    def step():
        _, _, _, slots, _ = attn.pages_extend(lens, add, table, stack, count, page, B, new_lens=lens, free_left=count)
        attn.kv8_append(kt, vt, slots, kc, vc, ks, vs)
        return slots, *attn.kv8_decode(qt.view(B, 1, Hq, d), kc, vc, ks, vs, table, lens, scale)

    side = torch.cuda.Stream()
    keep = [x.clone() for x in (lens, table, count, kc.view(torch.uint8), vc.view(torch.uint8), ks, vs)]
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        step()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        slots, o, lse = step()
    for x, y in zip((lens, table, count, kc.view(torch.uint8), vc.view(torch.uint8), ks, vs), keep):
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
        assert torch.equal(kc.cpu().double().nan_to_num(0.5), val[0].nan_to_num(0.5))
        assert torch.equal(vs.cpu().double().nan_to_num(-1), sc[1].nan_to_num(-1))
        (ro, bo), (rl, bl) = plain64.cached(qt.view(B, 1, Hq, d).double().cpu(), *(x.nan_to_num(0.0) for x in val),
                                            *(x.nan_to_num(1.0) for x in sc), table.cpu(), lens.tolist(), scale, True,
                                            "fp16")
        plain64.check(o, ro, bo, f"step {i}")
        plain64.check(lse, rl, bl, f"lse of step {i}")
    assert attn.attn_status() == 0


def test_stream_handle_with_keyword_arguments():
    """A handle says nothing of its device: that is the tensors', wherever they stand
    among the arguments."""
    from exact_tiled_attention_22_gb300 import attn
    lens = [90]
    q, kc, vc, ks, vs, table = (x.cuda() for x in problem(lens, 1, 4, 2, 64, 32, "bf16", seed=16))
    ln = torch.tensor(lens, dtype=torch.int32).cuda()
    want = attn.kv8_decode(q, kc, vc, ks, vs, table, ln)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for stream in (side.cuda_stream, 0):
        o, lse = attn.kv8_decode(q=q, k_cache=kc, v_cache=vc, k_scale=ks, v_scale=vs, block_table=table, lens=ln,
                                 stream=stream)
        torch.cuda.synchronize()
        assert torch.equal(o, want[0]) and torch.equal(lse, want[1])
    with pytest.raises(ValueError):
        attn.kv8_decode(q.cpu(), kc, vc, ks, vs, table, ln, stream=side.cuda_stream)


def test_more_rows_than_blocks_of_the_merge():
    """So many requests that a block of the merge takes several rows of several of
    them, empty ones and ones that several blocks of the split share among them."""
    g = torch.Generator().manual_seed(17)
    lens = torch.randint(0, 4, (1000,), generator=g)
    lens[torch.tensor([0, 1, 399, 700, 999])] = torch.tensor([1500, 0, 3000, 257, 0], dtype=lens.dtype)
    lens = lens.tolist()
    args = problem(lens, 1, 5, 5, 64, 16, "bf16", seed=18)
    decode_and_check(args, lens, 0.125, True, "bf16")


def test_tensors_freed_after_a_call_on_another_stream():
    """The memory of a query that is dropped after the call is not handed on while
    the call still waits for its stream."""
    from exact_tiled_attention_22_gb300 import attn
    lens = [300] * 64
    q, kc, vc, ks, vs, table = (x.cuda() for x in problem(lens, 1, 32, 4, 128, 32, "bf16", seed=19))
    ln = torch.tensor(lens, dtype=torch.int32).cuda()
    want = attn.kv8_decode(q, kc, vc, ks, vs, table, ln)
    side = torch.cuda.Stream()
    big = torch.randn(8192, 8192, device="cuda")
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        for _ in range(4):
            big @ big                       # the call waits behind these
    mine = q.clone()
    torch.cuda.current_stream().synchronize()
    o, lse = attn.kv8_decode(mine, kc, vc, ks, vs, table, ln, stream=side)
    del mine
    others = [torch.full_like(q, math.nan) for _ in range(8)]
    torch.cuda.synchronize()
    assert torch.equal(o, want[0]) and torch.equal(lse, want[1])
    del others


@pytest.mark.parametrize("H,d,page,T", [(8, 128, 16, 640), (8, 64, 64, 1000), (1, 128, 32, 5000), (3, 64, 128, 1700)])
def test_append_single_tokens_of_many_requests(H, d, page, T):
    """A decoding step of many requests, where a warp looks after 32 tokens and every one
    is a run of its own: at any place of its page, the scale growing or not, skipped ones
    and a few short prompts among them."""
    from exact_tiled_attention_22_gb300 import attn
    assert T * H * 2 > 64 * 152               # the launcher's border
    g = torch.Generator().manual_seed(T)
    P = T + 40
    kc, ks = cache(P, H, page, d, g)
    vc, vs = cache(P, H, page, d, g)
    pages = torch.randperm(P, generator=g)
    place = torch.randint(0, page, (T,), generator=g)
    place[::3] = 0
    slots = pages[:T] * page + place
    slots[5::50] = -1
    n = min(page, 17)
    for i, t in enumerate(range(64, T - 64, 320)):            # a run over the end of a warp's 32 tokens
        slots[t + 25:t + 25 + n] = pages[T + i] * page + torch.arange(n)
    x = [(torch.randn((T, H, d), generator=g) * torch.exp2(torch.randint(-6, 7, (T, 1, 1), generator=g).float())).to(
        DT["bf16"]) for _ in range(2)]
    dk, dv, dks, dvs = kc.cuda(), vc.cuda(), ks.cuda(), vs.cuda()
    attn.kv8_append(x[0].cuda(), x[1].cuda(), slots.cuda(), dk, dv, dks, dvs)
    for t, c, s, got, got_s in ((x[0], kc, ks, dk, dks), (x[1], vc, vs, dv, dvs)):
        val, sc = plain64.append(t.double(), slots.tolist(), c.double(), s.double())
        assert torch.equal(got_s.double().cpu(), sc) and torch.equal(got.cpu().double(), val)
