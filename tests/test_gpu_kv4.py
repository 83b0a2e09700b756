"""The 4-bit paged cache: attn_kv4_append equal to its definition in 64 bits
(plain4.py), attn_kv_read equal to what a cache in 4 or 8 bits stands for."""
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


F8 = torch.float8_e4m3fn


def i32(x):
    return torch.tensor(x, dtype=torch.int32).cuda()


def bits(x):
    return x.cpu().view(torch.int16)


# ------------------------------------------------------------------ append
def check_append(k, v, slots, kc, vc, ks, vs, kg=None, vg=None):
    """Codes and scales after a call, bit for bit.  kg, vg: the tensors to pass, where they are slices."""
    from exact_tiled_attention_22_gb300 import attn
    got = [x.cuda() for x in (kc, vc, ks, vs)]
    attn.kv4_append(k.cuda() if kg is None else kg, v.cuda() if vg is None else vg,
                    torch.tensor(slots, dtype=torch.int64).cuda(), *got)
    for x, c, s, gc, gs in ((k, kc, ks, got[0], got[2]), (v, vc, vs, got[1], got[3])):
        wc, ws = plain4.append(x.double(), slots, c, s)
        nan = torch.isnan(ws.float())
        assert torch.equal(torch.isnan(gs.cpu().float()), nan)
        assert torch.equal(bits(gs)[~nan], bits(ws)[~nan])
        same = gc.cpu() == wc
        same |= nan.repeat_interleave(16, -1)     # (what codes a NaN's group holds does not matter)
        assert same.all()
    return got


@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("H,d,dtype", [(1, 64, "fp16"), (3, 128, "bf16"), (2, 64, "bf16"), (5, 128, "fp16")])
def test_append_is_its_definition(page, H, d, dtype):
    """Whole pages, single tokens, no order, skipped tokens and slots outside the cache; every other
    place keeps its codes and scales."""
    g = torch.Generator().manual_seed(page + H)
    P = 9
    kc, ks = plain4.cache(P, H, page, d, g)
    vc, vs = plain4.cache(P, H, page, d, g)
    slots = list(range(3 * page, 4 * page)) + [page * 5, -1, page * 7 + page - 1, page + 3, page + 1, -7, P * page,
                                               P * page + 5, 1 << 40, 0, P * page - 1]
    T = len(slots)
    k, v = ((torch.randn((T, H, d), generator=g) * torch.exp2(torch.randint(-9, 10, (T, H, 1), generator=g).float()))
            .to(DT[dtype]) for _ in range(2))
    k[3] = 0.0
    v[4, 0, 32:64] = -0.0
    check_append(k, v, slots, kc, vc, ks, vs)


@pytest.mark.parametrize("T,H,d,page", [(1, 1, 64, 16), (1, 1, 128, 128), (7, 300, 64, 16), (5000, 3, 128, 64),
                                        (20000, 1, 64, 32), (1201, 7, 64, 16), (2, 4100, 128, 16), (700, 40, 128, 32),
                                        (21001, 8, 128, 16), (4003, 83, 64, 64)])
def test_append_launch_shapes(T, H, d, page):
    """From one token of one head to blocks of many tokens, tokens of many blocks and blocks that read ahead, k and v
    slices of one projection."""
    g = torch.Generator().manual_seed(T)
    P = T // page + 2
    x = torch.randn((T, 1 + 2 * H, d), generator=g).half()
    slots = torch.randperm(P * page, generator=g)[:T].tolist()
    kc, ks = plain4.cache(P, H, page, d, g)
    xg = x.cuda()
    check_append(x[:, 1:1 + H], x[:, 1 + H:], slots, kc, kc.flip(0), ks, ks.flip(0), xg[:, 1:1 + H], xg[:, 1 + H:])


@pytest.mark.parametrize("T,H,d", [(5, 2, 64), (21001, 8, 128)])
def test_append_tokens_on_16_byte_borders(T, H, d):
    """Token strides that are multiples of 8 only, and a first token between two 32-byte borders."""
    g = torch.Generator().manual_seed(T)
    flat = torch.randn(8 + T * (H * d + 8), generator=g).bfloat16()
    fg = flat.cuda()
    view = lambda f: f.as_strided((T, H, d), (H * d + 8, d, 1), 8)  # noqa: E731
    P = T // 16 + 1
    slots = torch.randperm(P * 16, generator=g)[:T].tolist()
    kc, ks = plain4.cache(P, H, 16, d, g)
    check_append(view(flat), view(flat), slots, kc, kc, ks, ks, view(fg), view(fg))


@pytest.mark.parametrize("s", [1.0, 75 / 64, 129 / 128, 85 / 32, 2.0 ** -14 * 1.5])
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
def test_append_borders(s, dtype):
    """Values on the borders between two codes, and a step of the type beside them, for scales that are and
    are not powers of two."""
    border = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], dtype=torch.float64) * s
    x = border.to(DT[dtype])
    near = torch.cat([x, torch.nextafter(x, x * 2), torch.nextafter(x, x * 0), torch.tensor([6 * s]).to(DT[dtype])])
    row = torch.zeros(1, 1, 64, dtype=DT[dtype])
    row[0, 0, :22], row[0, 0, 32:54] = near, -near
    kc, ks = plain4.cache(1, 1, 16, 64, torch.Generator().manual_seed(1))
    check_append(row, row.flip(2).contiguous(), [3], kc, kc, ks, ks)


def test_append_extremes():
    """Zeros, the smallest and largest numbers, infinities (saturate), NaN (its group reads as NaN)."""
    g = torch.Generator().manual_seed(2)
    kc, ks = plain4.cache(1, 1, 16, 128, g)
    for fill in (0.0, -0.0, 1e-38, -1e-40, 3e38, -3e38, math.inf, -math.inf, 2.0 ** 62, 7.0 * 2.0 ** 60, 2.0 ** -61):
        x = torch.full((1, 1, 128), fill).bfloat16()
        x[0, 0, 64:] = torch.randn(64, generator=g).bfloat16()
        x[0, 0, 96] = fill
        check_append(x, -x, [5], kc, kc, ks, ks)
    for dtype in (torch.float16, torch.bfloat16):
        x = torch.randn((2, 1, 128), generator=g).to(dtype)
        x[0, 0, 7], x[1, 0, 127] = math.nan, -math.nan
        x[1, 0, 40] = -math.inf
        x[1, 0, 0] = torch.finfo(dtype).max
        got = check_append(x, x, [1, 4], kc, kc, ks, ks)
        nan = torch.isnan(got[2].float())
        assert nan.sum() == 2 and nan[0, 0, 1, 0] and nan[0, 0, 4, 3]


# ------------------------------------------------------------------ read
def cache8(P, H, page, d, g):
    x = torch.randn((P, H, page, d), generator=g) * 60
    return x.clamp(-448, 448).to(F8), torch.exp2(torch.randint(-7, 0, (P, H), generator=g).float())


def stands_for(c, s, nbits):
    return c.double() * s.double()[..., None, None] if nbits == 8 else plain4.values(c, s)


def read_problem(nbits, lens, H, d, page, g):
    B = len(lens)
    need = [-(-n // page) for n in lens]
    P = sum(need) + 2
    make = cache8 if nbits == 8 else plain4.cache
    (kc, ks), (vc, vs) = make(P, H, page, d, g), make(P, H, page, d, g)
    table = torch.full((B, max(need) + 1), 1 << 30, dtype=torch.int32)
    ids, at = torch.randperm(P, generator=g).int(), 0
    for b in range(B):
        table[b, :need[b]] = ids[at:at + need[b]]
        at += need[b]
    return kc, vc, ks, vs, table


def check_read(nbits, args, lens, cu, T, dtype, given=True):
    """Rows of tokens bit for bit; all others as they were (where the outputs were given)."""
    from exact_tiled_attention_22_gb300 import attn
    kc, vc, ks, vs, table = args
    H, d = kc.shape[1], kc.shape[3] * 8 // nbits
    call = attn.kv8_read if nbits == 8 else attn.kv4_read
    out = [torch.full((T, H, d), -7.0 - i, dtype=DT[dtype], device="cuda") for i in range(2)] if given else [None, None]
    got = call(*(x.cuda() for x in args), i32(lens), i32(cu), T, DT[dtype], *out)
    fill = torch.full((T, H, d), math.inf, dtype=torch.float64)
    for i, (c, s) in enumerate(((kc, ks), (vc, vs))):
        want = plain4.rows(stands_for(c, s, nbits), table, lens, cu, fill)
        untouched = torch.isinf(want)
        want = plain4.to16(want, dtype)
        if given:
            assert got[i].data_ptr() == out[i].data_ptr()
            want[untouched] = -7.0 - i
            assert torch.equal(bits(got[i]), bits(want))
        else:
            assert torch.equal(bits(got[i])[~untouched], bits(want)[~untouched])
    return got


@pytest.mark.parametrize("nbits", [4, 8])
@pytest.mark.parametrize("lens,room,H,d,page,dtype", [
    ([1], 0, 1, 64, 16, "bf16"), ([1], 3, 1, 128, 128, "fp16"), ([0, 5, 0, 33, 0], 2, 2, 64, 16, "fp16"),
    ([127, 128, 129, 16, 17], 0, 3, 128, 32, "bf16"), ([700, 3, 1025], 40, 8, 128, 64, "bf16"),
    ([260, 5], 1, 5, 64, 64, "bf16"), ([40, 50], 7, 300, 64, 16, "fp16"), ([2, 0, 3] * 50, 1, 1, 64, 16, "fp16")])
def test_read(nbits, lens, room, H, d, page, dtype):
    """Rows of new tokens behind the cached ones, rows before the first and behind the last request: left as
    they were."""
    g = torch.Generator().manual_seed(sum(lens) + d)
    cu = [3]
    for n in lens:
        cu.append(cu[-1] + n + room)
    args = read_problem(nbits, lens, H, d, page, g)
    check_read(nbits, args, lens, cu, cu[-1] + 5, dtype)
    check_read(nbits, args, lens, cu, cu[-1] + 5, dtype, given=False)


@pytest.mark.parametrize("nbits", [4, 8])
def test_read_clips(nbits):
    """More tokens than rows, fewer rows than offsets say, lengths beyond the table, a negative one, pages that
    are not there."""
    from exact_tiled_attention_22_gb300 import attn
    g = torch.Generator().manual_seed(9)
    lens = [40, 40, 33]
    args = read_problem(nbits, lens, 2, 64, 16, g)
    table = args[4]
    table[0, 1], table[1, 0], table[2, 2] = -1, args[0].shape[0], 2 ** 31 - 1
    check_read(nbits, args, lens, [0, 40, 70, 103], 103, "bf16")      # request 1: 30 of its 40 tokens
    check_read(nbits, args, lens, [0, 40, 80, 113], 90, "fp16")       # 90 rows in all
    table[:, 3] = 0
    check_read(nbits, args, [-3, 1000, 16], [0, 0, 200, 216], 216, "bf16")
    for T in (0, 1):
        k, v = (attn.kv8_read if nbits == 8 else attn.kv4_read)(*(x.cuda() for x in args), i32([0] * 3), i32([0] * 4), T)
        assert k.shape == v.shape == (T, 2, 64) and k.dtype == torch.bfloat16


def test_read_saturates_and_keeps_nan():
    """A scale rounded up makes 6 s pass fp16's largest number, as a power of two does for e4m3: those read as
    the largest.  A group with a NaN scale, and an e4m3 NaN, read as NaN."""
    from exact_tiled_attention_22_gb300 import attn
    page, d = 16, 64
    x = torch.full((1, 1, d), 65504.0).half()
    x[0, 0, 1::2] = -65504.0
    ends = [torch.zeros((1, 1, page, d // 2), dtype=torch.uint8, device="cuda") for _ in range(2)]
    sc = [torch.ones((1, 1, page, 2), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    attn.kv4_append(x.cuda(), x.cuda(), torch.tensor([2]).cuda(), *ends, *sc)
    assert 6 * sc[0][0, 0, 2, 0].item() > 65504
    sc[1][0, 0, 2, 1] = math.nan
    k, v = attn.kv4_read(*ends, *sc, i32([[0]]), i32([3]), i32([0, 3]), 3, torch.float16)
    assert torch.equal(k[2].cpu(), x[0]) and torch.equal(v[2, :, :32].cpu(), x[0, :, :32])
    assert torch.isnan(v[2, :, 32:]).all() and (k[:2] == 0).all()
    c8 = [torch.zeros((1, 1, page, d), dtype=F8, device="cuda") for _ in range(2)]
    s8 = [torch.ones((1, 1), device="cuda") for _ in range(2)]
    attn.kv8_append(x.cuda(), x.cuda(), torch.tensor([0]).cuda(), *c8, *s8)
    c8[1].view(torch.uint8)[0, 0, 0, 5] = 0x7F
    k, v = attn.kv8_read(*c8, *s8, i32([[0]]), i32([1]), i32([0, 1]), 1, torch.float16)
    assert torch.equal(k[0].cpu(), x[0]) and torch.isnan(v[0, 0, 5]) and torch.isnan(v).sum() == 1


def test_read_of_many_requests():
    """More requests than a block has threads, most of them empty."""
    g = torch.Generator().manual_seed(4)
    lens = torch.where(torch.rand(3001, generator=g) < 0.2, torch.randint(0, 20, (3001,), generator=g), 0).tolist()
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    check_read(4, read_problem(4, lens, 1, 64, 16, g), lens, cu, cu[-1], "bf16")


# ------------------------------------------------------------------ errors, streams
def test_errors_of_append_and_read():
    """What the tensors cannot be raises ValueError, what the library refuses AttnError."""
    from exact_tiled_attention_22_gb300 import attn
    g = torch.Generator().manual_seed(3)
    kc, vc, ks, vs, table = (x.cuda() for x in read_problem(4, [20, 3], 2, 64, 16, g))
    k = torch.zeros((3, 2, 64), dtype=torch.float16, device="cuda")
    slots = torch.arange(3).cuda()
    for bad in (dict(k=k.float()), dict(k=k[0]), dict(v=k.bfloat16()), dict(v=k.cpu()), dict(k=k.transpose(1, 2)),
                dict(kc=kc.to(torch.int8)), dict(vc=vc[:-1]), dict(ks=ks.half()), dict(vs=vs[..., :1]),
                dict(slots=slots.int()), dict(slots=slots[:2]), dict(kc=kc[..., ::2])):
        a = dict(k=k, v=k, slots=slots, kc=kc, vc=vc, ks=ks, vs=vs)
        a.update(bad)
        with pytest.raises(ValueError):
            attn.kv4_append(*a.values())
    lens, cu = i32([20, 3]), i32([0, 20, 23])
    for bad in (dict(kc=kc.float()), dict(table=table.long()), dict(table=table[:1]), dict(lens=lens.cpu()),
                dict(cu=cu[:2]), dict(total=-1), dict(dtype=torch.float32), dict(k=k), dict(v=k.cpu()),
                dict(k=torch.zeros((23, 2, 64), device="cuda"))):
        a = dict(kc=kc, vc=vc, ks=ks, vs=vs, table=table, lens=lens, cu=cu, total=23, dtype=torch.float16, k=None, v=None)
        a.update(bad)
        with pytest.raises(ValueError):
            attn.kv4_read(*a.values())
    with pytest.raises(attn.AttnError) as e:
        attn.kv4_append(k, k, slots, *(x[:, :, :8].contiguous() for x in (kc, vc, ks, vs)))
    assert e.value.code == attn.ATTN_ERR_UNSUPPORTED
    out = torch.zeros((23, 2, 64), dtype=torch.float16, device="cuda")
    with pytest.raises(attn.AttnError) as e:
        attn.kv4_read(kc, vc, ks, vs, table, lens, cu, 23, torch.float16, out, out)
    assert e.value.code == attn.ATTN_ERR_INVALID
    got = attn.kv4_read(kc, vc, ks, vs, table, lens, cu, 23, torch.float16)
    assert torch.isfinite(got[0]).all()


def test_streams_of_append_and_read():
    """stream= and a captured, replayed pair on another stream than the tensors' own."""
    from exact_tiled_attention_22_gb300 import attn
    g = torch.Generator().manual_seed(8)
    lens, H, d, page = [50, 33], 2, 128, 32
    kc, vc, ks, vs, table = (x.cuda() for x in read_problem(4, lens, H, d, page, g))
    x = torch.randn((4, H, d), generator=g).bfloat16().cuda()
    slots = torch.cat([table[0, 1:2].long() * page + torch.arange(16, 18).cuda(), table[1, :1].long() * page,
                       torch.tensor([-1]).cuda()])
    ln, cu = i32(lens), i32([0, 50, 83])
    keep = [t.clone() for t in (kc, vc, ks, vs)]
    attn.kv4_append(x, x, slots, kc, vc, ks, vs)
    want = attn.kv4_read(kc, vc, ks, vs, table, ln, cu, 83)
    state = [t.clone() for t in (kc, vc, ks, vs)]
    side = torch.cuda.Stream()

    def reset():
        for t, o in zip((kc, vc, ks, vs), keep):
            t.copy_(o)
        torch.cuda.synchronize()

    reset()
    attn.kv4_append(x, x, slots, kc, vc, ks, vs, stream=side)
    got = attn.kv4_read(kc, vc, ks, vs, table, ln, cu, 83, stream=side.cuda_stream)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        attn.kv4_append(x, x, slots, kc, vc, ks, vs)
        got = attn.kv4_read(kc, vc, ks, vs, table, ln, cu, 83)
    for _ in range(2):
        reset()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        assert all(torch.equal(a, b) for a, b in zip((kc, vc, ks, vs), state))


# ------------------------------------------------------------------ the C ABI's mirrors
def test_raw_calls():
    """attn_kv4_append, attn_kv4_decode and attn_kv_read on the caller's buffers and stream: the bits of the
    conveniences."""
    from exact_tiled_attention_22_gb300 import attn
    g = torch.Generator().manual_seed(11)
    lens, H, Hq, d, page = [40, 900], 2, 8, 128, 32
    kc, vc, ks, vs, table = (x.cuda() for x in read_problem(4, lens, H, d, page, g))
    P, width = kc.shape[0], table.shape[1]
    new = torch.randn((2, 2, H, d), generator=g).bfloat16().cuda()
    q = torch.randn((2, 1, Hq, d), generator=g).bfloat16().cuda()
    slots = torch.stack([table[0, 1].long() * page + 7, table[1, 28].long() * page + 3])
    ln, cu = i32(lens), i32([0, 40, 940])
    mine = [x.clone() for x in (kc, vc, ks, vs)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    attn.check(attn.attn_kv4_append(new[:, 0], new[:, 1], 2 * H * d, 2 * H * d, slots, 2, H, d, *mine, P, page, "bf16", side))
    o, lse = torch.empty_like(q), torch.empty((2, Hq, 1), device="cuda")
    n = attn.attn_kv4_decode_workspace_size(1, Hq, H, d)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    attn.check(attn.attn_kv4_decode(q, *mine, table, ln, o, lse, 2, 1, Hq, H, d, P, page, width, 0.1, True, "bf16", ws, n, side))
    k, v = (torch.empty((940, H, d), dtype=torch.float16, device="cuda") for _ in range(2))
    attn.check(attn.attn_kv_read(*mine, table, ln, cu, k, v, 2, 940, H, d, P, page, width, 4, "fp16", side))
    side.synchronize()
    attn.kv4_append(new[:, 0], new[:, 1], slots, kc, vc, ks, vs)
    want = (kc, vc, ks, vs, *attn.kv4_decode(q, kc, vc, ks, vs, table, ln, 0.1),
            *attn.kv4_read(kc, vc, ks, vs, table, ln, cu, 940, torch.float16))
    for a, b in zip((*mine, o, lse, k, v), want):
        assert torch.equal(a, b)
    assert torch.isfinite(lse).all()
