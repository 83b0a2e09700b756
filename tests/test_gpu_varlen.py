"""Packed sequences (attn_varlen_fwd, attn_varlen_bwd) against attention written
out in 64 bits, element by element within derived bounds (plain64.py): lengths
around the tile sizes, empty sequences, queries without keys and keys without
queries, grouped heads, strided inputs, neighbours full of NaN."""
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


def cu(lens):
    return [0] + torch.tensor(lens).cumsum(0).tolist()


def draw(lens_q, lens_k, Hq, H, d, dtype, seed, extra=0):
    g = torch.Generator().manual_seed(seed)
    Tq, Tk = sum(lens_q) + extra, sum(lens_k) + extra
    mk = lambda t, h: torch.randn((t, h, d), generator=g).to(DT[dtype])  # noqa: E731
    return mk(Tq, Hq), mk(Tk, H), mk(Tk, H), mk(Tq, Hq)


def dev(x):
    return x.cuda()


def offsets(lens):
    return torch.tensor(cu(lens), dtype=torch.int32).cuda()


CASES = [
    # (lens_q, lens_k, Hq, Hkv, d, dtype, causal)
    ([1], [1], 1, 1, 64, "fp16", True),
    ([1, 1, 1], [1, 5, 129], 2, 1, 128, "bf16", True),
    ([127, 128, 129], [127, 128, 129], 2, 2, 64, "bf16", True),
    ([255, 1, 257, 0, 63], [255, 1, 257, 0, 63], 4, 1, 128, "fp16", True),
    ([300, 0, 5, 64], [300, 17, 0, 200], 3, 1, 64, "fp16", True),
    ([300, 0, 5, 64], [300, 17, 0, 200], 3, 3, 128, "bf16", False),
    ([130, 7], [20, 500], 4, 2, 64, "bf16", True),      # more queries than keys; a prefix
    ([640], [640], 16, 2, 128, "bf16", True),
    ([513, 70], [1025, 1000], 5, 5, 64, "fp16", True),
    ([200, 385], [129, 640], 6, 2, 128, "fp16", False),
    ([65], [300], 7, 1, 64, "bf16", True),
]
IDS = [f"{i}-{c[2]}x{c[3]}d{c[4]}{c[5]}{'c' if c[6] else ''}" for i, c in enumerate(CASES)]


@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_forward_and_gradients(case):
    from exact_tiled_attention_22_gb300 import attn
    lens_q, lens_k, Hq, H, d, dtype, causal = case
    q, k, v, do = draw(lens_q, lens_k, Hq, H, d, dtype, seed=sum(lens_q))
    scale = d ** -0.5
    cq, ck = offsets(lens_q), offsets(lens_k)
    o, lse = attn.varlen_fwd(dev(q), dev(k), dev(v), cq, ck, scale, causal)
    grads = attn.varlen_bwd(dev(q), dev(k), dev(v), o, lse, dev(do), cq, ck, scale, causal)
    attn.check(attn.attn_status())
    ref = plain64.packed(q.double(), k.double(), v.double(), cu(lens_q), cu(lens_k), scale, causal, dtype, do.double())
    for name, got in zip(("o", "lse", "dq", "dk", "dv"), (o, lse, *grads)):
        plain64.check(got, *ref[name], name)


@pytest.mark.parametrize("first", [0, 5])
def test_nothing_but_padding(first):
    """Offsets that begin behind row 0, and batches whose sequences are all empty:
    rows of no sequence keep what they held."""
    from exact_tiled_attention_22_gb300 import attn
    q, k, v, do = draw([40], [40], 4, 2, 64, "fp16", seed=70)
    for ends in ([first, first, first], [first, first + 3, first + 30]):
        c = torch.tensor(ends, dtype=torch.int32).cuda()
        marks = [torch.full(x.shape, 7.0, dtype=x.dtype, device="cuda") for x in (q, q, k, v)]
        o, lse = attn.varlen_fwd(dev(q), dev(k), dev(v), c, c, 0.125, True, o=marks[0])
        grads = attn.varlen_bwd(dev(q), dev(k), dev(v), o, lse, dev(do), c, c, 0.125, True, grads=marks[1:])
        attn.check(attn.attn_status())
        for x in (o, *grads):
            assert (x[:ends[0]] == 7.0).all() and (x[ends[-1]:] == 7.0).all()
        if ends[-1] > ends[0]:
            s = slice(ends[0], ends[-1])
            cut = [e - ends[0] for e in ends]
            ref = plain64.packed(*(x[s].double() for x in (q, k, v)), cut, cut, 0.125, True, "fp16", do[s].double())
            for name, got in zip(("o", "dq", "dk", "dv"), (o, *grads)):
                plain64.check(got[s], *ref[name], name)
            plain64.check(lse[:, s], *ref["lse"], "lse")


def test_offsets_that_do_not_ascend_stay_inside():
    """Outputs are unspecified, but nothing outside the given tensors is written
    and the next call is right."""
    from exact_tiled_attention_22_gb300 import attn
    q, k, v, do = (x.cuda() for x in draw([300], [300], 4, 2, 64, "bf16", seed=71))
    for ends in ([0, 300, 10, 290, 300], [-50, 5000, 2, 300, -1], [300, 200, 100, 0, 0], [0, 300, 0, 300, 300]):
        c = torch.tensor(ends, dtype=torch.int32).cuda()
        room = [torch.full((400, x.shape[1], 64), 7.0, dtype=x.dtype, device="cuda") for x in (q, q, k, v)]
        o, lse = attn.varlen_fwd(q, k, v, c, c, 0.125, True, o=room[0][50:350])
        attn.varlen_bwd(q, k, v, o, lse, do, c, c, 0.125, True, grads=[x[50:350] for x in room[1:]])
        attn.check(attn.attn_status())
        for x in room:
            assert (x[:50] == 7.0).all() and (x[350:] == 7.0).all()
    c = offsets([300])
    o, lse = attn.varlen_fwd(q, k, v, c, c, 0.125, True)
    ref = plain64.packed(*(x.double().cpu() for x in (q, k, v)), [0, 300], [0, 300], 0.125, True, "bf16")
    plain64.check(o, *ref["o"], "o")


def test_many_short_sequences():
    """More sequences than a warp and than a block of the scans, zeros among them."""
    from exact_tiled_attention_22_gb300 import attn
    g = torch.Generator().manual_seed(3)
    lens = torch.randint(0, 7, (700,), generator=g).tolist()
    q, k, v, do = draw(lens, lens, 2, 1, 64, "fp16", seed=4)
    c = offsets(lens)
    o, lse = attn.varlen_fwd(dev(q), dev(k), dev(v), c, c, 0.125, True)
    grads = attn.varlen_bwd(dev(q), dev(k), dev(v), o, lse, dev(do), c, c, 0.125, True)
    ref = plain64.packed(q.double(), k.double(), v.double(), cu(lens), cu(lens), 0.125, True, "fp16", do.double())
    for name, got in zip(("o", "lse", "dq", "dk", "dv"), (o, lse, *grads)):
        plain64.check(got, *ref[name], name)


@pytest.mark.parametrize("d,group", [(64, 2), (128, 3)])
def test_neighbours_and_padding_do_not_leak(d, group):
    """Sequences between others full of NaN and infinities, rows behind the last
    sequence left as they were."""
    from exact_tiled_attention_22_gb300 import attn
    lens = [70, 129, 200, 33]
    extra = 50
    q, k, v, do = draw(lens, lens, group, 1, d, "bf16", seed=11, extra=extra)
    c = cu(lens)
    for i, bad in ((0, math.nan), (2, math.inf)):
        for x in (q, k, v, do):
            x[c[i]:c[i + 1]] = bad
    for x in (q, k, v, do):
        x[c[-1]:] = math.nan
    cg = offsets(lens)
    marks = [torch.full(x.shape, 7.0, dtype=q.dtype, device="cuda") for x in (q, q, k, v)]
    o, lse = attn.varlen_fwd(dev(q), dev(k), dev(v), cg, cg, d ** -0.5, True, o=marks[0])
    # (lse comes from an uninitialised buffer: rows of no sequence are not read)
    grads = attn.varlen_bwd(dev(q), dev(k), dev(v), o, lse, dev(do), cg, cg, d ** -0.5, True, grads=marks[1:])
    attn.check(attn.attn_status())
    for x in (o, *grads):
        assert (x[c[-1]:] == 7.0).all()
    zero = lambda x: torch.nan_to_num(x.double(), 0.0, 0.0, 0.0)  # noqa: E731
    ref = plain64.packed(zero(q), zero(k), zero(v), c, c, d ** -0.5, True, "bf16", zero(do))
    for name, got in zip(("o", "lse", "dq", "dk", "dv"), (o, lse, *grads)):
        for i in (1, 3):
            s = slice(c[i], c[i + 1])
            val, bound = ref[name]
            if name == "lse":
                plain64.check(got[:, s], val[:, s], bound[:, s], f"{name} of sequence {i}")
            else:
                plain64.check(got[s], val[s], bound[s], f"{name} of sequence {i}")


@pytest.mark.parametrize("d", [64, 128])
def test_slices_of_one_projection(d):
    """q, k, v as slices of one [T, Hq + 2 Hkv, d] tensor: bit-equal to copies."""
    from exact_tiled_attention_22_gb300 import attn
    lens = [100, 300, 1]
    g = torch.Generator().manual_seed(5)
    x = torch.randn((sum(lens), 6 + 4, d), generator=g).half().cuda()
    q, k, v = x[:, :6], x[:, 6:8], x[:, 8:]
    do = torch.randn((sum(lens), 6, d), generator=g).half().cuda()
    c = offsets(lens)
    o, lse = attn.varlen_fwd(q, k, v, c, c, None, True)
    o2, lse2 = attn.varlen_fwd(q.contiguous(), k.contiguous(), v.contiguous(), c, c, None, True)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    _, dk, dv = attn.varlen_bwd(q, k, v, o, lse, do, c, c, None, True)
    _, dk2, dv2 = attn.varlen_bwd(q.contiguous(), k.contiguous(), v.contiguous(), o, lse, do, c, c, None, True)
    assert torch.equal(dk, dk2) and torch.equal(dv, dv2)


def test_equals_the_batched_forward():
    """Sequences of one length are the [B, N, H, d] call's batch (both within
    their own rounding)."""
    from exact_tiled_attention_22_gb300 import attn
    B, N, H, d = 3, 384, 4, 128
    g = torch.Generator().manual_seed(6)
    q, k, v = (torch.randn((B, N, H, d), generator=g).bfloat16().cuda() for _ in range(3))
    o, lse = attn.fwd(q, k, v, None, True)
    c = offsets([N] * B)
    o2, lse2 = attn.varlen_fwd(q.view(-1, H, d), k.view(-1, H, d), v.view(-1, H, d), c, c, None, True)
    assert (lse2.view(H, B, N).transpose(0, 1) - lse).abs().max() <= 2.0 ** -16 * (1 + lse.abs().max())
    top = v.float().abs().max()
    assert (o2.view(B, N, H, d).float() - o.float()).abs().max() <= 2 * 2 * 2.0 ** -8 * top


def test_autograd_and_differences():
    """attention_varlen's gradients against directional differences of the
    64-bit formula, and zeros for rows of no sequence."""
    from exact_tiled_attention_22_gb300 import attn
    lens_q, lens_k, Hq, H, d = [60, 131], [75, 131], 4, 2, 64
    q, k, v, w = draw(lens_q, lens_k, Hq, H, d, "fp16", seed=21, extra=9)
    cq, ck = cu(lens_q), cu(lens_k)
    scale = 0.125
    a = [dev(x).requires_grad_() for x in (q, k, v)]
    o = attn.attention_varlen(*a, offsets(lens_q), offsets(lens_k), scale, True)
    o.backward(dev(w))
    for x, n in zip(a, (cq[-1], ck[-1], ck[-1])):
        assert (x.grad[n:] == 0).all()
    assert (o[cq[-1]:] == 0).all()

    def loss(q, k, v):
        r = plain64.packed(q, k, v, cq, ck, scale, True, "fp16")["o"][0]
        return (r[:cq[-1]] * w.double()[:cq[-1]]).sum().item()

    ref = plain64.packed(q.double(), k.double(), v.double(), cq, ck, scale, True, "fp16", w.double())
    g = torch.Generator().manual_seed(8)
    for i, name in enumerate(("dq", "dk", "dv")):
        base = [x.double() for x in (q, k, v)]
        step = torch.randn(base[i].shape, generator=g, dtype=torch.float64)
        step[(cq if i == 0 else ck)[-1]:] = 0
        h = 1e-4
        lo, hi = list(base), list(base)
        lo[i], hi[i] = base[i] - h * step, base[i] + h * step
        slope = (loss(*hi) - loss(*lo)) / (2 * h)
        got = (a[i].grad.double().cpu() * step).sum().item()
        # the gradient's own bound along the step, and the difference's h^2 term
        tol = (torch.nan_to_num(ref[name][1]) * step.abs()).sum().item() + 1e-3
        assert abs(got - slope) <= tol, (name, got, slope, tol)


def test_captured_and_on_another_stream():
    """Forward and backward captured into a graph on a side stream, replayed on
    other values AND other lengths (both live on the device)."""
    from exact_tiled_attention_22_gb300 import attn
    T, Hq, H, d = 500, 4, 2, 64
    lens = [[100, 150, 250], [3, 497, 0]]
    xs = [draw(l, l, Hq, H, d, "bf16", seed=30 + i) for i, l in enumerate(lens)]
    q, k, v, do = (x.cuda() for x in xs[0])
    c = offsets(lens[0])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    ws = torch.empty(attn.attn_varlen_bwd_workspace_size(3, T, Hq, H, d), dtype=torch.uint8, device="cuda")

    def step():
        o, lse = attn.varlen_fwd(q, k, v, c, c, 0.125, True)
        return (o, lse, *attn.varlen_bwd(q, k, v, o, lse, do, c, c, 0.125, True, ws=ws))

    with torch.cuda.stream(side):
        step()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        out = step()
    for i in (1, 0):
        for t, x in zip((q, k, v, do), xs[i]):
            t.copy_(x.cuda())
        c.copy_(offsets(lens[i]))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        ref = plain64.packed(*(x.double() for x in xs[i][:3]), cu(lens[i]), cu(lens[i]), 0.125, True, "bf16",
                             xs[i][3].double())
        for name, got in zip(("o", "lse", "dq", "dk", "dv"), out):
            plain64.check(got, *ref[name], name)
    assert attn.attn_status() == 0


SPLIT = [
    # long enough that key tiles are cut into several items: at the causal limit,
    # in a prefix (more keys than queries), without a mask; odd numbers of steps
    ([4500], [4500], 1, 1, 64, "fp16", True),
    ([2300, 100, 1100], [2300, 100, 1100], 8, 1, 128, "bf16", True),
    ([1900, 333], [3500, 2000], 6, 2, 64, "bf16", True),
    ([1665, 40], [1500, 700], 4, 1, 128, "fp16", False),
    ([2113], [1000], 3, 1, 64, "bf16", True),
]


@pytest.mark.parametrize("case", SPLIT, ids=lambda c: f"{c[0][0]}-{c[2]}x{c[3]}d{c[4]}{c[5]}{'c' if c[6] else ''}")
def test_split_key_tiles(case):
    """Gradients of batches whose key tiles are shared by several work items, with
    a workspace full of NaN."""
    from exact_tiled_attention_22_gb300 import attn
    lens_q, lens_k, Hq, H, d, dtype, causal = case
    q, k, v, do = draw(lens_q, lens_k, Hq, H, d, dtype, seed=sum(lens_q))
    cq, ck = offsets(lens_q), offsets(lens_k)
    n = attn.attn_varlen_bwd_workspace_size(len(lens_q), sum(lens_q), Hq, H, d)
    ws = torch.full((n // 4 + 1,), math.nan, device="cuda").view(torch.uint8)
    o, lse = attn.varlen_fwd(dev(q), dev(k), dev(v), cq, ck, None, causal)
    grads = attn.varlen_bwd(dev(q), dev(k), dev(v), o, lse, dev(do), cq, ck, None, causal, ws=ws)
    attn.check(attn.attn_status())
    ref = plain64.packed(q.double(), k.double(), v.double(), cu(lens_q), cu(lens_k), d ** -0.5, causal, dtype,
                         do.double())
    for name, got in zip(("o", "lse", "dq", "dk", "dv"), (o, lse, *grads)):
        plain64.check(got, *ref[name], name)


SHARED = [
    # few queries on many keys: several blocks share the key range of a query tile
    ([64], [2400], 12, 4, 64, "fp16", True),
    ([1, 30], [3000, 1500], 3, 1, 128, "bf16", True),
    ([300], [5000], 2, 2, 128, "fp16", True),
    ([200, 5, 0], [1100, 4000, 30], 5, 1, 64, "bf16", False),
    ([1500], [1100], 1, 1, 64, "bf16", True),   # queries that see none of the keys
]


@pytest.mark.parametrize("case", SHARED, ids=lambda c: f"{c[0][0]}on{c[1][0]}-{c[2]}x{c[3]}d{c[4]}{c[5]}{'c' if c[6] else ''}")
def test_shared_key_ranges(case):
    from exact_tiled_attention_22_gb300 import attn
    lens_q, lens_k, Hq, H, d, dtype, causal = case
    q, k, v, _ = draw(lens_q, lens_k, Hq, H, d, dtype, seed=sum(lens_k))
    n = attn.attn_varlen_fwd_workspace_size(len(lens_q), sum(lens_q), sum(lens_k), Hq, H, d)
    assert n > 0
    ws = torch.full((n // 4,), math.nan, device="cuda").view(torch.uint8)
    o, lse = attn.varlen_fwd(dev(q), dev(k), dev(v), offsets(lens_q), offsets(lens_k), None, causal, ws=ws)
    attn.check(attn.attn_status())
    ref = plain64.packed(q.double(), k.double(), v.double(), cu(lens_q), cu(lens_k), d ** -0.5, causal, dtype)
    plain64.check(o, *ref["o"], "o")
    plain64.check(lse, *ref["lse"], "lse")


def test_repeats_are_equal():
    """O, LSE, dK, dV do not depend on the order in which blocks finish."""
    from exact_tiled_attention_22_gb300 import attn
    lens = [3900, 40, 333]
    q, k, v, do = (x.cuda() for x in draw(lens, lens, 8, 2, 128, "bf16", seed=40))
    c = offsets(lens)
    first = None
    for _ in range(3):
        o, lse = attn.varlen_fwd(q, k, v, c, c, None, True)
        _, dk, dv = attn.varlen_bwd(q, k, v, o, lse, do, c, c, None, True)
        now = (o, lse, dk, dv)
        assert first is None or all(torch.equal(a, b) for a, b in zip(first, now))
        first = now


def test_wait_limit_reports_a_timeout():
    """A load warp that holds back its copies: the waits run out, the call
    returns, attn_status says so, and the next call is right again."""
    from exact_tiled_attention_22_gb300 import attn
    lens = [200]
    q, k, v, do = (x.cuda() for x in draw(lens, lens, 2, 1, 64, "fp16", seed=50))
    c = offsets(lens)
    o, lse = attn.varlen_fwd(q, k, v, c, c, None, True)
    attn.check(attn.attn_status())
    try:
        attn.attn_set_wait_limit(50_000_000, 1)
        attn.varlen_fwd(q, k, v, c, c, None, True)
        assert attn.attn_status() == attn.ATTN_ERR_TIMEOUT
        attn.attn_set_wait_limit(50_000_000, 2)
        attn.varlen_bwd(q, k, v, o, lse, do, c, c, None, True)
        assert attn.attn_status() == attn.ATTN_ERR_TIMEOUT
    finally:
        attn.attn_set_wait_limit(0, 0)
    o2, lse2 = attn.varlen_fwd(q, k, v, c, c, None, True)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


@pytest.mark.parametrize("lens_q,lens_k", [([70, 40], [70, 40]), ([5, 64], [2000, 1500])])
def test_not_numbers_reach_their_rows_only(lens_q, lens_k):
    """A NaN query has a NaN row of O and of LSE, a NaN key those of the queries
    that see it (causal), whether a pair of tiles is one block's or several share it;
    all other rows keep their bits."""
    from exact_tiled_attention_22_gb300 import attn
    Hq, H, d = 4, 2, 64
    q, k, v, _ = draw(lens_q, lens_k, Hq, H, d, "bf16", seed=40)
    clean, clean_lse = attn.varlen_fwd(q.cuda(), k.cuda(), v.cuda(), offsets(lens_q), offsets(lens_k), None, True)
    q[2, 1, 5] = math.nan                      # query 2 of sequence 0, head 1
    hidden = 7                                 # the key that the last 7 queries of sequence 1 see
    k[sum(lens_k) - hidden, 1, 9] = math.nan   # key head 1: query heads 2, 3
    o, lse = attn.varlen_fwd(q.cuda(), k.cuda(), v.cuda(), offsets(lens_q), offsets(lens_k), None, True)
    bad = torch.zeros(sum(lens_q), Hq, dtype=torch.bool)
    bad[2, 1] = True
    bad[sum(lens_q) - hidden:, 2:] = True
    bad = bad.cuda()
    assert torch.equal(torch.isnan(o).all(-1), bad) and torch.equal(torch.isnan(o).any(-1), bad)
    assert torch.equal(torch.isnan(lse), bad.t())
    assert torch.equal(o[~bad], clean[~bad]) and torch.equal(lse[~bad.t()], clean_lse[~bad.t()])
    assert attn.attn_status() == 0


def test_a_captured_training_step():
    """attention_varlen and its backward captured together, replayed on other
    values and lengths: the eager results (dQ is summed in no fixed order)."""
    from exact_tiled_attention_22_gb300 import attn
    Hq, H, d, T = 4, 2, 128, 300
    lens = [[100, 150, 50], [3, 290, 0]]       # the second leaves seven rows of padding
    xs = [draw([T], [T], Hq, H, d, "bf16", seed=50 + i) for i in range(2)]
    q, k, v = (x.cuda().requires_grad_() for x in xs[0][:3])
    w = xs[0][3].cuda()
    c = offsets(lens[0])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())

    def step():
        o = attn.attention_varlen(q, k, v, c, c, None, True)
        return (o, *torch.autograd.grad(o, (q, k, v), w))

    with torch.cuda.stream(side):
        step()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        out = [x.detach() for x in step()]
    for i in (1, 0):
        with torch.no_grad():
            for t, x in zip((q, k, v, w), xs[i]):
                t.copy_(x.cuda())
        c.copy_(offsets(lens[i]))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        got = [x.clone() for x in out]
        want = [x.detach() for x in step()]
        assert torch.equal(got[0], want[0]) and torch.equal(got[2], want[2]) and torch.equal(got[3], want[3])
        # |dQ|: two fp32 sums of the same terms in different orders, then one bf16 rounding each
        assert (got[1].float() - want[1].float()).abs().max() <= 2.0 ** -7 * want[1].float().abs().max()
        n = sum(lens[i])
        for x in got:
            assert (x[n:] == 0).all()
    assert attn.attn_status() == 0


@pytest.mark.parametrize("B", [64, 65, 256, 257, 300, 513])
def test_searches_over_many_sequences(B):
    """Around the places where the search for a block's sequence changes its width:
    queries, keys or both missing in some, the last ones among them."""
    from exact_tiled_attention_22_gb300 import attn
    g = torch.Generator().manual_seed(B)
    lq = torch.randint(0, 40, (B,), generator=g)
    lk = torch.randint(0, 40, (B,), generator=g)
    lq[torch.rand(B, generator=g) < 0.3] = 0
    lk[torch.rand(B, generator=g) < 0.2] = 0
    lq[-1], lk[-1], lq[0] = 5, 9, 0
    lq, lk = lq.tolist(), lk.tolist()
    q, k, v, do = draw(lq, lk, 2, 2, 64, "bf16", seed=60)
    o, lse = attn.varlen_fwd(dev(q), dev(k), dev(v), offsets(lq), offsets(lk), 0.125, True)
    grads = attn.varlen_bwd(dev(q), dev(k), dev(v), o, lse, dev(do), offsets(lq), offsets(lk), 0.125, True)
    ref = plain64.packed(q.double(), k.double(), v.double(), cu(lq), cu(lk), 0.125, True, "bf16", do.double())
    for name, got in zip(("o", "lse", "dq", "dk", "dv"), (o, lse, *grads)):
        plain64.check(got, *ref[name], name)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Hq,H", [(1, 1), (3, 1)])
def test_whole_query_tiles_without_keys(Hq, H, d):
    """256 queries on 100 keys, causal, where a tile is 128 positions of one head: the
    first tile of every pair sees nothing while the second one does.  Its rows are
    zeros in every sequence and every time, whenever its queries arrive."""
    from exact_tiled_attention_22_gb300 import attn
    B, lq, lk = 200, 256, 100
    q, k, v, _ = draw([lq] * B, [lk] * B, Hq, H, d, "bf16", seed=d + Hq)
    cq, ck = offsets([lq] * B), offsets([lk] * B)
    q, k, v = q.cuda(), k.cuda(), v.cuda()
    first = None
    for _ in range(20):
        o, lse = attn.varlen_fwd(q, k, v, cq, ck, None, True)
        assert (o.view(B, lq, Hq, d)[:, :lq - lk] == 0).all()
        assert (lse.view(Hq, B, lq)[:, :, :lq - lk] == -math.inf).all()
        assert first is None or (torch.equal(o, first[0]) and torch.equal(lse, first[1]))
        first = (o, lse)
    attn.check(attn.attn_status())
    n = 3  # sequences in 64 bits
    ref = plain64.packed(q[:n * lq].double().cpu(), k[:n * lk].double().cpu(), v[:n * lk].double().cpu(),
                         cu([lq] * n), cu([lk] * n), d ** -0.5, True, "bf16")
    plain64.check(o[:n * lq], *ref["o"], "o")
    plain64.check(lse[:, :n * lq], *ref["lse"], "lse")


GROUPS = [
    # (lens_q, lens_k, Hq, Hkv, d, dtype, causal): groups above 8, with a ragged first tile.  A
    # batch of 128 queries or more a sequence takes tiles of the largest power of two in
    # the group (48: 16 heads of 8 positions), a shorter one the whole group (48: 2 positions)
    ([300, 40], [300, 40], 16, 1, 64, "bf16", True),
    ([70, 33], [70, 51], 32, 2, 128, "fp16", True),
    ([150, 130], [150, 259], 48, 1, 64, "fp16", True),
    ([21, 90], [130, 90], 48, 1, 128, "bf16", False),
    ([200], [333], 64, 1, 128, "bf16", True),
    ([150, 129], [150, 129], 65, 1, 64, "bf16", True),
    ([60, 5, 30], [60, 200, 1], 65, 1, 128, "fp16", True),
    ([20, 90], [20, 300], 127, 1, 64, "bf16", False),
    ([140, 3], [140, 3], 128, 1, 128, "fp16", True),
    ([130, 3], [260, 3], 256, 1, 64, "bf16", True),
    ([135], [70], 256, 1, 128, "bf16", True),       # the first tiles see no key
    # few keys: one key tile of many steps, which are cut into chunks
    ([6000], [128], 2, 2, 64, "bf16", False),
    ([3100, 5], [100, 260], 32, 1, 64, "fp16", False),
]


@pytest.mark.parametrize("case", GROUPS, ids=lambda c: f"{c[0][0]}on{c[1][0]}-{c[2]}x{c[3]}d{c[4]}{c[5]}{'c' if c[6] else ''}")
def test_large_groups(case):
    test_forward_and_gradients(case)
