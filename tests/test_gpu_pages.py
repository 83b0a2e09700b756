"""Block tables and slot maps on the GPU (attn_pages_extend, attn_pages_release)
against a plain allocator loop; every number equal."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from exact_tiled_attention_22_gb300 import build
    build.build()
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    yield


def extend_ref(lens, add, table, free, count, page, T):
    """The definition, request by request."""
    table = [row[:] for row in table]
    B, width = len(lens), len(table[0])
    new, granted, cu, total, left = [], [], [0], 0, count
    slots = [-1] * T
    for b in range(B):
        ok = lens[b] >= 0 and add[b] >= 0 and -(-(lens[b] + add[b]) // page) <= width
        need = -(-(lens[b] + add[b]) // page) - -(-lens[b] // page) if ok else 0
        total += need
        served = ok and (need == 0 or total <= count)
        if served:
            for k in range(need):
                table[b][-(-lens[b] // page) + k] = free[count - 1 - (total - need + k)]
            left = min(left, count - total) if need else left
            for i in range(add[b]):
                t, pos = cu[-1] + i, lens[b] + i
                if t < T and table[b][pos // page] >= 0:
                    slots[t] = table[b][pos // page] * page + pos % page
        granted.append(add[b] if served else 0)
        new.append(lens[b] + granted[-1])
        cu.append(cu[-1] + max(add[b], 0))
    return new, granted, cu, slots, left, table


def run(lens, add, table, free, count, page, T, in_place=False):
    from exact_tiled_attention_22_gb300 import attn
    i32 = lambda x: torch.tensor(x, dtype=torch.int32).cuda()  # noqa: E731
    ln, cnt, tb = i32(lens), i32([count]), i32(table)
    new, granted, cu, slots, left = attn.pages_extend(
        ln, i32(add), tb, i32(free), cnt, page, T, new_lens=ln if in_place else None,
        free_left=cnt if in_place else None)
    return new.tolist(), granted.tolist(), cu.tolist(), slots.tolist(), left.item(), tb.tolist()


def state(B, hi, page, width, spare, seed):
    """Lengths, a table with distinct pages for them, and a stack of free pages."""
    g = torch.Generator().manual_seed(seed)
    lens = torch.randint(0, hi + 1, (B,), generator=g).tolist()
    pages = torch.randperm(B * width + spare, generator=g).tolist()
    table = []
    for n in lens:
        row = [-1] * width
        for j in range(-(-n // page)):
            row[j] = pages.pop()
        table.append(row)
    return lens, table, pages


@pytest.mark.parametrize("B,hi,add_hi,page,short", [
    (1, 0, 1, 16, False), (1, 100, 1, 64, False), (7, 300, 40, 16, False), (33, 50, 1, 32, True),
    (256, 900, 1, 64, False), (1000, 60, 90, 128, False), (1025, 5, 3, 16, True), (3000, 40, 2, 32, False),
    (40, 100, 2000, 16, True)])
@pytest.mark.parametrize("in_place", [False, True])
def test_extend(B, hi, add_hi, page, short, in_place):
    width = -(-(hi + add_hi) // page)
    lens, table, free = state(B, hi, page, width, 5, seed=B + page)
    add = torch.randint(0, add_hi + 1, (B,), generator=torch.Generator().manual_seed(B)).tolist()
    if B == 1:
        add = [add_hi]
    need = sum(-(-(a + b) // page) - -(-a // page) for a, b in zip(lens, add))
    count = need // 2 if short else min(len(free), need + 3)
    T = sum(add) + 3
    assert run(lens, add, table, free, count, page, T, in_place) == extend_ref(lens, add, table, free, count, page, T)


def test_refused_requests():
    """Negative counts and lengths, rows that are too short, an empty stack, tokens
    past the slot map."""
    table = [[3, -1], [4, 9], [5, -1], [6, -1], [7, 8]]
    lens, add = [16, 32, -1, 5, 20], [1, 1, 4, -2, 2]
    for count in (0, 1, 3):
        for T in (0, 1, 7, 20):
            args = (lens, add, table, [11, 12, 13], count, 16, T)
            assert run(*args) == extend_ref(*args)


def test_release_returns_pages():
    from exact_tiled_attention_22_gb300 import attn
    B, page, width = 300, 16, 6
    lens, table, free = state(B, 90, page, width, 0, seed=9)
    count = 4
    g = torch.Generator().manual_seed(1)
    done = torch.randint(0, 2, (B,), generator=g).tolist()
    want = free[:count]
    for b in range(B):
        if done[b]:
            want += table[b][:-(-lens[b] // page)]
    i32 = lambda x: torch.tensor(x, dtype=torch.int32).cuda()  # noqa: E731
    stack = i32(free[:count] + [-7] * (B * width))
    ln, cnt = i32(lens), i32([count])
    new, left = attn.pages_release(ln, i32(done), i32(table), stack, cnt, page, new_lens=ln, free_left=cnt)
    assert left.item() == len(want) and stack.tolist()[:len(want)] == want
    assert (stack[len(want):] == -7).all()
    assert new.tolist() == [0 if f else n for n, f in zip(lens, done)]
    # a stack that is too small keeps what fits
    small = i32(free[:count] + [-7] * 3)
    _, left = attn.pages_release(i32(lens), i32(done), i32(table), small, i32([count]), page)
    assert left.item() == count + 3 and small.tolist() == want[:count + 3]


def test_extend_in_a_graph():
    """A captured step that updates lengths and stack in place: each replay is the
    next step."""
    from exact_tiled_attention_22_gb300 import attn
    B, page, width = 5, 16, 4
    lens, table, free = state(B, 20, page, width, 0, seed=2)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32).cuda()  # noqa: E731
    ln, tb, st, cnt, add = i32(lens), i32(table), i32(free), i32([len(free)]), i32([1] * B)
    start = [x.clone() for x in (ln, tb, cnt)]
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        attn.pages_extend(ln, add, tb, st, cnt, page, B, new_lens=ln, free_left=cnt)
    side.synchronize()
    for x, y in zip((ln, tb, cnt), start):
        x.copy_(y)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        _, _, _, slots, _ = attn.pages_extend(ln, add, tb, st, cnt, page, B, new_lens=ln, free_left=cnt)
    count = len(free)
    for _ in range(30):
        lens, _, _, want, count, table = extend_ref(lens, [1] * B, table, free, count, page, B)
        graph.replay()
        torch.cuda.synchronize()
        assert (ln.tolist(), slots.tolist(), cnt.item(), tb.tolist()) == (lens, want, count, table)


@pytest.mark.parametrize("B", [1023, 1024, 1025, 3000, 8192])
@pytest.mark.parametrize("in_place", [False, True])
def test_release_of_many(B, in_place):
    """Around one pass of the block's threads and far beyond, lengths past the table's row
    and negative ones among them."""
    from exact_tiled_attention_22_gb300 import attn
    page, width, count = 16, 3, 7
    g = torch.Generator().manual_seed(B)
    lens = torch.randint(-2, page * width + 20, (B,), generator=g).tolist()
    done = torch.randint(0, 3, (B,), generator=g).tolist()   # any number but 0 is a yes
    table = torch.randperm(B * width, generator=g).view(B, width).tolist()
    want = list(range(-count, 0))
    for b in range(B):
        if done[b]:
            want += table[b][:max(0, min(width, -(-lens[b] // page)))]
    i32 = lambda x: torch.tensor(x, dtype=torch.int32).cuda()  # noqa: E731
    for cap in (count + B * width, len(want), len(want) - 5):
        stack = i32((want[:count] + [-7] * cap)[:cap])
        ln, cnt = i32(lens), i32([count])
        new, left = attn.pages_release(ln, i32(done), i32(table), stack, cnt, page, new_lens=ln if in_place else None,
                                       free_left=cnt if in_place else None)
        kept = want[:cap]
        assert left.item() == len(kept) and stack.tolist() == kept + [-7] * (cap - len(kept))
        assert new.tolist() == [0 if f else n for n, f in zip(lens, done)]
